// The gradient of the router's balance loss (balance.cuh says what is computed).
//
// A CTA takes a stretch of rows; the g of the sequence it is in lie in shared memory, a row is read, turned into its gradient in
// registers and written by 8, 16 or 32 lanes.  4096 x 128 FP32 4.5 us; 65537 x 250, sigmoid, in 37 sequences, a tenth of the tokens
// masked, 32 us, 131 MB at 4.1 TB/s (65536 x 256 without masks 31, softmax 29): 350 warp instructions a row at 24 warps an SM, whose
// latency the loads of one row ahead do not cover.  20000 x 1000 BF16 28 us with two CTAs to an SM, 38 with one.
#include "balance.cuh"

namespace nvfp4 {
namespace balance {
namespace {

template <typename T, int kPer, int kLanes, int kN, bool kSigmoid>
__global__ void __launch_bounds__(kThreads, kPer <= 16 ? 3 : 2)
    backward_kernel(const T* __restrict__ logits, const BalanceParams p, int64_t rows_per_cta, const int32_t* __restrict__ counts,
                    const int32_t* __restrict__ tokens, const float* __restrict__ dloss, T* __restrict__ dl, int64_t ld_out,
                    int accumulate) {
    constexpr int kStep = kThreads / kLanes;
    __shared__ __align__(16) float s_g[kPer * kLanes];
    const int sub = threadIdx.x % kLanes, E = p.E;
    const int64_t end = min((static_cast<int64_t>(blockIdx.x) + 1) * rows_per_cta, p.T);
    int64_t row = static_cast<int64_t>(blockIdx.x) * rows_per_cta, s = find_sequence(p.offsets, p.S, row);
    while (row < end) {
        // rows [row, stop) of sequence s, or of none
        int64_t stop = end;
        const bool inside = s >= 0 && s < p.S;
        if (p.offsets != nullptr && s < p.S) stop = min(end, static_cast<int64_t>(p.offsets[s + 1]));
        if (stop <= row) {                                  // empty, as any number behind it may be
            s = max(s + 1, find_sequence(p.offsets, p.S, row));
            continue;
        }
        __syncthreads();                                    // the last sequence's are used up
        if (inside) {
            const float n = static_cast<float>(tokens[s]);
            const float scale = n > 0.0f ? dloss[s] * (static_cast<float>(E) / (static_cast<float>(p.k) * n * n)) : 0.0f;
            for (int e = threadIdx.x; e < kPer * kLanes; e += kThreads) s_g[e] = e < E ? scale * static_cast<float>(counts[s * E + e]) : 0.0f;
        }
        __syncthreads();
        int64_t t = row + threadIdx.x / kLanes;
        float next[kPer];                 // the next row's logits are on their way while a row is worked on
        bool next_real;
        const auto fetch = [&](int64_t at) {
            next_real = at < stop && inside && (p.mask == nullptr || p.mask[at] != 0);
            if (next_real) {
                load_row<T, kPer, kLanes, kN>(logits + at * p.ld, E, sub, next);
            } else {
#pragma unroll
                for (int i = 0; i < kPer; ++i) next[i] = 0.0f;   // takes no warp out of its way
            }
        };
        fetch(t);
        for (int64_t base = row; base < stop; base += kStep, t += kStep) {
            float v[kPer], rest[kSigmoid ? kPer : 1];
#pragma unroll
            for (int i = 0; i < kPer; ++i) v[i] = next[i];
            const bool real = next_real;
            if (base + kStep < stop) fetch(t + kStep);
            bool bad;
            const float r = row_terms<kPer, kLanes, kSigmoid>(kSigmoid ? MOE_SCORE_SIGMOID : MOE_SCORE_SOFTMAX, v, rest, bad);
            if (bad) set_device_error(p.err, NVFP4_ERR_NONFINITE);
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < kPer; i += kN) {
#pragma unroll
                for (int j = 0; j < kN; ++j) {
                    v[i + j] *= r;
                    dot = fmaf(s_g[expert_of<kLanes, kN>(i, sub) + j], v[i + j], dot);
                }
            }
            dot = lanes_sum<kLanes>(dot);
            if (t >= stop || (accumulate && !real)) continue;
            T* out = dl + t * ld_out;
#pragma unroll
            for (int i = 0; i < kPer; i += kN) {
                const int e = expert_of<kLanes, kN>(i, sub);
                if (e >= E) continue;
                float d[kN];
#pragma unroll
                for (int j = 0; j < kN; ++j) {
                    d[j] = v[i + j] * (s_g[e + j] - dot);
                    if (kSigmoid) d[j] *= rest[i + j];
                    if (!real) d[j] = 0.0f;
                }
                if (accumulate) {
                    Vec<T, kN> was;
                    was.word = *reinterpret_cast<const decltype(was.word)*>(out + e);
#pragma unroll
                    for (int j = 0; j < kN; ++j) d[j] += to_f32(was.e[j]);
                }
                store_vec<T, kN>(out + e, d);
            }
        }
        row = stop;
        ++s;
    }
}

template <typename T>
cudaError_t backward(const void* logits, const BalanceParams& p, const int32_t* counts, const int32_t* tokens,
                     const float* dloss, void* dl, int64_t ld_out, bool accumulate, cudaStream_t st) {
    const int in = load_width<T>(logits, p.ld, p.E), out = load_width<T>(dl, ld_out, p.E);
    return by_experts(p.E, [&](auto per, auto lanes) {
        return by_width<T>(in < out ? in : out, [&](auto width) {
            constexpr int kPer = decltype(per)::value, kLanes = decltype(lanes)::value, kN = decltype(width)::value;
            constexpr int64_t kRows = kThreads / kLanes;    // of a CTA at a time
            auto* kernel = p.score == MOE_SCORE_SOFTMAX ? backward_kernel<T, kPer, kLanes, kN, false>
                                                        : backward_kernel<T, kPer, kLanes, kN, true>;
            // turns of a CTA: all of them run at once (of 65537 x 250, 683 CTAs in a wave and a half took 36 us)
            const int64_t at_once = kRows * (kPer <= 16 ? 3 : 2) * device_sm_count();
            const int64_t turns = (p.T + at_once - 1) / at_once;
            const int64_t rows = turns * kRows;
            return launch_pdl(false, kernel, dim3(static_cast<unsigned>((p.T + rows - 1) / rows)), dim3(kThreads), 0, st,
                              static_cast<const T*>(logits), p, rows, counts, tokens, dloss, static_cast<T*>(dl), ld_out,
                              accumulate ? 1 : 0);
        });
    });
}

}  // namespace
}  // namespace balance

cudaError_t launch_balance_loss_backward(const void* logits, int type, const BalanceArgs& a, const int32_t* counts,
                                         const int32_t* tokens, const float* dloss, void* dl, int64_t ld_out, bool accumulate,
                                         int* err, cudaStream_t st) {
    using namespace balance;
    const BalanceParams p = {a.T, a.E, a.ld, a.score, a.k, a.ids, a.mask, a.offsets, a.S, err};
    switch (type) {
        case NVFP4_TYPE_F32: return backward<float>(logits, p, counts, tokens, dloss, dl, ld_out, accumulate, st);
        case NVFP4_TYPE_BF16: return backward<__nv_bfloat16>(logits, p, counts, tokens, dloss, dl, ld_out, accumulate, st);
        default: return backward<__half>(logits, p, counts, tokens, dloss, dl, ld_out, accumulate, st);
    }
}

}  // namespace nvfp4
