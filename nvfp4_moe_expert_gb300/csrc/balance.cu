// The router's balance loss over packed sequences, with per-expert counts, and its gradient.
//
//   p_te = softmax(l_t)_e, or sigmoid(l_te) / sum_j sigmoid(l_tj); 0 for a masked expert (l = -inf or NaN)
//   of the n tokens of a sequence that are not masked:  c_e = slots that chose e,  P_e = 1/n sum_t p_te
//   loss = E / (k n) sum_e c_e P_e
//   with g_e = dloss E c_e / (k n^2):  softmax  dl_te = p_te (g_e - sum_j g_j p_tj)
//                                      sigmoid  dl_te = p_te (1 - s_te) (g_e - sum_j g_j p_tj),  s the sigmoid
//
// A token is taken by 8, 16 or 32 lanes, so that a lane has at most 16 experts (32 of more than 512).
#include "cluster.cuh"
#include "common.cuh"
#include "ops.cuh"
#include "scores.cuh"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kSplit = 8;                 // CTAs (one cluster) that share a sequence

template <int kLanes>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
template <int kLanes>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

// Expert of a lane's i-th element, with loads of kN elements.
template <int kLanes, int kN>
__device__ __forceinline__ int expert_of(int i, int sub) { return (i / kN * kLanes + sub) * kN + i % kN; }

// A lane's part of a row; -inf behind its end.
template <typename T, int kPer, int kLanes, int kN>
__device__ __forceinline__ void load_row(const T* row, int E, int sub, float (&v)[kPer]) {
#pragma unroll
    for (int i = 0; i < kPer; i += kN) {
        const int e = expert_of<kLanes, kN>(i, sub);
        if (e < E) {
            load_vec<T, kN>(row + e, *reinterpret_cast<float(*)[kN]>(v + i));
        } else {
#pragma unroll
            for (int j = 0; j < kN; ++j) v[i + j] = -INFINITY;
        }
    }
}

// Turns logits into terms v whose quotients by their sum are the row's p, and returns 1 / sum (0 where all experts are
// masked).  kRest: rest_e becomes 1 - s_e (sigmoids only).  bad: the row holds a NaN or +inf.
template <int kPer, int kLanes, bool kRest>
__device__ __forceinline__ float row_terms(int score, float (&v)[kPer], float (&rest)[kRest ? kPer : 1], bool& bad) {
    float m = -INFINITY;
    bad = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        m = fmaxf(m, v[i]);               // passes NaN over
        bad |= !(v[i] < INFINITY);
    }
    m = lanes_max<kLanes>(m);
    if (__any_sync(kAll, bad)) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = score == MOE_SCORE_SOFTMAX ? softmax_logit(masked_nan(v[i]), m) : masked_nan(v[i]);
    }
    float sum = 0.0f;
    if (score == MOE_SCORE_SOFTMAX) {
        const float shift = softmax_shift(m);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            v[i] = expf(v[i] - shift);
            sum += v[i];
        }
    } else {
        const bool low = m < 0.0f;        // relative to the largest, which does not underflow then
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const float t = expf(-fabsf(v[i])), y = reciprocal_1_2(1.0f + t);
            if (kRest) rest[i] = v[i] < 0.0f ? y : t * y;
            v[i] = low ? (m < kLowestLogit ? 0.0f : expf(v[i] - m) * y) : v[i] < 0.0f ? t * y : y;
            sum += v[i];
        }
    }
    sum = lanes_sum<kLanes>(sum);
    return sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
}

// Rows [begin, end) of a sequence, inside [0, T] whatever the offsets say.
__device__ __forceinline__ void sequence_rows(const int32_t* offsets, int64_t s, int64_t T, int64_t& begin, int64_t& end) {
    if (offsets == nullptr) {
        begin = 0;
        end = T;
        return;
    }
    begin = min(max(static_cast<int64_t>(offsets[s]), int64_t(0)), T);
    end = min(max(static_cast<int64_t>(offsets[s + 1]), begin), T);
}

struct BalanceParams {
    int64_t T;
    int E;
    int64_t ld;
    int score, k;
    const int32_t* ids;
    const uint8_t* mask;
    const int32_t* offsets;
    int64_t S;
    int* err;
};

// One cluster of kSplit CTAs to a sequence; each takes a stretch of its rows and holds the sums of p and the counts,
// which the CTAs then join in order, a part of the experts each.
template <typename T, int kPer, int kLanes, int kN>
__global__ void __cluster_dims__(kSplit, 1, 1) __launch_bounds__(kThreads)
    balance_sequence_kernel(const T* __restrict__ logits, const BalanceParams p, float* __restrict__ loss,
                            int32_t* __restrict__ counts, float* __restrict__ probs, int32_t* __restrict__ tokens) {
    constexpr int kGroups = 32 / kLanes;
    extern __shared__ float s_sum[];                        // [kWarps][E], then [E] sums and [E] counts
    __shared__ int s_tokens;
    __shared__ float s_loss, s_part[kWarps];
    const int E = p.E;
    int* s_count = reinterpret_cast<int*>(s_sum + kWarps * E);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % kLanes;
    const uint32_t rank = cluster_rank();
    const int64_t s = blockIdx.x / kSplit;
    int64_t begin, end;
    sequence_rows(p.offsets, s, p.T, begin, end);
    const int64_t share = (end - begin + kSplit - 1) / kSplit;
    begin = min(begin + static_cast<int64_t>(rank) * share, end);
    end = min(begin + share, end);
    for (int e = threadIdx.x; e < E; e += kThreads) s_count[e] = 0;
    if (threadIdx.x == 0) s_tokens = 0;
    __syncthreads();

    float acc[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = 0.0f;
    int mine = 0;
    for (int64_t base = begin; base < end; base += kWarps * kGroups) {
        const int64_t t = base + warp * kGroups + lane / kLanes;
        const bool real = t < end && (p.mask == nullptr || p.mask[t] != 0);
        float v[kPer], none[1];
        if (real) {
            load_row<T, kPer, kLanes, kN>(logits + t * p.ld, E, sub, v);
            mine += sub == 0;
            for (int j = sub; j < p.k; j += kLanes) {
                const int id = p.ids[t * p.k + j];
                if (static_cast<unsigned>(id) < static_cast<unsigned>(E)) atomicAdd(s_count + id, 1);
                else set_device_error(p.err, NVFP4_ERR_BAD_EXPERT_ID);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) v[i] = -INFINITY;
        }
        bool bad;
        const float r = row_terms<kPer, kLanes, false>(p.score, v, none, bad);
        if (bad) set_device_error(p.err, NVFP4_ERR_NONFINITE);
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] = fmaf(v[i], r, acc[i]);
    }
#pragma unroll
    for (int o = 16; o >= kLanes; o >>= 1) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] += __shfl_xor_sync(kAll, acc[i], o);
    }
    if (lane < kLanes) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = expert_of<kLanes, kN>(i, sub);
            if (e < E) s_sum[warp * E + e] = acc[i];
        }
    }
    if (mine) atomicAdd(&s_tokens, mine);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) {
        float sum = s_sum[e];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) sum += s_sum[w * E + e];
        s_sum[e] = sum;
    }
    cluster_barrier();

    int n = 0;
#pragma unroll
    for (int c = 0; c < kSplit; ++c) n += cluster_load_s32(cluster_addr(&s_tokens, c));
    const int part = (E + kSplit - 1) / kSplit;             // at most 128
    const int e = static_cast<int>(rank) * part + static_cast<int>(threadIdx.x);
    float term = 0.0f;
    if (static_cast<int>(threadIdx.x) < part && e < E) {
        int count = 0;
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < kSplit; ++c) {
            count += cluster_load_s32(cluster_addr(s_count + e, c));
            sum += cluster_load_f32(cluster_addr(s_sum + e, c));
        }
        const float mean = n > 0 ? sum / static_cast<float>(n) : 0.0f;
        counts[s * E + e] = count;
        probs[s * E + e] = mean;
        term = static_cast<float>(count) * mean;
    }
    term = lanes_sum<32>(term);
    if (lane == 0) s_part[warp] = term;
    __syncthreads();
    if (threadIdx.x == 0) {
        s_loss = 0.0f;
        for (int w = 0; w < kWarps; ++w) s_loss += s_part[w];
    }
    cluster_barrier();
    if (rank == 0 && threadIdx.x == 0) {
        float sum = 0.0f;
        for (int c = 0; c < kSplit; ++c) sum += cluster_load_f32(cluster_addr(&s_loss, c));
        loss[s] = n > 0 ? sum * (static_cast<float>(E) / (static_cast<float>(p.k) * static_cast<float>(n))) : 0.0f;
        tokens[s] = n;
    }
    cluster_barrier();                                      // no CTA leaves while another reads its shared memory
}

// Sequence of a row: the last whose offset is not above it; -1 in front of the first, S behind the last.  Of a whole
// warp and the same row in all lanes: a round looks at 32 offsets.
__device__ __forceinline__ int64_t find_sequence(const int32_t* offsets, int64_t S, int64_t row) {
    if (offsets == nullptr) return 0;
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, hi = S + 1;                             // offsets in front of lo are <= row, from hi on above it
    while (lo < hi) {
        const int64_t step = (hi - lo + 31) / 32, at = lo + lane * step;
        const unsigned below = __ballot_sync(kAll, at < hi && offsets[at] <= row);
        const int c = __popc(below);
        if (c == 0) break;
        lo += (c - 1) * step + 1;
        hi = min(hi, lo - 1 + step);
    }
    return lo - 1;
}

// Rows in stretches of kRows to a CTA, a row to kLanes lanes; the g of a sequence stay in registers.
template <typename T, int kPer, int kLanes, int kN>
__global__ void __launch_bounds__(kThreads)
    balance_backward_kernel(const T* __restrict__ logits, const BalanceParams p, int64_t rows_per_cta,
                            const int32_t* __restrict__ counts, const int32_t* __restrict__ tokens,
                            const float* __restrict__ dloss, T* __restrict__ dl, int64_t ld_out, int accumulate) {
    constexpr int kGroups = 32 / kLanes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % kLanes, E = p.E;
    const int64_t begin = static_cast<int64_t>(blockIdx.x) * rows_per_cta, end = min(begin + rows_per_cta, p.T);
    int64_t s = find_sequence(p.offsets, p.S, begin + warp * kGroups), held = -1;
    float g[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) g[i] = 0.0f;
    for (int64_t base = begin; base < end; base += kWarps * kGroups) {
        const int64_t t = base + warp * kGroups + lane / kLanes;
        if (p.offsets != nullptr) {
            while (t < end && s < p.S && t >= p.offsets[s + 1]) ++s;
        }
        const bool real = t < end && s >= 0 && s < p.S && (p.mask == nullptr || p.mask[t] != 0);
        float v[kPer], rest[kPer];
        if (real) {
            load_row<T, kPer, kLanes, kN>(logits + t * p.ld, E, sub, v);
            if (s != held) {
                held = s;
                const float n = static_cast<float>(tokens[s]);
                const float scale = n > 0.0f ? dloss[s] * (static_cast<float>(E) / (static_cast<float>(p.k) * n * n)) : 0.0f;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int e = expert_of<kLanes, kN>(i, sub);
                    g[i] = e < E ? scale * static_cast<float>(counts[s * E + e]) : 0.0f;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) v[i] = -INFINITY;
        }
        bool bad;
        const float r = row_terms<kPer, kLanes, true>(p.score, v, rest, bad);
        if (bad) set_device_error(p.err, NVFP4_ERR_NONFINITE);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            v[i] *= r;
            dot = fmaf(g[i], v[i], dot);
        }
        dot = lanes_sum<kLanes>(dot);
        if (t >= end || (accumulate && !real)) continue;
        T* out = dl + t * ld_out;
#pragma unroll
        for (int i = 0; i < kPer; i += kN) {
            const int e = expert_of<kLanes, kN>(i, sub);
            if (e >= E) continue;
            float d[kN];
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                d[j] = v[i + j] * (g[i + j] - dot);
                if (p.score != MOE_SCORE_SOFTMAX) d[j] *= rest[i + j];
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
}

// By the experts: kPer of them to each of kLanes lanes.
template <typename F>
cudaError_t by_experts(int E, F&& f) {
    if (E <= 128) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 8>());
    if (E <= 256) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 16>());
    if (E <= 512) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 32>());
    return f(std::integral_constant<int, 32>(), std::integral_constant<int, 32>());
}
// Loads of 16 bytes where every row starts and ends on their boundary, of single elements otherwise.
template <typename T>
bool wide_rows(const void* a, int64_t ld, int E) {
    constexpr int64_t kN = 16 / sizeof(T);
    return (reinterpret_cast<uintptr_t>(a) & 15) == 0 && ld % kN == 0 && E % kN == 0;
}

template <typename T>
cudaError_t forward(const void* logits, const BalanceParams& p, float* loss, int32_t* counts, float* probs, int32_t* tokens,
                    cudaStream_t st) {
    return by_experts(p.E, [&](auto per, auto lanes) {
        constexpr int kPer = decltype(per)::value, kLanes = decltype(lanes)::value;
        auto* kernel = wide_rows<T>(logits, p.ld, p.E) ? balance_sequence_kernel<T, kPer, kLanes, 16 / sizeof(T)>
                                                       : balance_sequence_kernel<T, kPer, kLanes, 1>;
        return launch_pdl(false, kernel, dim3(static_cast<unsigned>(p.S * kSplit)), dim3(kThreads),
                          static_cast<size_t>(p.E) * (kWarps + 1) * sizeof(float), st, static_cast<const T*>(logits), p, loss,
                          counts, probs, tokens);
    });
}

template <typename T>
cudaError_t backward(const void* logits, const BalanceParams& p, const int32_t* counts, const int32_t* tokens,
                     const float* dloss, void* dl, int64_t ld_out, bool accumulate, cudaStream_t st) {
    return by_experts(p.E, [&](auto per, auto lanes) {
        constexpr int kPer = decltype(per)::value, kLanes = decltype(lanes)::value;
        constexpr int64_t kRows = kThreads / kLanes;        // of a CTA at a time
        auto* kernel = wide_rows<T>(logits, p.ld, p.E) && wide_rows<T>(dl, ld_out, p.E)
                           ? balance_backward_kernel<T, kPer, kLanes, 16 / sizeof(T)>
                           : balance_backward_kernel<T, kPer, kLanes, 1>;
        int64_t turns = p.T / (kRows * 4 * device_sm_count());
        turns = turns < 1 ? 1 : turns > 16 ? 16 : turns;
        const int64_t rows = turns * kRows;
        return launch_pdl(false, kernel, dim3(static_cast<unsigned>((p.T + rows - 1) / rows)), dim3(kThreads), 0, st,
                          static_cast<const T*>(logits), p, rows, counts, tokens, dloss, static_cast<T*>(dl), ld_out,
                          accumulate ? 1 : 0);
    });
}

}  // namespace

cudaError_t launch_balance_loss(const void* logits, int type, const BalanceArgs& a, float* loss, int32_t* counts, float* probs,
                                int32_t* tokens, int* err, cudaStream_t st) {
    const BalanceParams p = {a.T, a.E, a.ld, a.score, a.k, a.ids, a.mask, a.offsets, a.S, err};
    switch (type) {
        case NVFP4_TYPE_F32: return forward<float>(logits, p, loss, counts, probs, tokens, st);
        case NVFP4_TYPE_BF16: return forward<__nv_bfloat16>(logits, p, loss, counts, probs, tokens, st);
        default: return forward<__half>(logits, p, loss, counts, probs, tokens, st);
    }
}

cudaError_t launch_balance_loss_backward(const void* logits, int type, const BalanceArgs& a, const int32_t* counts,
                                         const int32_t* tokens, const float* dloss, void* dl, int64_t ld_out, bool accumulate,
                                         int* err, cudaStream_t st) {
    const BalanceParams p = {a.T, a.E, a.ld, a.score, a.k, a.ids, a.mask, a.offsets, a.S, err};
    switch (type) {
        case NVFP4_TYPE_F32: return backward<float>(logits, p, counts, tokens, dloss, dl, ld_out, accumulate, st);
        case NVFP4_TYPE_BF16: return backward<__nv_bfloat16>(logits, p, counts, tokens, dloss, dl, ld_out, accumulate, st);
        default: return backward<__half>(logits, p, counts, tokens, dloss, dl, ld_out, accumulate, st);
    }
}

}  // namespace nvfp4
