// The router's balance loss over packed sequences, with per-expert counts, and its gradient: what their kernels share.
//
//   p_te = softmax(l_t)_e, or sigmoid(l_te) / sum_j sigmoid(l_tj); 0 for a masked expert (l = -inf or NaN)
//   of the n tokens of a sequence that are not masked:  c_e = slots that chose e,  P_e = 1/n sum_t p_te
//   loss = E / (k n) sum_e c_e P_e
//   with g_e = dloss E c_e / (k n^2):  softmax  dl_te = p_te (g_e - sum_j g_j p_tj)
//                                      sigmoid  dl_te = p_te (1 - s_te) (g_e - sum_j g_j p_tj),  s the sigmoid
//
// A token is taken by 8, 16 or 32 lanes, so that a lane has at most 16 experts (32 of more than 512).
#pragma once

#include <type_traits>

#include "cluster.cuh"
#include "common.cuh"
#include "ops.cuh"
#include "scores.cuh"

namespace nvfp4 {
namespace balance {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr unsigned kAll = 0xFFFFFFFFu;

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
// masked).  kRest: rest_e becomes 1 - s_e (sigmoids only).  bad: the row holds a NaN or +inf.  What rows hardly ever need
// (NaN, +inf, sigmoids that may underflow) is looked for by the warp as a whole: a choice for each element took half as
// many instructions again.  -inf, a masked expert or none, gives 0 by itself.
template <int kPer, int kLanes, bool kRest>
__device__ __forceinline__ float row_terms(int score, float (&v)[kPer], float (&rest)[kRest ? kPer : 1], bool& bad) {
    float m = v[0], probe = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        m = fmaxf(m, v[i]);               // passes NaN over
        probe += v[i];                    // below +inf without a NaN or +inf (it may reach that without, which does no harm)
    }
    m = lanes_max<kLanes>(m);
    bad = false;
    if (__any_sync(kAll, !(probe < INFINITY))) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            bad |= !(v[i] < INFINITY);
            v[i] = score == MOE_SCORE_SOFTMAX ? softmax_logit(masked_nan(v[i]), m) : masked_nan(v[i]);
        }
        if (m != m) m = -INFINITY;        // nothing but NaN
    }
    float sum = 0.0f;
    if (score == MOE_SCORE_SOFTMAX) {
        const float shift = softmax_shift(m);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            v[i] = expf(v[i] - shift);
            sum += v[i];
        }
    } else if (__any_sync(kAll, m < 0.0f)) {   // relative to the largest, which does not underflow then
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const float t = expf(-fabsf(v[i])), y = reciprocal_1_2(1.0f + t);
            if (kRest) rest[i] = v[i] < 0.0f ? y : t * y;
            v[i] = m < 0.0f ? (m < kLowestLogit ? 0.0f : expf(v[i] - m) * y) : v[i] < 0.0f ? t * y : y;
            sum += v[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const float t = expf(-fabsf(v[i])), y = reciprocal_1_2(1.0f + t), ty = t * y;
            if (kRest) rest[i] = v[i] < 0.0f ? y : ty;
            v[i] = v[i] < 0.0f ? ty : y;
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

// By the experts: kPer of them to each of kLanes lanes.
template <typename F>
cudaError_t by_experts(int E, F&& f) {
    if (E <= 128) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 8>());
    if (E <= 256) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 16>());
    if (E <= 512) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 32>());
    return f(std::integral_constant<int, 32>(), std::integral_constant<int, 32>());
}
// Elements of a load: 16 bytes where every row starts and ends on their boundary, two, or one.
template <typename T>
int load_width(const void* a, int64_t ld, int E) {
    const int64_t bits = static_cast<int64_t>(reinterpret_cast<uintptr_t>(a) / sizeof(T)) | ld | E;
    return reinterpret_cast<uintptr_t>(a) % sizeof(T) ? 1 : bits % (16 / sizeof(T)) == 0 ? 16 / sizeof(T) : bits % 2 == 0 ? 2 : 1;
}
template <typename T, typename F>
cudaError_t by_width(int width, F&& f) {
    if (width == 16 / sizeof(T)) return f(std::integral_constant<int, 16 / sizeof(T)>());
    if (width == 2) return f(std::integral_constant<int, 2>());
    return f(std::integral_constant<int, 1>());
}

}  // namespace balance
}  // namespace nvfp4
