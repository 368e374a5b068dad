// Routing of given router logits: scores (softmax or sigmoid), an optional selection bias,
// expert groups, top-k, renormalisation and a scaling factor; and the gradient of the weights.
//
//   s_e  = softmax(l)_e, or 1 / (1 + e^-l_e); 0 for a masked expert (l_e = -inf or NaN)
//   o_e  = l_e without a bias (softmax and sigmoid are monotonic, and logits do not saturate),
//          s_e + b_e with one; the order is o descending, the lower id first on equal values,
//          masked experts last
//   groups of E / n_group consecutive experts: the topk_group groups with the largest score stay,
//          score = max o, or the sum of the two largest s_e (+ b_e)
//   w_j  = scale * s_j / sum of the chosen s (renormalised; 0 where the sum is 0), or scale * s_j
//
// All sums and scores are FP32, taken in one fixed order, so a token's result does not depend on
// the batch it is in.
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "ops.cuh"

namespace nvfp4 {
namespace {

constexpr int kWarps = 8;                 // tokens (one per warp) of a block
constexpr unsigned kAll = 0xFFFFFFFFu;

template <typename T>
__device__ __forceinline__ float load_f32(const T* p);
template <>
__device__ __forceinline__ float load_f32<float>(const float* p) { return __ldg(p); }
template <>
__device__ __forceinline__ float load_f32<__nv_bfloat16>(const __nv_bfloat16* p) { return __bfloat162float(*p); }
template <>
__device__ __forceinline__ float load_f32<__half>(const __half* p) { return __half2float(*p); }

template <typename T>
__device__ __forceinline__ void store_f32(T* p, float v);
template <>
__device__ __forceinline__ void store_f32<float>(float* p, float v) { *p = v; }
template <>
__device__ __forceinline__ void store_f32<__nv_bfloat16>(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ void store_f32<__half>(__half* p, float v) { *p = __float2half_rn(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

// A logit with NaN replaced by the mask.
__device__ __forceinline__ float masked_nan(float l) { return l != l ? -INFINITY : l; }

// e^(l - m) of a softmax whose largest logit is m: 1 where l = m (also for m = +inf), 0 where l is
// masked (also where every logit is, m = -inf).
__device__ __forceinline__ float softmax_term(float l, float m) {
    if (l == -INFINITY) return 0.0f;
    return l == m ? 1.0f : expf(l - m);
}
__device__ __forceinline__ float sigmoid(float l) { return l == -INFINITY ? 0.0f : __fdiv_rn(1.0f, 1.0f + expf(-l)); }

// Order-preserving key of an order value: larger first as unsigned; +-0 equal.  Masked: kMasked;
// an expert outside the kept groups, one already chosen, or none: 0.
constexpr uint32_t kMasked = 1u;
__device__ __forceinline__ uint32_t order_key(float o) {
    const uint32_t b = __float_as_uint(o + 0.0f);          // -0 + 0 = +0
    if (!(o > -INFINITY)) return kMasked;                  // -inf and NaN
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);     // finite values and +inf: all above kMasked
}

// One warp per token; lane holds experts lane + 32 i, i < V.
template <typename T, int V>
__global__ void __launch_bounds__(32 * kWarps)
    route_topk_kernel(const T* __restrict__ logits, int64_t tokens, int E, int64_t ld, RouteParams p,
                      const float* __restrict__ bias, int32_t* __restrict__ ids, float* __restrict__ weights,
                      int* err) {
    extern __shared__ float s_row[];                       // [kWarps][E]: group score inputs
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (t >= tokens) return;
    const T* row = logits + t * ld;

    float l[V];
    bool finite = true;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        const float v = e < E ? load_f32(row + e) : -INFINITY;
        finite = finite && !(v != v || v == INFINITY);
        l[i] = masked_nan(v);
    }
    if (!finite) set_device_error(err, NVFP4_ERR_NONFINITE);

    const bool top2 = p.n_group > 1 && p.group_score == MOE_GROUP_TOP2;
    const bool need_scores = bias != nullptr || top2;
    float s[V];
    if (need_scores) {
        if (p.score == MOE_SCORE_SOFTMAX) {
            float m = l[0];
#pragma unroll
            for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
            m = warp_max(m);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                s[i] = softmax_term(l[i], m);
                sum += s[i];
            }
            sum = warp_sum(sum);
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] = sum > 0.0f ? __fdiv_rn(s[i], sum) : 0.0f;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] = sigmoid(l[i]);
        }
        if (bias != nullptr) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane + 32 * i;
                s[i] = e < E && l[i] > -INFINITY ? s[i] + __ldg(bias + e) : -INFINITY;
            }
        }
    }
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = lane + 32 * i < E ? order_key(bias != nullptr ? s[i] : l[i]) : 0u;

    if (p.n_group > 1) {
        float* sr = s_row + warp * E;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            if (e < E) sr[e] = top2 ? (l[i] > -INFINITY ? s[i] : -INFINITY) : __uint_as_float(key[i]);
        }
        __syncwarp();
        const int size = E / p.n_group;
        uint32_t gk = 0u;                                   // lane g < n_group: key of group g
        if (lane < p.n_group) {
            const float* g = sr + lane * size;
            if (top2) {
                float a = -INFINITY, b = -INFINITY;         // the two largest, masked ones left out
                for (int i = 0; i < size; ++i) {
                    const float v = g[i];
                    if (v > a) {
                        b = a;
                        a = v;
                    } else if (v > b) {
                        b = v;
                    }
                }
                gk = order_key(b > -INFINITY ? a + b : a);
            } else {
                for (int i = 0; i < size; ++i) gk = max(gk, __float_as_uint(g[i]));
            }
        }
        int ahead = 0;
        for (int g = 0; g < p.n_group; ++g) {
            const uint32_t o = __shfl_sync(kAll, gk, g);
            ahead += (o > gk || (o == gk && g < lane)) ? 1 : 0;
        }
        const uint32_t kept = __ballot_sync(kAll, lane < p.n_group && ahead < p.topk_group);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            if (e < E && !((kept >> (e / size)) & 1u)) key[i] = 0u;
        }
    }

    // k rounds: the largest key, then the lowest id that has it
    int my_id = 0;
    for (int j = 0; j < p.k; ++j) {
        uint32_t best = key[0];
        int at = lane;
#pragma unroll
        for (int i = 1; i < V; ++i) {
            if (key[i] > best) {
                best = key[i];
                at = lane + 32 * i;
            }
        }
        const uint32_t top = __reduce_max_sync(kAll, best);
        const int id = static_cast<int>(__reduce_min_sync(kAll, best == top ? static_cast<uint32_t>(at) : kAll));
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (id == lane + 32 * i) key[i] = 0u;
        }
        if (lane == j) my_id = id;
    }

    // the chosen experts' scores, lane j < k holding slot j
    const bool slot = lane < p.k;
    const float lj = slot ? masked_nan(load_f32(row + my_id)) : -INFINITY;
    float w;
    if (p.score == MOE_SCORE_SIGMOID) {
        w = sigmoid(lj);
    } else if (p.renormalize) {
        w = softmax_term(lj, warp_max(lj));                 // the softmax over the chosen
    } else {
        float m = l[0];
#pragma unroll
        for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
        m = warp_max(m);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) sum += softmax_term(l[i], m);
        sum = warp_sum(sum);
        w = sum > 0.0f ? __fdiv_rn(softmax_term(lj, m), sum) : 0.0f;
    }
    if (p.renormalize) {
        const float sum = warp_sum(w);
        w = sum > 0.0f ? __fdiv_rn(w, sum) : 0.0f;
    }
    if (slot) {
        ids[t * p.k + lane] = my_id;
        weights[t * p.k + lane] = w * p.scale;
    }
}

// Gradient of the weights with respect to the logits; the choice itself has none.  With
// g_j = scale * dw_j, and sums over the chosen:
//   softmax, renormalised:  dl_c = q_c (g_c - sum_j g_j q_j),  q = softmax over the chosen
//   sigmoid, renormalised:  dl_c = q_c (1 - s_c) (g_c - sum_j g_j q_j),  q_c = s_c / sum_j s_j
//   sigmoid:                dl_c = g_c s_c (1 - s_c)
//   softmax:                dl_e = s_e ([e chosen] g_e - sum_j g_j s_j), every expert
// One warp per token; lane holds experts lane + 32 i of the output row, and slot `lane`.
template <typename T, int V>
__global__ void __launch_bounds__(32 * kWarps)
    route_topk_backward_kernel(const T* __restrict__ logits, int64_t tokens, int E, int64_t ld, RouteParams p,
                               const int32_t* __restrict__ ids, const float* __restrict__ dw, T* __restrict__ dl,
                               int64_t ld_out, int* err) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (t >= tokens) return;
    const T* row = logits + t * ld;
    int id = -1;
    float g = 0.0f, lj = -INFINITY;
    if (lane < p.k) {
        id = __ldg(ids + t * p.k + lane);
        if (id < 0 || id >= E) {
            set_device_error(err, NVFP4_ERR_BAD_EXPERT_ID);
            id = -1;
        } else {
            g = p.scale * __ldg(dw + t * p.k + lane);
            lj = masked_nan(load_f32(row + id));
        }
    }
    float v[V];
    float d;
    if (p.score == MOE_SCORE_SOFTMAX && !p.renormalize) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            v[i] = e < E ? masked_nan(load_f32(row + e)) : -INFINITY;
            m = fmaxf(m, v[i]);
        }
        m = warp_max(m);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[i] = softmax_term(v[i], m);
            sum += v[i];
        }
        sum = warp_sum(sum);
        const float r = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
        d = g * (softmax_term(lj, m) * r);
        const float c = -warp_sum(d) * r;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= c;
    } else {
        float s, rest = 1.0f;                               // rest = 1 - s
        if (p.score == MOE_SCORE_SOFTMAX) {
            s = softmax_term(lj, warp_max(lj));
        } else {
            s = sigmoid(lj);
            rest = lj == -INFINITY ? 1.0f : __fdiv_rn(1.0f, 1.0f + expf(lj));
        }
        float dot = 0.0f;
        if (p.renormalize) {
            const float sum = warp_sum(s);
            s = sum > 0.0f ? __fdiv_rn(s, sum) : 0.0f;
            dot = warp_sum(g * s);
        }
        d = s * rest * (g - dot);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.0f;
    }
    for (int j = 0; j < p.k; ++j) {
        const int e = __shfl_sync(kAll, id, j);
        const float dj = __shfl_sync(kAll, d, j);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (e == lane + 32 * i) v[i] += dj;
        }
    }
    T* out = dl + t * ld_out;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        if (e < E) store_f32(out + e, v[i]);
    }
}

// f(type tag, lane width) for the logits' type and the experts per lane.
template <typename T, typename F>
cudaError_t by_width(int E, F f) {
    if (E <= 32) return f(T{}, std::integral_constant<int, 1>{});
    if (E <= 64) return f(T{}, std::integral_constant<int, 2>{});
    if (E <= 128) return f(T{}, std::integral_constant<int, 4>{});
    if (E <= 256) return f(T{}, std::integral_constant<int, 8>{});
    if (E <= 512) return f(T{}, std::integral_constant<int, 16>{});
    return f(T{}, std::integral_constant<int, 32>{});
}
template <typename F>
cudaError_t by_type(int type, int E, F f) {
    switch (type) {
        case NVFP4_TYPE_F32: return by_width<float>(E, f);
        case NVFP4_TYPE_BF16: return by_width<__nv_bfloat16>(E, f);
        default: return by_width<__half>(E, f);
    }
}

}  // namespace

cudaError_t launch_route_topk(const void* logits, int type, int64_t T, int E, int64_t ld, const RouteParams& p,
                              const float* bias, int32_t* ids, float* weights, int* err, cudaStream_t st) {
    const unsigned grid = static_cast<unsigned>((T + kWarps - 1) / kWarps);
    const size_t smem = p.n_group > 1 ? static_cast<size_t>(kWarps) * E * 4 : 0;
    return by_type(type, E, [&](auto tag, auto v) {
        using L = decltype(tag);
        return launch_pdl(false, route_topk_kernel<L, decltype(v)::value>, grid, 32 * kWarps, smem, st,
                          static_cast<const L*>(logits), T, E, ld, p, bias, ids, weights, err);
    });
}

cudaError_t launch_route_topk_backward(const void* logits, int type, int64_t T, int E, int64_t ld,
                                       const RouteParams& p, const int32_t* ids, const float* dw, void* dl,
                                       int64_t ld_out, int* err, cudaStream_t st) {
    const unsigned grid = static_cast<unsigned>((T + kWarps - 1) / kWarps);
    return by_type(type, E, [&](auto tag, auto v) {
        using L = decltype(tag);
        return launch_pdl(false, route_topk_backward_kernel<L, decltype(v)::value>, grid, 32 * kWarps, 0, st,
                          static_cast<const L*>(logits), T, E, ld, p, ids, dw, static_cast<L*>(dl), ld_out, err);
    });
}

}  // namespace nvfp4
