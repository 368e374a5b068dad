// Routing of given router logits: scores (softmax or sigmoid), an optional selection bias,
// expert groups, top-k, renormalisation and a scaling factor; and the gradient of the weights.
//
//   s_e  = softmax(l)_e, or 1 / (1 + e^-l_e); 0 for a masked expert (l_e = -inf or NaN)
//   o_e  = l_e without a bias (softmax and sigmoid are monotonic, and logits do not saturate),
//          s_e + b_e with one; the order is o descending, the lower id first on equal values,
//          masked experts last
//   groups of E / n_group consecutive experts: the topk_group groups with the largest score stay,
//          score = max o, or the sum of the two largest s_e (+ b_e)
//   w_j  = scale * s_j / sum of the chosen s (renormalised; 0 where the sum is 0), or scale * s_j; the ratios are taken
//          of scores relative to the largest chosen one, which do not underflow
//
// All sums and scores are FP32, taken in one fixed order, so a token's result does not depend on
// the batch it is in.  The order and the weights go by the same s_e, bit for bit (with the hardware's approximate
// exponential and reciprocal for the order, experts and groups a few units in the last place apart changed places;
// 65537 x 256, sigmoid + bias, 8 groups: 41.4 us on the device, 44.8 so).
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "ops.cuh"
#include "scores.cuh"

namespace nvfp4 {
namespace {

constexpr int kWarps = 8;                 // tokens (one per warp) of a block
constexpr unsigned kAll = 0xFFFFFFFFu;

// Order-preserving bits of a float: larger first as unsigned, +-0 equal; all above 0, which stands for no value.
__device__ __forceinline__ uint32_t ordered(float o) {
    const uint32_t b = __float_as_uint(o + 0.0f);          // -0 + 0 = +0
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

// Routing.  A token is taken by 8, 16 or 32 lanes (kLanes), so that a lane has at most 16 experts (32 of more than 512)
// and what a token needs whatever E is, its addresses, the bound, the candidates' ranks and the weights, is shared by the
// warp's four, two or one.  Lane s of a token holds experts V s + i, i < V; kN: elements of a load (rows aligned to them).
//
// The k largest keys: the k-th largest of the two largest of each half of the lanes' keys is a lower bound of the k-th
// largest, which about k + 2 of 256 keys reach; those are put side by side in shared memory (a lane finds its own
// by a bit mask) and each is ranked against the others.  Where more than 32 reach it (many equal keys, few lanes with
// keys), the picks are taken one by one.
//
// Bound by instructions: 595 to a token of 256 experts in 8 groups with sigmoids and a bias, beside the 1 KB that is read
// (65537 of them take 44.8 us, 73% of the issue slots; measured against today's form when its scores were approximate and
// it took 40: 121 with one reduction and a search of all keys for each pick, 70 with each lane's keys sorted, 47 with one
// token to a warp, 52 with 8 lanes and 32 experts to a lane, whose registers leave too few warps).  Groups that are not
// whole lanes cost a third more (8 of 31: 60.3 us).  Smaller batches are bound by latency: 16384 x 128 BF16 5.7 us with
// 3.4 blocks to an SM, 53% of the issue slots.
template <int V, int kLanes>
struct Shared {
    static constexpr int tokens = 32 / kLanes;
    static constexpr int pitch = V + 4;                        // words of a lane's keys: 16-byte words without bank conflicts
    static constexpr int pad = kLanes < 32 ? kLanes : 0;       // and the tokens' consecutive words
    __align__(16) uint32_t key[tokens][kLanes * pitch + pad];
    __align__(16) unsigned long long cand[tokens][32];
    int id[tokens][32];
};

template <int kLanes>
__device__ __forceinline__ float token_sum(float v) {
#pragma unroll
    for (int x = 1; x < kLanes; x <<= 1) v += __shfl_xor_sync(kAll, v, x);
    return v;
}
template <int kLanes, typename U>
__device__ __forceinline__ U token_max(U v) {
#pragma unroll
    for (int x = 1; x < kLanes; x <<= 1) v = max(v, __shfl_xor_sync(kAll, v, x));
    return v;
}

// The largest of a token's keys: one instruction where the token has the warp (65536 x 512 57.1 -> 48.2 us); several
// tokens' would go one after the other (65536 x 128 17.2 us by shuffles, 20.4).
template <int kLanes>
__device__ __forceinline__ uint32_t key_max(uint32_t v) {
    return kLanes == 32 ? __reduce_max_sync(kAll, v) : token_max<kLanes>(v);
}

template <typename T, int V, int kLanes, int kN>
__global__ void __launch_bounds__(32 * kWarps)
    route_topk_kernel(const T* __restrict__ logits, int64_t tokens, int E, int64_t ld, RouteParams p,
                            const float* __restrict__ bias, int32_t* __restrict__ ids, float* __restrict__ weights,
                            int* err) {
    using S = Shared<V, kLanes>;
    __shared__ S s_warps[kWarps];
    constexpr int kPitch = S::pitch, kTokens = S::tokens;
    const int lane = threadIdx.x & 31, slot = lane / kLanes, sub = lane % kLanes;
    S& sh = s_warps[threadIdx.x >> 5];
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kTokens;
    if (first >= tokens) return;
    const bool real = first + slot < tokens;                   // a warp's last tokens may be one that is there, again
    const int64_t t = real ? first + slot : tokens - 1;
    const T* row = logits + t * ld;
    const int e0 = V * sub;

    // the logits, -inf where there is no expert; a row of finite ones needs none of the checks for masks
    float l[V], probe = 0.0f;
    uint32_t* my_keys = sh.key[slot] + sub * kPitch;
    const bool whole = e0 + V <= E;
    if constexpr (kN > 1) {
        if (whole) {
#pragma unroll
            for (int i = 0; i < V; i += kN) load_vec<T, kN>(row + e0 + i, *reinterpret_cast<float(*)[kN]>(l + i));
        } else {
#pragma unroll
            for (int i = 0; i < V; i += kN) {
                if (e0 + i + kN <= E) {
                    load_vec<T, kN>(row + e0 + i, *reinterpret_cast<float(*)[kN]>(l + i));
                } else {
#pragma unroll
                    for (int j = i; j < i + kN; ++j) l[j] = e0 + j < E ? load_one(row + e0 + j) : -INFINITY;
                }
            }
        }
    } else {
        // rows on no such boundary: side by side from memory, each lane's own from shared memory (65537 x 251 in FP32
        // 33 us, 48 with each lane's own from memory)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = sub + kLanes * i;
            sh.key[slot][e / V * kPitch + e % V] = __float_as_uint(e < E ? load_one(row + e) : -INFINITY);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 w = *reinterpret_cast<const float4*>(my_keys + i);
            l[i] = w.x, l[i + 1] = w.y, l[i + 2] = w.z, l[i + 3] = w.w;
        }
    }
    if (whole) {
#pragma unroll
        for (int i = 0; i < V; ++i) probe = fmaf(l[i], 0.0f, probe);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) probe = fmaf(e0 + i < E ? l[i] : 0.0f, 0.0f, probe);
    }
    const bool clean = __all_sync(kAll, probe == 0.0f);
    if (!clean) {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            bad = bad || !(l[i] < INFINITY);                   // +inf and NaN
            l[i] = masked_nan(l[i]);
        }
        if (bad) set_device_error(err, NVFP4_ERR_NONFINITE);
    }

    // a softmax over all experts: its largest logit, its terms (in o) and their sum, where the order or the weights
    // need them
    const bool top2 = p.n_group > 1 && p.group_score == MOE_GROUP_TOP2;
    const bool scored = bias != nullptr || top2;
    const bool softmax = p.score == MOE_SCORE_SOFTMAX;
    const bool full = softmax && !p.renormalize;
    float all_max = 0.0f, all_sum = 0.0f, all_rc = 0.0f;
    float o[V];
    if (softmax && (scored || full)) {
        float m = l[0];
#pragma unroll
        for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
        all_max = token_max<kLanes>(m);
        const float shift = softmax_shift(all_max);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            o[i] = expf(softmax_logit(l[i], all_max) - shift);
            all_sum += o[i];
        }
        all_sum = token_sum<kLanes>(all_sum);
        if (!(all_sum > 0.0f)) all_sum = 1.0f;                 // all masked: every term is 0
        all_rc = __frcp_rn(all_sum);
    }

    // order values o where they are not the logits: the scores, computed as the weights are, plus the bias; the scores
    // are also what "top2" adds up
    if (scored) {
        if (softmax) {
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = quotient(o[i], all_sum, all_rc);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = sigmoid(l[i]);
        }
        if (bias != nullptr) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                float b[4];
                if (p.bias_wide && e0 + i + 4 <= E) {
                    load_vec<float, 4>(bias + e0 + i, b);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) b[j] = e0 + i + j < E ? __ldg(bias + e0 + i + j) : 0.0f;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i + j] = fmaxf(o[i + j] + b[j], -INFINITY);   // a NaN bias: -inf
            }
        }
        if (!clean) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (!(l[i] > -INFINITY)) o[i] = -INFINITY;     // masked
            }
        }
    }
    uint32_t key[V];
    const bool by_logit = bias == nullptr;
    if (by_logit) {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = ordered(l[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = ordered(o[i]);
    }
    if (!whole) {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = e0 + i < E ? key[i] : 0u;
    }

    if (p.n_group > 1) {
        const int size = E / p.n_group;
        if (p.group_lanes > 0) {
            // a group is group_lanes whole lanes (a power of two of them)
            uint32_t gk;
            if (top2) {
                float a = -INFINITY, b = -INFINITY;            // the two largest; masked values stay out
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    b = fmaxf(b, fminf(a, o[i]));
                    a = fmaxf(a, o[i]);
                }
                for (int x = 1; x < p.group_lanes; x <<= 1) {
                    const float a2 = __shfl_xor_sync(kAll, a, x), b2 = __shfl_xor_sync(kAll, b, x);
                    b = fmaxf(fminf(a, a2), fmaxf(b, b2));
                    a = fmaxf(a, a2);
                }
                gk = ordered(b > -INFINITY ? a + b : a);
            } else {
                gk = key[0];
#pragma unroll
                for (int i = 1; i < V; ++i) gk = max(gk, key[i]);
                for (int x = 1; x < p.group_lanes; x <<= 1) gk = max(gk, __shfl_xor_sync(kAll, gk, x));
            }
            if (e0 >= E) gk = 0u;
            // kept if fewer than topk_group groups come before it
            const int group = sub / p.group_lanes;
            int ahead = 0;
            for (int g = 0; g < p.n_group; ++g) {
                const uint32_t other = __shfl_sync(kAll, gk, g * p.group_lanes, kLanes);
                ahead += other > gk || (other == gk && g < group) ? 1 : 0;
            }
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = ahead < p.topk_group ? key[i] : 0u;
        } else {
            // any group size: the values through shared memory, a power of two of lanes to a group (one if there are
            // more groups than lanes); each group's key then lies in sh.id
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                *reinterpret_cast<uint4*>(my_keys + i) =
                    top2 ? make_uint4(__float_as_uint(o[i]), __float_as_uint(o[i + 1]), __float_as_uint(o[i + 2]),
                                      __float_as_uint(o[i + 3]))
                         : make_uint4(key[i], key[i + 1], key[i + 2], key[i + 3]);
            }
            __syncwarp();
            const int share = 1 << p.group_share, at_once = kLanes >> p.group_share, part = sub & (share - 1);
            for (int base = 0; base < p.n_group; base += at_once) {
                const int g = base + (sub >> p.group_share), end = g < p.n_group ? (g + 1) * size : 0;
                uint32_t gk = 0u;
                if (top2) {
                    float a = -INFINITY, b = -INFINITY;
                    for (int e = g * size + part; e < end; e += share) {
                        const float f = __uint_as_float(sh.key[slot][e / V * kPitch + e % V]);
                        b = fmaxf(b, fminf(a, f));
                        a = fmaxf(a, f);
                    }
                    for (int x = 1; x < share; x <<= 1) {
                        const float a2 = __shfl_xor_sync(kAll, a, x), b2 = __shfl_xor_sync(kAll, b, x);
                        b = fmaxf(fminf(a, a2), fmaxf(b, b2));
                        a = fmaxf(a, a2);
                    }
                    gk = ordered(b > -INFINITY ? a + b : a);
                } else {
                    for (int e = g * size + part; e < end; e += share) gk = max(gk, sh.key[slot][e / V * kPitch + e % V]);
                    for (int x = 1; x < share; x <<= 1) gk = max(gk, __shfl_xor_sync(kAll, gk, x));
                }
                if (end > 0 && part == 0) sh.id[slot][g] = static_cast<int>(gk);
            }
            __syncwarp();
            uint32_t kept = 0u;                                // bit g: group g
            for (int g = sub; g < p.n_group; g += kLanes) {
                const uint32_t gk = static_cast<uint32_t>(sh.id[slot][g]);
                int ahead = 0;
                for (int h = 0; h < p.n_group; ++h) {
                    const uint32_t other = static_cast<uint32_t>(sh.id[slot][h]);
                    ahead += other > gk || (other == gk && h < g) ? 1 : 0;
                }
                kept |= (ahead < p.topk_group ? 1u : 0u) << g;
            }
            __syncwarp();
#pragma unroll
            for (int x = 1; x < kLanes; x <<= 1) kept |= __shfl_xor_sync(kAll, kept, x);
            int group = e0 / size, left = (group + 1) * size - e0;   // this expert's; past E the keys are 0
#pragma unroll
            for (int i = 0; i < V; ++i) {
                key[i] = (kept >> (group & 31)) & 1u ? key[i] : 0u;
                if (--left == 0) ++group, left = size;
            }
        }
    }

    // the bound: the k-th largest of the two largest keys of each half of the lanes' (equal ones together)
    uint32_t m[2] = {0u, 0u}, m2[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int h = 2 * i / V;
        m2[h] = max(m2[h], min(m[h], key[i]));
        m[h] = max(m[h], key[i]);
    }
    uint32_t bound = 0u;
    for (int j = 0; j < p.k; ++j) {
        bound = key_max<kLanes>(max(m[0], m[1]));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool gone = m[h] == bound;
            m[h] = gone ? m2[h] : m[h];
            m2[h] = gone ? 0u : m2[h];
        }
    }
    bound = max(bound, 1u);                                    // keys of 0 take no part
    // the keys that reach it, side by side
    uint32_t hits = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) hits |= key[i] >= bound ? 1u << i : 0u;
#pragma unroll
    for (int i = 0; i < V; i += 4) *reinterpret_cast<uint4*>(my_keys + i) = make_uint4(key[i], key[i + 1], key[i + 2], key[i + 3]);
    unsigned long long* cand = sh.cand[slot];
#pragma unroll
    for (int i = 0; i < 32 / kLanes; ++i) cand[sub + kLanes * i] = 0ull;
    const int count = __popc(hits);
    int at = count;
#pragma unroll
    for (int x = 1; x < kLanes; x <<= 1) {
        const int below = __shfl_up_sync(kAll, at, x, kLanes);
        at += sub >= x ? below : 0;
    }
    const int n = __shfl_sync(kAll, at, kLanes - 1, kLanes);
    at -= count;
    const int most = __reduce_max_sync(kAll, n);
    __syncwarp();
    if (most <= 32) {
        while (hits) {
            const int i = __ffs(static_cast<int>(hits)) - 1;
            hits &= hits - 1u;
            cand[at++] = (static_cast<unsigned long long>(my_keys[i]) << 32) | static_cast<uint32_t>(~(e0 + i));
        }
        __syncwarp();
        for (int c = sub; c < most; c += kLanes) {
            const unsigned long long mine = cand[c];
            int rank = 0;
            for (int d = 0; d < most; d += 4) {
                const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(cand + d);
                const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(cand + d + 2);
                rank += (x.x > mine ? 1 : 0) + (x.y > mine ? 1 : 0) + (y.x > mine ? 1 : 0) + (y.y > mine ? 1 : 0);
            }
            if (mine != 0ull && rank < p.k) sh.id[slot][rank] = static_cast<int>(~static_cast<uint32_t>(mine));
        }
    } else {
        // many equal keys, or few lanes with keys: one pick after the other
        for (int j = 0; j < p.k; ++j) {
            unsigned long long best = 0ull;
            for (int i = 0; i < V; ++i) {
                const unsigned long long v = (static_cast<unsigned long long>(my_keys[i]) << 32) | static_cast<uint32_t>(~(e0 + i));
                best = v > best ? v : best;
            }
            const unsigned long long top = token_max<kLanes>(best);
            if (best == top) {
                my_keys[~static_cast<uint32_t>(top) - e0] = 0u;
                sh.id[slot][j] = static_cast<int>(~static_cast<uint32_t>(top));
            }
        }
    }
    __syncwarp();

    // the chosen experts' scores, slot j in lane j % kLanes
    constexpr int kSlots = 32 / kLanes;
    float w[kSlots];
    int id[kSlots];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        const int j = sub + kLanes * i;
        id[i] = 0;
        w[i] = -INFINITY;
        if (j < p.k) {
            id[i] = sh.id[slot][j];
            w[i] = masked_nan(load_one(row + id[i]));
        }
        top = fmaxf(top, w[i]);
    }
    if (softmax) {
        const float mx = full ? all_max : token_max<kLanes>(top);      // renormalised: the softmax over the chosen
        const float shift = softmax_shift(mx);
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            if (kLanes * i < p.k) w[i] = expf(softmax_logit(w[i], mx) - shift);
        }
    } else if (p.renormalize) {
        const float mx = token_max<kLanes>(top);
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            if (kLanes * i < p.k) w[i] = sigmoid_ratio(w[i], mx);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            if (kLanes * i < p.k) w[i] = sigmoid(w[i]);
        }
    }
    if (p.renormalize) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            if (kLanes * i < p.k) sum += sub + kLanes * i < p.k ? w[i] : 0.0f;
        }
        sum = token_sum<kLanes>(sum);
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            if (kLanes * i < p.k) w[i] = sum > 0.0f ? __fdiv_rn(w[i], sum) : 0.0f;
        }
    } else if (full) {
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            if (kLanes * i < p.k) w[i] = quotient(w[i], all_sum, all_rc);
        }
    }
    if (!real) return;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        const int j = sub + kLanes * i;
        if (j < p.k) {
            ids[t * p.k + j] = id[i];
            weights[t * p.k + j] = w[i] * p.scale;
        }
    }
}

// Gradient of the weights with respect to the logits; the choice itself has none.  With
// g_j = scale * dw_j, and sums over the chosen:
//   softmax, renormalised:  dl_c = q_c (g_c - sum_j g_j q_j),  q = softmax over the chosen
//   sigmoid, renormalised:  dl_c = q_c (1 - s_c) (g_c - sum_j g_j q_j),  q_c = s_c / sum_j s_j
//   sigmoid:                dl_c = g_c s_c (1 - s_c)
//   softmax:                dl_e = s_e ([e chosen] g_e - sum_j g_j s_j), every expert
// The row is written with what an expert that was not chosen gets, in words of four experts side by side (kN elements to
// a load and store), and the chosen ones over it.
//
// Small batches take the time of a launch and its three dependent loads (4096 x 128 in FP32: 2.4 us); large ones are
// bound by the row written (and, for the softmax over all experts, read).

// Slot j's expert, g = scale * dw and logit; -1, 0 and -inf where there is none.
template <typename T>
__device__ __forceinline__ void load_slot(const T* row, const int32_t* ids, const float* dw, bool live, int E, float scale,
                                          int& id, float& g, float& lj, int* err) {
    id = live ? __ldg(ids) : -1;
    g = live ? scale * __ldg(dw) : 0.0f;
    lj = -INFINITY;
    if (live && (id < 0 || id >= E)) {
        set_device_error(err, NVFP4_ERR_BAD_EXPERT_ID);
        id = -1;
        g = 0.0f;
    }
    if (id >= 0) lj = masked_nan(load_one(row + id));
}

// Zeros at p, `bytes` of them (elements of kSize bytes), by a warp: whole 16-byte words but for the ends.
template <int kSize>
__device__ __forceinline__ void zero_span(uint8_t* p, int bytes) {
    using U = typename Word<kSize>::type;
    const int lane = threadIdx.x & 31, head = min(bytes, static_cast<int>(-reinterpret_cast<uintptr_t>(p) & 15));
    uint4* words = reinterpret_cast<uint4*>(p + head);
    const int n = (bytes - head) / 16, tail = (bytes - head) % 16;
    for (int i = lane; i < n; i += 32) words[i] = make_uint4(0u, 0u, 0u, 0u);
    if (lane * kSize < head) *reinterpret_cast<U*>(p + lane * kSize) = 0;
    if (lane * kSize < tail) *reinterpret_cast<U*>(p + bytes - tail + lane * kSize) = 0;
}

// Every weight but the softmax's over all experts: only the chosen logits take part.  A token is taken by kLanes >= k
// lanes, slot j in lane j; the warp writes its tokens' zeros first, which waits for nothing.  65537 x 256 in FP32 take
// 16.8 us for the 73 MB they cannot do without (4.4 TB/s): without the zeros it is 10.8, without the loads of the logits
// (a sector each) 11.1, so the one waits for most of the other.  (With one token to a warp 21.4 us, and with the zeros
// of odd rows element by element 65537 x 251 in BF16 21.5 instead of 10.2.)
template <typename T, int kLanes>
__global__ void __launch_bounds__(32 * kWarps)
    route_topk_backward_kernel(const T* __restrict__ logits, int64_t tokens, int E, int64_t ld, RouteParams p,
                               const int32_t* __restrict__ ids, const float* __restrict__ dw, T* __restrict__ dl,
                               int64_t ld_out, int* err) {
    constexpr int kTokens = 32 / kLanes;
    const int lane = threadIdx.x & 31, sub = lane % kLanes;
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kTokens;
    if (first >= tokens) return;
    const int64_t t = first + lane / kLanes;
    const bool live = t < tokens && sub < p.k;
    int id;
    float g, lj;
    const int here = static_cast<int>(min(tokens - first, static_cast<int64_t>(kTokens)));
    uint8_t* rows = reinterpret_cast<uint8_t*>(dl + first * ld_out);
    constexpr int kSize = sizeof(T);
    if (ld_out == E) {
        zero_span<kSize>(rows, here * E * kSize);
    } else {
        for (int i = 0; i < here; ++i) zero_span<kSize>(rows + i * ld_out * kSize, E * kSize);
    }
    load_slot(logits + t * ld, ids + t * p.k + sub, dw + t * p.k + sub, live, E, p.scale, id, g, lj, err);
    float s, rest = 1.0f;                                       // rest = 1 - s
    if (p.score == MOE_SCORE_SOFTMAX) {
        const float m = token_max<kLanes>(lj);
        s = expf(softmax_logit(lj, m) - softmax_shift(m));
    } else {
        s = p.renormalize ? sigmoid_ratio(lj, token_max<kLanes>(lj)) : sigmoid(lj);
        rest = sigmoid(-lj);
    }
    float dot = 0.0f;
    if (p.renormalize) {
        const float sum = token_sum<kLanes>(s);
        s = sum > 0.0f ? __fdiv_rn(s, sum) : 0.0f;
        dot = token_sum<kLanes>(g * s);
    }
    __syncwarp();                                               // orders the warp's writes
    if (id >= 0) dl[t * ld_out + id] = from_f32<T>(s * rest * (g - dot));
}

// Four experts' values at e of a row of E.
template <typename T, int kN>
__device__ __forceinline__ void store4(T* out, int e, int E, const float (&v)[4]) {
    if (e + 4 <= E) {
#pragma unroll
        for (int i = 0; i < 4; i += kN) store_vec<T, kN>(out + e + i, *reinterpret_cast<const float(*)[kN]>(v + i));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (e + i < E) out[e + i] = from_f32<T>(v[i]);
        }
    }
}

// The softmax over all experts.  A token is taken by kLanes lanes; lane s of them has the words of four experts at
// 4 (s + kLanes i), i < kWords, whatever the alignment, so sums are taken in one order, and slots s + kLanes i.  Rows
// of 16-bit logits on odd boundaries go through shared memory, side by side from and to memory (65537 x 251 in BF16 27.3 us
// without, 23.4 with it; in FP32, element by element, 26.3 and 31.2).
//
// Bound by memory, the row read and written: 65537 x 250 in FP32 take 23.9 us, 131 MB at 5.5 TB/s (25.2 us, bound by
// instructions, with one token to a warp whatever E).
template <typename T, int kWords, int kLanes, int kN>
__global__ void __launch_bounds__(32 * kWarps)
    route_topk_backward_full_kernel(const T* __restrict__ logits, int64_t tokens, int E, int64_t ld, RouteParams p,
                                    const int32_t* __restrict__ ids, const float* __restrict__ dw, T* __restrict__ dl,
                                    int64_t ld_out, int* err) {
    constexpr int kTokens = 32 / kLanes, kSlots = 32 / kLanes;
    const int lane = threadIdx.x & 31, sub = lane % kLanes;
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kTokens;
    if (first >= tokens) return;
    const bool real = first + lane / kLanes < tokens;           // a warp's last tokens may be one that is there, again
    const int64_t t = real ? first + lane / kLanes : tokens - 1;
    const T* row = logits + t * ld;
    T* out = dl + t * ld_out;
    constexpr bool kShared = kN == 1 && sizeof(T) == 2;
    constexpr int kCols = 4 * kWords * kLanes, kPitch = kCols + (kLanes < 32 ? kLanes : 0);
    __shared__ __align__(16) float s_rows[kShared ? kWarps : 1][kTokens * kPitch];
    float* staged = s_rows[kShared ? threadIdx.x >> 5 : 0] + lane / kLanes * kPitch;
    float v[kWords][4], probe = 0.0f;
    if (kShared) {
#pragma unroll
        for (int e = sub; e < kCols; e += kLanes) staged[e] = e < E ? load_one(row + e) : -INFINITY;
        __syncwarp();
    }
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
        const int e = 4 * (sub + kLanes * j);
        if (kShared) {
            const float4 w = *reinterpret_cast<const float4*>(staged + e);
            v[j][0] = w.x, v[j][1] = w.y, v[j][2] = w.z, v[j][3] = w.w;
        } else if (e + 4 <= E) {
#pragma unroll
            for (int i = 0; i < 4; i += kN) load_vec<T, kN>(row + e + i, *reinterpret_cast<float(*)[kN]>(v[j] + i));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j][i] = e + i < E ? load_one(row + e + i) : -INFINITY;
        }
    }
    int id[kSlots];
    float g[kSlots], lj[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        const int j = sub + kLanes * i;
        if (kLanes * i < p.k) load_slot(row, ids + t * p.k + j, dw + t * p.k + j, j < p.k, E, p.scale, id[i], g[i], lj[i], err);
    }
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
        const int e = 4 * (sub + kLanes * j);
#pragma unroll
        for (int i = 0; i < 4; ++i) m = fmaxf(m, v[j][i]);      // passes NaN over
        if (e + 4 <= E) {
#pragma unroll
            for (int i = 0; i < 4; ++i) probe = fmaf(v[j][i], 0.0f, probe);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) probe = fmaf(e + i < E ? v[j][i] : 0.0f, 0.0f, probe);
        }
    }
    m = token_max<kLanes>(m);
    const float shift = softmax_shift(m);
    if (!__all_sync(kAll, probe == 0.0f)) {                     // masks, infinities or NaN
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j][i] = softmax_logit(masked_nan(v[j][i]), m);
        }
    }
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[j][i] = expf(v[j][i] - shift);
            sum += v[j][i];
        }
    }
    sum = token_sum<kLanes>(sum);
    const float r = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
    float s[kSlots], own[kSlots], dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        if (kLanes * i >= p.k) continue;
        s[i] = expf(softmax_logit(lj[i], m) - shift);
        own[i] = g[i] * (s[i] * r);
        dot += own[i];
    }
    const float c = -token_sum<kLanes>(dot) * r;
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
        const int e = 4 * (sub + kLanes * j);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] *= c;
        if (kShared) *reinterpret_cast<float4*>(staged + e) = make_float4(v[j][0], v[j][1], v[j][2], v[j][3]);
        else if (real) store4<T, kN>(out, e, E, v[j]);
    }
    if (kShared) {
        __syncwarp();
#pragma unroll
        for (int e = sub; e < kCols; e += kLanes) {
            if (real && e < E) out[e] = from_f32<T>(staged[e]);
        }
    }
    __syncwarp();                                               // orders the warp's writes
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        if (kLanes * i < p.k && real && id[i] >= 0) out[id[i]] = from_f32<T>(s[i] * c + own[i]);
    }
}

template <typename T, int V, int kLanes, int kN>
cudaError_t launch_route(const void* logits, int64_t tokens, int E, int64_t ld, RouteParams p, const float* bias,
                         int32_t* ids, float* weights, int* err, cudaStream_t st) {
    // a group of whole lanes, a power of two of them
    const int size = E / p.n_group, lanes = size / V;
    p.group_lanes = size % V == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
    p.group_share = 0;
    while ((2 << p.group_share) * p.n_group <= kLanes) ++p.group_share;
    p.bias_wide = (reinterpret_cast<uintptr_t>(bias) & 15) == 0;
    constexpr int kPerBlock = kWarps * 32 / kLanes;
    return launch_pdl(false, route_topk_kernel<T, V, kLanes, kN>, static_cast<unsigned>((tokens + kPerBlock - 1) / kPerBlock),
                      32 * kWarps, 0, st, static_cast<const T*>(logits), tokens, E, ld, p, bias, ids, weights, err);
}
template <typename T, int V, int kLanes>
cudaError_t route_by_word(const void* logits, int64_t tokens, int E, int64_t ld, const RouteParams& p, const float* bias,
                          int32_t* ids, float* weights, int* err, cudaStream_t st) {
    constexpr int kWide = V * sizeof(T) < 16 ? V : 16 / static_cast<int>(sizeof(T));
    const int64_t bits = static_cast<int64_t>(reinterpret_cast<uintptr_t>(logits)) | (ld * static_cast<int64_t>(sizeof(T)));
    if (bits % (kWide * static_cast<int64_t>(sizeof(T))) == 0)
        return launch_route<T, V, kLanes, kWide>(logits, tokens, E, ld, p, bias, ids, weights, err, st);
    return launch_route<T, V, kLanes, 1>(logits, tokens, E, ld, p, bias, ids, weights, err, st);
}
// The kernel goes by E alone, so a token's result does not depend on how many there are.
template <typename T>
cudaError_t route_by_width(const void* logits, int64_t tokens, int E, int64_t ld, const RouteParams& p, const float* bias,
                           int32_t* ids, float* weights, int* err, cudaStream_t st) {
    if (E <= 32) return route_by_word<T, 4, 8>(logits, tokens, E, ld, p, bias, ids, weights, err, st);
    if (E <= 64) return route_by_word<T, 8, 8>(logits, tokens, E, ld, p, bias, ids, weights, err, st);
    if (E <= 128) return route_by_word<T, 16, 8>(logits, tokens, E, ld, p, bias, ids, weights, err, st);
    if (E <= 256) return route_by_word<T, 16, 16>(logits, tokens, E, ld, p, bias, ids, weights, err, st);
    if (E <= 512) return route_by_word<T, 16, 32>(logits, tokens, E, ld, p, bias, ids, weights, err, st);
    return route_by_word<T, 32, 32>(logits, tokens, E, ld, p, bias, ids, weights, err, st);
}

// By the experts (of a softmax over all of them) or the slots.
template <typename T>
struct Backward {
    const T* logits;
    int64_t tokens;
    int E;
    int64_t ld;
    const RouteParams& p;
    const int32_t* ids;
    const float* dw;
    T* dl;
    int64_t ld_out;
    int* err;
    cudaStream_t st;

    template <typename Kernel>
    cudaError_t run(Kernel kernel, int per_warp) const {
        const int per_block = kWarps * per_warp;
        return launch_pdl(false, kernel, static_cast<unsigned>((tokens + per_block - 1) / per_block), 32 * kWarps, 0, st, logits,
                          tokens, E, ld, p, ids, dw, dl, ld_out, err);
    }
    template <int kN>
    cudaError_t full() const {
        if (E <= 128) return run(route_topk_backward_full_kernel<T, 4, 8, kN>, 4);
        if (E <= 256) return run(route_topk_backward_full_kernel<T, 4, 16, kN>, 2);
        if (E <= 512) return run(route_topk_backward_full_kernel<T, 4, 32, kN>, 1);
        return run(route_topk_backward_full_kernel<T, 8, 32, kN>, 1);
    }
    cudaError_t operator()() const {
        if (p.score != MOE_SCORE_SOFTMAX || p.renormalize) {
            if (p.k <= 8) return run(route_topk_backward_kernel<T, 8>, 4);
            if (p.k <= 16) return run(route_topk_backward_kernel<T, 16>, 2);
            return run(route_topk_backward_kernel<T, 32>, 1);
        }
        constexpr int64_t kSize = sizeof(T);
        const int64_t bits = static_cast<int64_t>(reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(dl)) |
                             (ld * kSize) | (ld_out * kSize);
        if (bits % (4 * kSize) == 0) return full<4>();
        if (bits % (2 * kSize) == 0) return full<2>();
        return full<1>();
    }
};
template <typename T>
cudaError_t backward(const void* logits, int64_t tokens, int E, int64_t ld, const RouteParams& p, const int32_t* ids,
                     const float* dw, void* dl, int64_t ld_out, int* err, cudaStream_t st) {
    return Backward<T>{static_cast<const T*>(logits), tokens, E, ld, p, ids, dw, static_cast<T*>(dl), ld_out, err, st}();
}

}  // namespace

cudaError_t launch_route_topk(const void* logits, int type, int64_t T, int E, int64_t ld, const RouteParams& p,
                              const float* bias, int32_t* ids, float* weights, int* err, cudaStream_t st) {
    switch (type) {
        case NVFP4_TYPE_F32: return route_by_width<float>(logits, T, E, ld, p, bias, ids, weights, err, st);
        case NVFP4_TYPE_BF16: return route_by_width<__nv_bfloat16>(logits, T, E, ld, p, bias, ids, weights, err, st);
        default: return route_by_width<__half>(logits, T, E, ld, p, bias, ids, weights, err, st);
    }
}

cudaError_t launch_route_topk_backward(const void* logits, int type, int64_t T, int E, int64_t ld,
                                       const RouteParams& p, const int32_t* ids, const float* dw, void* dl,
                                       int64_t ld_out, int* err, cudaStream_t st) {
    switch (type) {
        case NVFP4_TYPE_F32: return backward<float>(logits, T, E, ld, p, ids, dw, dl, ld_out, err, st);
        case NVFP4_TYPE_BF16: return backward<__nv_bfloat16>(logits, T, E, ld, p, ids, dw, dl, ld_out, err, st);
        default: return backward<__half>(logits, T, E, ld, p, ids, dw, dl, ld_out, err, st);
    }
}

}  // namespace nvfp4
