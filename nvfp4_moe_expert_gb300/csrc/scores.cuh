// What the kernels of router logits share: elements of the three types, wide loads and stores, and
// the scores (softmax terms and sigmoids) that the routing, its gradient and the balance loss go by.
#pragma once

#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace nvfp4 {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// kN consecutive elements (kN * sizeof(T) <= 16, a power of two, and the address a multiple of it).
template <int kBytes>
struct Word;
template <>
struct Word<2> { using type = unsigned short; };
template <>
struct Word<4> { using type = uint32_t; };
template <>
struct Word<8> { using type = uint2; };
template <>
struct Word<16> { using type = uint4; };
template <typename T, int kN>
struct Vec {
    union {
        typename Word<kN * sizeof(T)>::type word;
        T e[kN];
    };
    __device__ Vec() {}
};
template <typename T, int kN>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[kN]) {
    Vec<T, kN> w;
    w.word = __ldg(reinterpret_cast<const decltype(w.word)*>(p));
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = to_f32(w.e[i]);
}
template <typename T, int kN>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[kN]) {
    Vec<T, kN> w;
#pragma unroll
    for (int i = 0; i < kN; ++i) w.e[i] = from_f32<T>(v[i]);
    *reinterpret_cast<decltype(w.word)*>(p) = w.word;
}
template <typename T>
__device__ __forceinline__ float load_one(const T* p) {
    float v[1];
    load_vec<T, 1>(p, v);
    return v[0];
}

// A logit with NaN replaced by the mask.
__device__ __forceinline__ float masked_nan(float l) { return l != l ? -INFINITY : l; }

// The terms of a softmax with largest logit m are expf(l - m), 0 where l is masked.  Where m is infinite l and m
// are replaced by what gives them: all masked (m = -inf), or the +inf ones equal and the others 0.
__device__ __forceinline__ float softmax_shift(float m) { return m == INFINITY || m == -INFINITY ? 0.0f : m; }
__device__ __forceinline__ float softmax_logit(float l, float m) { return m == INFINITY ? (l == INFINITY ? 0.0f : -INFINITY) : l; }
// The quotient of a term t <= 1 by a sum 1 <= d <= 1024 with rc = RN(1 / d): t rc and Markstein's step, the rounded quotient
// but for t below 2^-100, where the step's remainder underflows.  (With __fdiv_rn for every expert the kernel took 80
// registers instead of 64, and 65537 x 256 without scores in the order 34.1 us instead of 29.8.)
__device__ __forceinline__ float quotient(float t, float d, float rc) {
    const float q = __fmul_rn(t, rc);
    return __fmaf_rn(__fmaf_rn(-q, d, t), rc, q);
}

// A sigmoid by t = e^-|l|, which does not overflow: s = y where l >= 0 and t y below, y = 1 / (1 + t); 0 at -inf, 1 at +inf.
// 1 - s is the sigmoid of -l.  (By 1 / (1 + e^-l) scores below e^-88, in FP32's range, were 0.)
// y: 1 <= d <= 2, so one Newton-Raphson step, y + y (1 - d y), takes the hardware's reciprocal (2^-23) to within rounding
// (65537 x 256 in 8 groups 59.4 us a call with __frcp_rn, whose range every d is checked for, 51.2 when it was replaced).
__device__ __forceinline__ float reciprocal_1_2(float d) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(d));
    return __fmaf_rn(y, __fmaf_rn(-d, y, 1.0f), y);
}
__device__ __forceinline__ float sigmoid(float l) {
    const float t = expf(-fabsf(l)), y = reciprocal_1_2(1.0f + t);
    return l < 0.0f ? t * y : y;
}
// Sigmoids relative to that of the largest chosen logit, m: e^(min(l, 0) - min(m, 0)) y(l), a common factor of e^-min(m, 0)
// more than the sigmoids, so their ratios do not underflow with them.  All 0 where every chosen logit is masked or lies
// below -709 (a mask by the type's lowest value), where a score is 0 in 64 bits too.
constexpr float kLowestLogit = -709.0f;
__device__ __forceinline__ float sigmoid_ratio(float l, float m) {
    const float y = reciprocal_1_2(1.0f + expf(-fabsf(l)));
    return m < kLowestLogit ? 0.0f : expf(fminf(l, 0.0f) - fminf(m, 0.0f)) * y;
}

}  // namespace nvfp4
