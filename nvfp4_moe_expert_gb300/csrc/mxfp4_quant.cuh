// The MXFP4 row quantiser's device code, shared by the quantiser kernel (mxfp4.cu) and the product of
// few tokens, which quantises its rows in shared memory (linear.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "nvfp4_quant.cuh"
#include "ops.cuh"
#include "ptx.cuh"

namespace nvfp4 {
namespace {

// Eight elements of 16 bits, in one 16-byte word, as FP32.
__device__ __forceinline__ void expand8(const __nv_bfloat16*, const uint4& a, float (&v)[8]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void expand8(const __half*, const uint4& a, float (&v)[8]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// Eight consecutive elements as FP32; kVec: the first on a 16-byte boundary.
template <bool kVec>
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    if (kVec) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __ldg(p + i);
    }
}
template <bool kVec, typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
    uint4 a;
    if (kVec) {
        a = __ldg(reinterpret_cast<const uint4*>(p));
    } else {
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __ldg(q + 2 * i) | (static_cast<uint32_t>(__ldg(q + 2 * i + 1)) << 16);
        a = make_uint4(w[0], w[1], w[2], w[3]);
    }
    expand8(p, a, v);
}

// E8M0 code of a block whose largest magnitude has the FP32 bits `top` (NaN and Inf: 255).
__device__ __forceinline__ uint32_t e8m0_of_max(uint32_t top) {
    if (top >= 0x7F800000u) return 255u;
    if (top < 0x00800000u) return 0u;                 // zero or an FP32 subnormal: exponent below -127
    const int e = static_cast<int>(top >> 23) - 2;    // biased exponent of the scale
    return e > 0 ? static_cast<uint32_t>(e) : 0u;
}
// 2^(127 - code): the factor that divides by the scale; codes 0..252 occur (FP32 exponents).
__device__ __forceinline__ float e8m0_inverse(uint32_t code) { return __uint_as_float((254u - code) << 23); }

// The scale of a block whose largest magnitude (FP32 bits) this lane's eight elements have `top` of,
// with the block's four lanes in step (every lane of the warp calls this).
__device__ __forceinline__ uint32_t mx_block_scale(uint32_t top, int* err) {
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    const uint32_t code = e8m0_of_max(top);
    if (code == 255u) set_device_error(err, NVFP4_ERR_NONFINITE);
    return code;
}

// v scaled by 2^(127 - scale) as eight codes in one word; zeros where the scale is NaN.
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8], uint32_t scale) {
    const uint64_t inv = f32x2_splat(e8m0_inverse(scale == 255u ? 0u : scale));
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        uint64_t pair;
        asm("mov.b64 %0, {%1, %2};" : "=l"(pair) : "f"(v[j]), "f"(v[j + 1]));
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(pair) : "l"(pair), "l"(inv));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(q[j]), "=f"(q[j + 1]) : "l"(pair));
    }
    return scale == 255u ? 0u : e2m1x8(q);
}

// Eight elements as one word of codes, and their block's scale (in all four of its lanes).
__device__ __forceinline__ void mx_quantize8(const float (&v)[8], uint32_t& word, uint32_t& scale, int* err) {
    uint32_t top = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    scale = mx_block_scale(top, err);
    word = mx_codes8(v, scale);
}

// The same of eight 16-bit elements in one word; the maximum is taken on pairs of them (NaN wins).
__device__ __forceinline__ uint32_t max_pairs(const __nv_bfloat16*, uint32_t a, uint32_t b) { return bf16x2_max_nan(a, b); }
__device__ __forceinline__ uint32_t max_pairs(const __half*, uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t high_f32_bits(const __nv_bfloat16*, uint32_t m) { return m & 0xFFFF0000u; }
__device__ __forceinline__ uint32_t high_f32_bits(const __half*, uint32_t m) {
    return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(m >> 16))));
}
template <typename X>
__device__ __forceinline__ void mx_quantize_word(const X* type, const uint4& w, uint32_t& word, uint32_t& scale, int* err) {
    constexpr uint32_t kAbs = 0x7FFF7FFFu;
    uint32_t m = max_pairs(type, max_pairs(type, w.x & kAbs, w.y & kAbs), max_pairs(type, w.z & kAbs, w.w & kAbs));
    m = max_pairs(type, m, m << 16);                  // high half: the largest of both halves
    scale = mx_block_scale(high_f32_bits(type, m), err);
    float v[8];
    expand8(type, w, v);
    word = mx_codes8(v, scale);
}

// Eight elements of a lane as they are loaded: one word where they are 16 bits wide and aligned.
template <typename X, bool kVec>
struct MxHeld {
    static constexpr bool one_word = kVec && sizeof(X) == 2;
    uint4 w;
    float f[one_word ? 1 : 8];
    __device__ __forceinline__ void load(const X* src, bool live) {
        if constexpr (one_word) {
            w = live ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0u, 0u, 0u, 0u);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = 0.0f;
            if (live) load8<kVec>(src, f);
        }
    }
    // the code word and, in every lane of a block's four, the scale
    __device__ __forceinline__ void quantise(uint32_t& word, uint32_t& scale, int* err) const {
        if constexpr (one_word) {
            mx_quantize_word(static_cast<const X*>(nullptr), w, word, scale, err);
        } else {
            mx_quantize8(f, word, scale, err);
        }
    }
};

}  // namespace
}  // namespace nvfp4
