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

// E8M0 code of a block whose largest magnitude has the FP32 bits `top` (NaN and Inf: 255).
__device__ __forceinline__ uint32_t e8m0_of_max(uint32_t top) {
    if (top >= 0x7F800000u) return 255u;
    if (top < 0x00800000u) return 0u;                 // zero or an FP32 subnormal: exponent below -127
    const int e = static_cast<int>(top >> 23) - 2;    // biased exponent of the scale
    return e > 0 ? static_cast<uint32_t>(e) : 0u;
}
// 2^(127 - code): the factor that divides by the scale; codes 0..252 occur (FP32 exponents).
__device__ __forceinline__ float e8m0_inverse(uint32_t code) { return __uint_as_float((254u - code) << 23); }

// Pairs of 16-bit elements: the larger of each (NaN wins), and their FP32 values.
__device__ __forceinline__ uint32_t max_pairs(const __nv_bfloat16*, uint32_t a, uint32_t b) { return bf16x2_max_nan(a, b); }
__device__ __forceinline__ uint32_t max_pairs(const __half*, uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ void expand_pair(const __nv_bfloat16*, uint32_t w, float& lo, float& hi) {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ void expand_pair(const __half*, uint32_t w, float& lo, float& hi) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    lo = f.x;
    hi = f.y;
}

// One block of 32 elements, held by one lane as it was loaded: no lane needs another's values, and the
// scale's few instructions are shared by 32 elements.  (With 8 elements to a lane the rows kernel issued
// 3.5 times the instructions an element and was bound by them.)
// kAlign: rows start on 32-byte (2) or 16-byte (1) boundaries, or on the elements' own (0).
template <typename X, int kAlign>
struct MxBlock {
    static constexpr int kWords = 8 * sizeof(X);
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const X* src, bool live) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
        if (!live) return;
        if constexpr (kAlign == 2) {
#pragma unroll
            for (int i = 0; i < kWords; i += 8)
                asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                             : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]), "=r"(w[i + 4]), "=r"(w[i + 5]),
                               "=r"(w[i + 6]), "=r"(w[i + 7])
                             : "l"(reinterpret_cast<const uint32_t*>(src) + i));
        } else if constexpr (kAlign == 1) {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + i / 4);
                w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
            }
        } else if constexpr (sizeof(X) == 4) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(src) + i);
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const uint16_t* q = reinterpret_cast<const uint16_t*>(src) + 2 * i;
                w[i] = __ldg(q) | (static_cast<uint32_t>(__ldg(q + 1)) << 16);
            }
        }
    }

    // FP32 bits of the largest magnitude; at least 0x7F800000 if there is an Inf or NaN.
    __device__ __forceinline__ uint32_t top() const {
        if constexpr (sizeof(X) == 4) {
            uint32_t m = 0u;
#pragma unroll
            for (int i = 0; i < kWords; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
            return m;
        } else {
            const X* type = nullptr;
            uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
            for (int i = 1; i < kWords; ++i) m = max_pairs(type, m, w[i] & 0x7FFF7FFFu);
            float lo, hi;
            expand_pair(type, m, lo, hi);
            return max(__float_as_uint(lo), __float_as_uint(hi));
        }
    }

    // The block's 32 codes and its scale.
    __device__ __forceinline__ void quantise(uint4& codes, uint32_t& scale, int* err) const {
        scale = e8m0_of_max(top());
        if (scale == 255u) set_device_error(err, NVFP4_ERR_NONFINITE);
        const uint64_t inv = f32x2_splat(e8m0_inverse(scale == 255u ? 0u : scale));
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float q[8];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                float lo, hi;
                if constexpr (sizeof(X) == 4) lo = __uint_as_float(w[8 * i + j]), hi = __uint_as_float(w[8 * i + j + 1]);
                else expand_pair(static_cast<const X*>(nullptr), w[4 * i + j / 2], lo, hi);
                uint64_t pair;
                asm("mov.b64 %0, {%1, %2};" : "=l"(pair) : "f"(lo), "f"(hi));
                asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(pair) : "l"(pair), "l"(inv));
                asm("mov.b64 {%0, %1}, %2;" : "=f"(q[j]), "=f"(q[j + 1]) : "l"(pair));
            }
            c[i] = scale == 255u ? 0u : e2m1x8(q);
        }
        codes = make_uint4(c[0], c[1], c[2], c[3]);
    }
};

// kAlign of rows [..][ld] of elements of `size` bytes at p.
inline int mx_align(const void* p, int64_t ld, int size) {
    const int64_t bits = static_cast<int64_t>(reinterpret_cast<uintptr_t>(p)) | (ld * size);
    return bits % 32 == 0 ? 2 : bits % 16 == 0 ? 1 : 0;
}

}  // namespace
}  // namespace nvfp4
