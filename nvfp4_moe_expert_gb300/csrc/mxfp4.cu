// MXFP4 rows: E2M1 elements with one E8M0 (power of two) scale per 32 of them, in the storage the
// dense product reads (codes row-major, scales in 512-byte tiles of 128 rows x 128 columns).
//
//   scale of a block: 2^(floor(log2 max|x|) - 2), the exponent held to [-127, 127]: the largest
//   magnitude lands in [4, 8), of which E2M1 (largest value 6) saturates (6, 8); a zero block has
//   the smallest scale and zero codes; a block with an Inf or NaN has the NaN scale 255
//   code = E2M1(x / scale), to nearest, ties to even, saturating: the quotient by a power of two
//   is exact, so there is one rounding
//
// Both ways are bound by memory: 16384 x 8192 BF16 to codes 52 us (340 MB, 6.5 TB/s), back 54 us (6.3 TB/s).
#include "mxfp4_quant.cuh"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;

// A lane takes whole blocks of 32 elements; a row's blocks are counted with those that fill up its last
// scale word, and the rows with those that fill up the last tile (both get zeros).
constexpr int kHeld = 2;           // blocks of a lane in flight

struct Blocks {
    uint32_t per_row, live, count;   // blocks of a row, those with elements, blocks of all rows
};

template <typename T, int kAlign>
__global__ void __launch_bounds__(kThreads)
    mxfp4_quantize_rows_kernel(const T* __restrict__ x, int64_t rows, int64_t cols, int64_t ld, Blocks blocks,
                               uint8_t* __restrict__ codes, uint8_t* __restrict__ sf, int* err) {
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t step = gridDim.x * kThreads;
    for (uint32_t first = blockIdx.x * kThreads + threadIdx.x; first < blocks.count; first += kHeld * step) {
        MxBlock<T, kAlign> held[kHeld];
        uint32_t r[kHeld], at[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const uint32_t b = first + i * step;
            r[i] = b / blocks.per_row;
            at[i] = b - r[i] * blocks.per_row;
            held[i].load(x + r[i] * ld + at[i] * kMxBlock, b < blocks.count && r[i] < rows && at[i] < blocks.live);
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            if (first + i * step >= blocks.count) break;
            uint4 c;
            uint32_t scale;
            held[i].quantise(c, scale, err);
            if (at[i] < blocks.live) *reinterpret_cast<uint4*>(codes + r[i] * (cols / 2) + at[i] * (kMxBlock / 2)) = c;
            sf[mx_sf_offset(r[i], at[i], cols)] = static_cast<uint8_t>(scale);
        }
    }
}

__device__ __forceinline__ float e8m0_value(uint32_t code) {
    if (code == 255u) return __uint_as_float(0x7FC00000u);
    return code == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(code << 23);
}

// Four E2M1 codes (16 bits of `c`) as two words of BF16 pairs: a byte permutation looks the low and the high
// bytes of the eight magnitudes up (0, 0.5, 1, 1.5, 2, 3, 4, 6 = 0000, 3F00, 3F80, 3FC0, 4000, 4040, 4080,
// 40C0), and the codes' sign bits go on top.
__device__ __forceinline__ void e2m1x4_bf16(uint32_t c, uint32_t& w0, uint32_t& w1) {
    const uint32_t sel = c & 0x7777u;
    const uint32_t lo = __byte_perm(0xC0800000u, 0xC0804000u, sel), hi = __byte_perm(0x3F3F3F00u, 0x40404040u, sel);
    w0 = __byte_perm(lo, hi, 0x5140u) | ((c & 0x8u) << 12) | ((c & 0x80u) << 24);
    w1 = __byte_perm(lo, hi, 0x7362u) | ((c & 0x800u) << 4) | ((c & 0x8000u) << 16);
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// One block of 32 values to a lane: 16 bytes of codes in, 64 (BF16) or 128 (FP32) bytes out.  The product
// with a power of two is exact in BF16 (its smallest subnormal is 2^-133, the smallest product 2^-128).
template <typename T, int kAlign>
__device__ __forceinline__ void store_block(T* p, const uint4& codes, uint32_t scale) {
    const uint32_t s16 = __float_as_uint(e8m0_value(scale)) >> 16;
    const uint32_t s2 = s16 | (s16 << 16);
    const uint32_t c[4] = {codes.x, codes.y, codes.z, codes.w};
    constexpr int kWords = 8 * sizeof(T);
    uint32_t w[kWords];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t v[2];
        e2m1x4_bf16(c[i >> 1] >> (16 * (i & 1)), v[0], v[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            v[j] = bf16x2_mul(v[j], s2);
            if constexpr (sizeof(T) == 2) w[2 * i + j] = v[j];
            else w[4 * i + 2 * j] = v[j] << 16, w[4 * i + 2 * j + 1] = v[j] & 0xFFFF0000u;
        }
    }
    if constexpr (kAlign == 2) {
#pragma unroll
        for (int i = 0; i < kWords; i += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(reinterpret_cast<uint32_t*>(p) + i),
                         "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]),
                         "r"(w[i + 7])
                         : "memory");
    } else if constexpr (kAlign == 1) {
#pragma unroll
        for (int i = 0; i < kWords; i += 4)
            *(reinterpret_cast<uint4*>(p) + i / 4) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) reinterpret_cast<uint32_t*>(p)[i] = w[i];
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
    }
}

template <typename T, int kAlign>
__global__ void __launch_bounds__(kThreads)
    mxfp4_dequantize_rows_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ sf, int64_t cols,
                                 Blocks blocks, T* __restrict__ out, int64_t ld) {
    const uint32_t step = gridDim.x * kThreads;
    for (uint32_t first = blockIdx.x * kThreads + threadIdx.x; first < blocks.count; first += kHeld * step) {
        uint4 c[kHeld];
        uint32_t scale[kHeld], r[kHeld], at[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const uint32_t b = first + i * step;
            r[i] = b / blocks.per_row;
            at[i] = b - r[i] * blocks.per_row;
            if (b < blocks.count) {
                c[i] = __ldg(reinterpret_cast<const uint4*>(codes + r[i] * (cols / 2)) + at[i]);
                scale[i] = __ldg(sf + mx_sf_offset(r[i], at[i], cols));
            }
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            if (first + i * step < blocks.count) store_block<T, kAlign>(out + r[i] * ld + at[i] * kMxBlock, c[i], scale[i]);
        }
    }
}

// Thread blocks that fill the SMs.
unsigned grid_for(uint32_t count) {
    const uint32_t blocks = (count + kThreads - 1) / kThreads, most = static_cast<uint32_t>(device_sm_count()) * 8;
    return blocks < most ? blocks : most;
}

template <typename T>
cudaError_t quantize(const void* x, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes, uint8_t* sf, int* err,
                     cudaStream_t st) {
    const int64_t rows_pad = (rows + kTileM - 1) / kTileM * kTileM;
    const uint32_t per_row = static_cast<uint32_t>(4 * mx_sf_tiles(cols));
    const Blocks b = {per_row, static_cast<uint32_t>(cols / kMxBlock), static_cast<uint32_t>(rows_pad * per_row)};
    const int align = mx_align(x, ld, sizeof(T));
    auto k = align == 2   ? mxfp4_quantize_rows_kernel<T, 2>
             : align == 1 ? mxfp4_quantize_rows_kernel<T, 1>
                          : mxfp4_quantize_rows_kernel<T, 0>;
    return launch_pdl(false, k, grid_for(b.count), kThreads, 0, st, static_cast<const T*>(x), rows, cols, ld, b, codes, sf,
                      err);
}

template <typename T>
cudaError_t dequantize(const uint8_t* codes, const uint8_t* sf, int64_t rows, int64_t cols, void* out, int64_t ld,
                       cudaStream_t st) {
    const uint32_t per_row = static_cast<uint32_t>(cols / kMxBlock);
    const Blocks b = {per_row, per_row, static_cast<uint32_t>(rows * per_row)};
    const int align = mx_align(out, ld, sizeof(T));
    auto k = align == 2   ? mxfp4_dequantize_rows_kernel<T, 2>
             : align == 1 ? mxfp4_dequantize_rows_kernel<T, 1>
                          : mxfp4_dequantize_rows_kernel<T, 0>;
    return launch_pdl(false, k, grid_for(b.count), kThreads, 0, st, codes, sf, cols, b, static_cast<T*>(out), ld);
}

}  // namespace

cudaError_t launch_mxfp4_quantize_rows(const void* x, int type, int64_t rows, int64_t cols, int64_t ld,
                                       uint8_t* codes, uint8_t* sf, int* err, cudaStream_t st) {
    switch (type) {
        case NVFP4_TYPE_F32: return quantize<float>(x, rows, cols, ld, codes, sf, err, st);
        case NVFP4_TYPE_BF16: return quantize<__nv_bfloat16>(x, rows, cols, ld, codes, sf, err, st);
        default: return quantize<__half>(x, rows, cols, ld, codes, sf, err, st);
    }
}

cudaError_t launch_mxfp4_dequantize_rows(const uint8_t* codes, const uint8_t* sf, int64_t rows, int64_t cols,
                                         void* out, int type, int64_t ld, cudaStream_t st) {
    return type == NVFP4_TYPE_F32 ? dequantize<float>(codes, sf, rows, cols, out, ld, st)
                                  : dequantize<__nv_bfloat16>(codes, sf, rows, cols, out, ld, st);
}

}  // namespace nvfp4
