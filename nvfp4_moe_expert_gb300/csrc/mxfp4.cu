// MXFP4 rows: E2M1 elements with one E8M0 (power of two) scale per 32 of them, in the storage the
// dense product reads (codes row-major, scales in 512-byte tiles of 128 rows x 128 columns).
//
//   scale of a block: 2^(floor(log2 max|x|) - 2), the exponent held to [-127, 127]: the largest
//   magnitude lands in [4, 8), of which E2M1 (largest value 6) saturates (6, 8); a zero block has
//   the smallest scale and zero codes; a block with an Inf or NaN has the NaN scale 255
//   code = E2M1(x / scale), to nearest, ties to even, saturating: the quotient by a power of two
//   is exact, so there is one rounding
#include "mxfp4_quant.cuh"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;

// A warp's piece: 256 columns of a row (8 elements, a quarter of a block, to a lane, read as one 16-byte
// word of BF16 or FP16), kPieces of them at once so that enough loads are in flight; pieces are counted
// row by row.  One 4-byte word of codes to a lane (128 bytes to a warp), one of scales to 16 lanes.
constexpr int kPieces = 4;

struct Pieces {
    uint32_t per_row, count;   // pieces of a row and of all rows
    __device__ __forceinline__ void place(uint32_t i, uint32_t& r, uint32_t& at) const {
        r = i / per_row;
        at = i - r * per_row;
    }
};

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads)
    mxfp4_quantize_rows_kernel(const T* __restrict__ x, int64_t rows, int64_t cols, int64_t ld, Pieces pieces,
                               uint8_t* __restrict__ codes, uint8_t* __restrict__ sf, int* err) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const uint32_t warps = gridDim.x * (kThreads / 32);
    const int sf_cols = static_cast<int>(mx_sf_tiles(cols)) * kMxTileCols;
    for (uint32_t w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); w * kPieces < pieces.count; w += warps) {
        MxHeld<T, kVec> held[kPieces];
        uint32_t r, at;
        pieces.place(w * kPieces, r, at);
        uint32_t r_of[kPieces], at_of[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            r_of[i] = r;
            at_of[i] = at;
            const int c = static_cast<int>(at) * 256 + 8 * lane;
            held[i].load(x + r * ld + c, r < rows && c < cols);
            if (++at == pieces.per_row) {
                at = 0;
                ++r;
            }
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            if (w * kPieces + i >= pieces.count) break;
            const int c = static_cast<int>(at_of[i]) * 256 + 8 * lane;
            uint32_t word, scale;
            held[i].quantise(word, scale, err);
            uint32_t scales = scale;                                 // 16 lanes' four scales, in the first of them
            scales |= __shfl_down_sync(0xFFFFFFFFu, scale, 4) << 8;
            scales |= __shfl_down_sync(0xFFFFFFFFu, scale, 8) << 16;
            scales |= __shfl_down_sync(0xFFFFFFFFu, scale, 12) << 24;
            if (c < cols) *reinterpret_cast<uint32_t*>(codes + r_of[i] * (cols / 2) + c / 2) = word;
            if ((lane & 15) == 0 && c < sf_cols)
                *reinterpret_cast<uint32_t*>(sf + mx_sf_offset(r_of[i], c / kMxBlock, cols)) = scales;
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

// Eight values to a lane: one word of codes in, 16 (BF16) or 32 (FP32) bytes out.  The product with a
// power of two is exact in BF16 (its smallest subnormal is 2^-133, the smallest product 2^-128).
template <typename T>
__device__ __forceinline__ void store8(T* p, uint32_t c, uint32_t scale, bool vec) {
    const uint32_t s16 = __float_as_uint(e8m0_value(scale)) >> 16;
    const uint32_t s2 = s16 | (s16 << 16);
    uint32_t w[4];
    e2m1x4_bf16(c, w[0], w[1]);
    e2m1x4_bf16(c >> 16, w[2], w[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16x2_mul(w[i], s2);
    if constexpr (sizeof(T) == 2) {
        if (vec) {
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            uint16_t* q = reinterpret_cast<uint16_t*>(p);
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
        }
    } else {
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
        if (vec) {
            reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = v[i];
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    mxfp4_dequantize_rows_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ sf, int64_t rows,
                                 int64_t cols, Pieces pieces, T* __restrict__ out, int64_t ld, bool vec) {
    const int lane = threadIdx.x & 31;
    const uint32_t warps = gridDim.x * (kThreads / 32);
    for (uint32_t w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); w * kPieces < pieces.count; w += warps) {
        uint32_t r, at, c[kPieces], scale[kPieces], r_of[kPieces], at_of[kPieces];
        pieces.place(w * kPieces, r, at);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            r_of[i] = r;
            at_of[i] = at;
            const int k = static_cast<int>(at) * 256 + 8 * lane;
            c[i] = scale[i] = 0u;
            if (r < rows && k < cols) {
                c[i] = __ldg(reinterpret_cast<const uint32_t*>(codes + r * (cols / 2) + k / 2));
                scale[i] = __ldg(sf + mx_sf_offset(r, k / kMxBlock, cols));
            }
            if (++at == pieces.per_row) {
                at = 0;
                ++r;
            }
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int k = static_cast<int>(at_of[i]) * 256 + 8 * lane;
            if (r_of[i] < rows && k < cols) store8(out + r_of[i] * ld + k, c[i], scale[i], vec);
        }
    }
}

// Pieces of `rows` rows (fewer than 2^31, as the entry points see to), and enough blocks to fill the SMs.
void split(int64_t rows, int64_t cols, Pieces& p, unsigned& grid) {
    const int64_t per_row = (cols + 255) / 256, count = rows * per_row;
    p = {static_cast<uint32_t>(per_row), static_cast<uint32_t>(count)};
    const int64_t blocks = (count + kPieces * (kThreads / 32) - 1) / (kPieces * (kThreads / 32));
    const int64_t most = static_cast<int64_t>(device_sm_count()) * 8;
    grid = static_cast<unsigned>(blocks < most ? blocks : most);
}

bool aligned16(const void* p, int64_t ld, int size) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * size) % 16 == 0;
}

template <typename T>
cudaError_t quantize(const void* x, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes, uint8_t* sf, int* err,
                     cudaStream_t st) {
    Pieces p;
    unsigned grid;
    split((rows + kTileM - 1) / kTileM * kTileM, cols, p, grid);
    auto k = aligned16(x, ld, sizeof(T)) ? mxfp4_quantize_rows_kernel<T, true> : mxfp4_quantize_rows_kernel<T, false>;
    return launch_pdl(false, k, grid, kThreads, 0, st, static_cast<const T*>(x), rows, cols, ld, p, codes, sf, err);
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
    Pieces p;
    unsigned grid;
    split(rows, cols, p, grid);
    if (type == NVFP4_TYPE_F32)
        return launch_pdl(false, mxfp4_dequantize_rows_kernel<float>, grid, kThreads, 0, st, codes, sf, rows, cols, p,
                          static_cast<float*>(out), ld, aligned16(out, ld, 4));
    return launch_pdl(false, mxfp4_dequantize_rows_kernel<__nv_bfloat16>, grid, kThreads, 0, st, codes, sf, rows, cols, p,
                      static_cast<__nv_bfloat16*>(out), ld, aligned16(out, ld, 2));
}

}  // namespace nvfp4
