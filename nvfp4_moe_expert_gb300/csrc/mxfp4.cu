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

// Four threads per block of 32 elements, 16 threads per word of four scales: thread u of a row
// takes elements 8u..8u+7, so the row is read in consecutive 16-byte (BF16, FP16) pieces.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads)
    mxfp4_quantize_rows_kernel(const T* __restrict__ x, int64_t rows, int64_t cols, int64_t ld,
                               uint8_t* __restrict__ codes, uint8_t* __restrict__ sf, int* err) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t per_row = 16 * mx_sf_tiles(cols);                  // threads per row
    const int64_t rows_pad = (rows + kTileM - 1) / kTileM * kTileM;
    const int64_t total = rows_pad * per_row;
    const int lane = threadIdx.x & 31;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i - lane < total;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const bool in = i < total;                                   // whole groups of 16 threads
        const int64_t r = in ? i / per_row : 0;
        const int64_t u = in ? i - r * per_row : 0;
        const bool live = in && r < rows && 8 * u < cols;            // whole blocks: cols % 32 == 0
        float v[8];
        if (live) {
            load8<kVec>(x + r * ld + 8 * u, v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        }
        uint32_t word, scale;
        mx_quantize8(v, word, scale, err);
        uint32_t scales = scale;                                     // this group of 16 threads' four scales
        scales |= __shfl_down_sync(0xFFFFFFFFu, scale, 4) << 8;
        scales |= __shfl_down_sync(0xFFFFFFFFu, scale, 8) << 16;
        scales |= __shfl_down_sync(0xFFFFFFFFu, scale, 12) << 24;
        if (in) {
            if (8 * u < cols) *reinterpret_cast<uint32_t*>(codes + r * (cols / 2) + 4 * u) = word;
            if ((u & 15) == 0) *reinterpret_cast<uint32_t*>(sf + mx_sf_offset(r, u / 4, cols)) = scales;
        }
    }
}

// The value of element code c (E2M1) times 2^(scale - 127), exact in BF16 and FP32.
__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const uint32_t m = c & 7u;
    const float v = m < 2u ? 0.5f * static_cast<float>(m)
                           : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
    return (c & 8u) ? -v : v;
}
__device__ __forceinline__ float e8m0_value(uint32_t code) {
    if (code == 255u) return __uint_as_float(0x7FC00000u);
    return code == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(code << 23);
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8], bool vec);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&v)[8], bool vec) {
    if (vec) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = v[i];
    }
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[8], bool vec) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    if (vec) {
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        uint16_t* q = reinterpret_cast<uint16_t*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    mxfp4_dequantize_rows_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ sf, int64_t rows,
                                 int64_t cols, T* __restrict__ out, int64_t ld, bool vec) {
    const int64_t per_row = cols / 8;
    const int64_t total = rows * per_row;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t r = i / per_row, u = i - r * per_row;
        const uint32_t c = __ldg(reinterpret_cast<const uint32_t*>(codes + r * (cols / 2)) + u);
        const float s = e8m0_value(__ldg(sf + mx_sf_offset(r, u / 4, cols)));
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = e2m1_value(c >> (4 * j)) * s;
        store8(out + r * ld + 8 * u, v, vec);
    }
}

unsigned grid_for(int64_t threads) {
    const int64_t most = static_cast<int64_t>(device_sm_count()) * 8;
    const int64_t blocks = (threads + kThreads - 1) / kThreads;
    return static_cast<unsigned>(blocks < most ? blocks : most);
}

bool aligned16(const void* p, int64_t ld, int size) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * size) % 16 == 0;
}

template <typename T>
cudaError_t quantize(const void* x, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes, uint8_t* sf, int* err,
                     cudaStream_t st) {
    const int64_t rows_pad = (rows + kTileM - 1) / kTileM * kTileM;
    const unsigned grid = grid_for(rows_pad * 16 * mx_sf_tiles(cols));
    auto k = aligned16(x, ld, sizeof(T)) ? mxfp4_quantize_rows_kernel<T, true> : mxfp4_quantize_rows_kernel<T, false>;
    return launch_pdl(false, k, grid, kThreads, 0, st, static_cast<const T*>(x), rows, cols, ld, codes, sf, err);
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
    const unsigned grid = grid_for(rows * (cols / 8));
    if (type == NVFP4_TYPE_F32)
        return launch_pdl(false, mxfp4_dequantize_rows_kernel<float>, grid, kThreads, 0, st, codes, sf, rows, cols,
                          static_cast<float*>(out), ld, aligned16(out, ld, 4));
    return launch_pdl(false, mxfp4_dequantize_rows_kernel<__nv_bfloat16>, grid, kThreads, 0, st, codes, sf, rows, cols,
                      static_cast<__nv_bfloat16*>(out), ld, aligned16(out, ld, 2));
}

}  // namespace nvfp4
