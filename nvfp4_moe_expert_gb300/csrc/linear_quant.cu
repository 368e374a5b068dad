// The NVFP4 quantisation of a dense product's x: bit for bit what nvfp4_quantize_rows gives for its rows (the
// arithmetic is nvfp4_quant.cuh's) but for the NaN outer scale of a row with an Inf or NaN, laid out for few rows as
// well as many.
//
// A row is taken by 1, 2 or 4 warps, each lane holding at most four blocks of 16 elements (32 consecutive bytes
// each, a warp's side by side), so the row is read once, the maximum found and the codes made from the
// registers.  The rows kernel of quant.cu has whole 64-element groups to a lane, up to 256 elements one after
// the other: 6 us for one row of 4096 to 16 of them, where this one takes 2.
//
// The rows past T of the last 128-row tile are not written: what the tensor cores make of them is not read.
#include "nvfp4_quant.cuh"
#include "ops.cuh"

namespace nvfp4 {
namespace {

constexpr int kMaxHeld = 4;                          // blocks of 16 to a lane
constexpr int kPassCols = 32 * kBlock;               // columns of a warp's pass: one block to a lane
constexpr int kWarpsQ = 4;                           // warps of a thread block

template <int kWarpsPerRow, int kHeld>
__global__ void __launch_bounds__(32 * kWarpsQ, 8)
    quantize_x_kernel(const uint16_t* __restrict__ x, int64_t rows, int cols, int64_t ld, uint8_t* __restrict__ codes,
                      uint8_t* __restrict__ sf, float* __restrict__ g, int* err) {
    constexpr int kRows = kWarpsQ / kWarpsPerRow;    // rows of a thread block
    __shared__ uint32_t s_top[2][kWarpsQ];
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = warp % kWarpsPerRow, slot = warp / kWarpsPerRow;
    int turn = 0;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * kRows; base < rows; base += static_cast<int64_t>(gridDim.x) * kRows) {
        const int64_t r = base + slot;
        uint4 v[kHeld][2];
        uint32_t top = 0u, block_top[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int c = kBlock * (32 * (i * kWarpsPerRow + part) + lane);
            v[i][0] = v[i][1] = make_uint4(0u, 0u, 0u, 0u);
            if (r < rows && c < cols) {
                const uint4* s = reinterpret_cast<const uint4*>(x + r * ld + c);
                v[i][0] = __ldg(s);
                v[i][1] = __ldg(s + 1);
            }
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            block_top[i] = block_absmax_bits(v[i][0], v[i][1]);
            top = max(top, block_top[i]);
        }
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        if (kWarpsPerRow > 1) {
            if (lane == 0) s_top[turn][warp] = top;
            __syncthreads();                          // the other turn's values are read before the next one's
#pragma unroll
            for (int i = 0; i < kWarpsPerRow; ++i) top = max(top, s_top[turn][slot * kWarpsPerRow + i]);
            turn ^= 1;
        }
        if (r >= rows) continue;                      // past the last row: nothing to write
        const bool first = part == 0 && lane == 0;
        const float gr = nv_outer_scale(top, first ? err : nullptr);
        if (first) g[r] = gr;
        const NvRow row = nv_row(gr);
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int c = kBlock * (32 * (i * kWarpsPerRow + part) + lane);
            if (c >= cols) continue;
            uint32_t w0, w1, scale;
            nv_quantize16(v[i][0], v[i][1], __uint_as_float(block_top[i]), row, w0, w1, scale);
            *reinterpret_cast<uint2*>(codes + r * (cols / 2) + c / 2) = make_uint2(w0, w1);
            sf[sf_offset(r, c / kBlock, cols)] = static_cast<uint8_t>(scale);
        }
    }
}

template <int kWarpsPerRow, int kHeld>
cudaError_t launch(const uint16_t* x, int64_t rows, int cols, int64_t ld, uint8_t* codes, uint8_t* sf, float* g, int* err,
                   cudaStream_t st) {
    const int64_t blocks = (rows + kWarpsQ / kWarpsPerRow - 1) / (kWarpsQ / kWarpsPerRow);
    const int64_t most = static_cast<int64_t>(device_sm_count()) * 8;
    return launch_pdl(false, quantize_x_kernel<kWarpsPerRow, kHeld>, static_cast<unsigned>(blocks < most ? blocks : most),
                      32 * kWarpsQ, 0, st, x, rows, cols, ld, codes, sf, g, err);
}

}  // namespace

cudaError_t launch_nvfp4_quantize_x(const uint16_t* x, int64_t rows, int cols, int64_t ld, uint8_t* codes, uint8_t* sf,
                                    float* g, int* err, cudaStream_t st) {
    static_assert(4 * kMaxHeld * kPassCols >= 8192, "the widest row");
    const int passes = (cols + kPassCols - 1) / kPassCols;
    if (passes <= 1) return launch<1, 1>(x, rows, cols, ld, codes, sf, g, err, st);
    if (passes <= 2) return launch<1, 2>(x, rows, cols, ld, codes, sf, g, err, st);
    if (passes <= 3) return launch<1, 3>(x, rows, cols, ld, codes, sf, g, err, st);
    if (passes <= 4) return launch<1, 4>(x, rows, cols, ld, codes, sf, g, err, st);
    if (passes <= 6) return launch<2, 3>(x, rows, cols, ld, codes, sf, g, err, st);
    if (passes <= 8) return launch<2, 4>(x, rows, cols, ld, codes, sf, g, err, st);
    if (passes <= 12) return launch<4, 3>(x, rows, cols, ld, codes, sf, g, err, st);
    return launch<4, 4>(x, rows, cols, ld, codes, sf, g, err, st);
}

}  // namespace nvfp4
