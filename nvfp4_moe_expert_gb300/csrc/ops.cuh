// Host launchers of the routing operators and of the dense 4-bit products (each defined in the
// .cu that holds its kernels).  Arguments have been checked by the C entry points.
#pragma once

#include "common.cuh"

namespace nvfp4 {

struct RouteParams {
    int score, k, n_group, topk_group, group_score, renormalize;
    float scale;
    // set by the launcher
    int group_lanes;   // lanes of a group, 0 if a group is no power of two of whole lanes
    int group_share;   // log2 of the lanes that search a group of any other size
    int bias_wide;     // bias lies on a 16-byte boundary
};

// logits [T][ld] of NVFP4_TYPE_*; ids, weights [T][k]
cudaError_t launch_route_topk(const void* logits, int type, int64_t T, int E, int64_t ld, const RouteParams& p,
                              const float* bias, int32_t* ids, float* weights, int* err, cudaStream_t st);
// dl [T][ld_out], the logits' type
cudaError_t launch_route_topk_backward(const void* logits, int type, int64_t T, int E, int64_t ld,
                                       const RouteParams& p, const int32_t* ids, const float* dw, void* dl,
                                       int64_t ld_out, int* err, cudaStream_t st);

// Columns of one 512-byte scale tile: 4 scales of 16 (NVFP4) or 32 (MXFP4) elements.
constexpr int kMxBlock = 32;
constexpr int kMxTileCols = 128;
__host__ __device__ inline int64_t mx_sf_tiles(int64_t cols) { return (cols + kMxTileCols - 1) / kMxTileCols; }
// Byte of the E8M0 scale of (row r, 32-element block b).
__host__ __device__ inline size_t mx_sf_offset(int64_t r, int64_t b, int64_t cols) {
    return static_cast<size_t>(((r >> 7) * mx_sf_tiles(cols) + (b >> 2)) * kSfAtomBytes + (r & 31) * 16 +
                               ((r & 127) >> 5) * 4 + (b & 3));
}

// x [rows][ld] of NVFP4_TYPE_*
cudaError_t launch_mxfp4_quantize_rows(const void* x, int type, int64_t rows, int64_t cols, int64_t ld,
                                       uint8_t* codes, uint8_t* sf, int* err, cudaStream_t st);
cudaError_t launch_mxfp4_dequantize_rows(const uint8_t* codes, const uint8_t* sf, int64_t rows, int64_t cols,
                                         void* out, int type, int64_t ld, cudaStream_t st);

// out[t, n] = sum_k a[t, k] b[n, k] (+ bias[n]), a and b quantised rows of the same format
struct LinearArgs {
    bool mx;                  // MXFP4 (no outer scales) or NVFP4
    int64_t T;
    int N, K;
    const uint8_t* a_codes;   // [T][K/2]
    const uint8_t* a_sf;
    const float* a_g;         // [T] (NVFP4)
    const uint8_t* b_codes;   // [N][K/2]
    const uint8_t* b_sf;
    const float* b_g;         // [N] (NVFP4)
    const float* bias;        // [N] or nullptr
    void* out;                // [T][ldo] of NVFP4_TYPE_*
    int out_type;
    int64_t ldo;
    int* err;
};
// The same with x not quantised yet, [T][ld] of NVFP4_TYPE_* (a's operand pointers unused): for the
// few tokens linear_quantises_x takes, which one kernel serves.
struct LinearInput {
    const void* x;
    int type;
    int64_t ld;
};
bool linear_quantises_x(bool mx, int64_t T, int64_t K);
cudaError_t launch_linear_x(const LinearInput& x, const LinearArgs& a, cudaStream_t st);

// x [rows][ld] BF16 (cols % 64 == 0, at most 8192) to NVFP4 rows for a_codes, a_sf and a_g.
cudaError_t launch_nvfp4_quantize_x(const uint16_t* x, int64_t rows, int cols, int64_t ld, uint8_t* codes, uint8_t* sf,
                                    float* g, int* err, cudaStream_t st);

// pdl: launched as a programmatic dependent of the kernel that quantises a
cudaError_t launch_linear(const LinearArgs& a, cudaStream_t st, bool pdl);
// Its kernel for many tokens, and the pairs of CTAs that run at once.
cudaError_t launch_linear_pair(const LinearArgs& a, cudaStream_t st, bool pdl);
int linear_pair_count();

}  // namespace nvfp4
