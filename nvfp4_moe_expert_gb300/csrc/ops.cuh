// Host launchers of the routing operators, of the dense 4-bit products and of what stands beside them (each defined in the
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

// Rows of a balance loss: logits [T][ld] of NVFP4_TYPE_*, ids [T][k], mask [T] or nullptr, offsets [S + 1] or nullptr (one
// sequence of all rows)
struct BalanceArgs {
    int64_t T;
    int E;
    int64_t ld;
    int score, k;
    const int32_t* ids;
    const uint8_t* mask;
    const int32_t* offsets;
    int64_t S;
};
// loss, tokens [S]; counts, probs [S][E]; ws: balance_workspace(T, E, S) bytes
size_t balance_workspace(int64_t T, int E, int64_t S);
cudaError_t launch_balance_loss(const void* logits, int type, const BalanceArgs& a, float* loss, int32_t* counts,
                                float* probs, int32_t* tokens, void* ws, int* err, cudaStream_t st);
// dl [T][ld_out], the logits' type; a.ids unused
cudaError_t launch_balance_loss_backward(const void* logits, int type, const BalanceArgs& a, const int32_t* counts,
                                         const int32_t* tokens, const float* dloss, void* dl, int64_t ld_out,
                                         bool accumulate, int* err, cudaStream_t st);

// Low-rank adapters: out [T][ldo] = y [T][ldy] + scale_a (x_t A_a^T) B_a^T, a = ids[t] (negative: none); down A [L][R][K],
// up B [L][N][R], x [T][ldx] of `type` (BF16 or FP16); y, out of y_type; h [T][R] = x_t A_a^T or nullptr
struct LoraArgs {
    const void* x;
    int64_t T, ldx;
    int type;
    const void* down;
    const void* up;
    const float* scale;
    const int32_t* ids;
    int L, R;
    int64_t K, N;
    const void* y;
    int64_t ldy;
    void* out;
    int64_t ldo;
    int y_type;
    float* h;
    void* ws;                 // lora_workspace(T, L) bytes
    int* err;
};
size_t lora_workspace(int64_t T, int L);
cudaError_t launch_lora_add(const LoraArgs& a, cudaStream_t st);
// dx (+)= scale_a (dy_t B_a) A_a, ddown [L][R][K], dup [L][N][R]; BF16 x, dy and adapters
struct LoraBackwardArgs {
    const void* dy;
    const void* x;
    int64_t T, lddy, ldx;
    const float* h;
    const void* down;
    const void* up;
    const float* scale;
    const int32_t* ids;
    int L, R;
    int64_t K, N;
    void* dx;
    int64_t lddx;
    int dx_type;
    bool accumulate;
    float* ddown;
    float* dup;
    void* ws;                 // lora_backward_workspace(T, L, R, K, N) bytes
    int* err;
};
size_t lora_backward_workspace(int64_t T, int L, int R, int64_t K, int64_t N);
cudaError_t launch_lora_add_backward(const LoraBackwardArgs& a, cudaStream_t st);

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
