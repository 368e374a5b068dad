// Low-rank adapters: what the launchers share.
#pragma once

#include <mutex>
#include <type_traits>

#include "lora.cuh"

namespace nvfp4 {
namespace lora {

constexpr int kMaxAdapters = 1024;        // the sort holds a count for each adapter and warp in shared memory
constexpr int kMaxRank = 128;
constexpr int kMaxDevices = 64;
constexpr int kInCta = kThreads;          // up to so many tokens a CTA finds its tile by itself

inline size_t align_256(size_t n) { return (n + 255) / 256 * 256; }
// Tiles at most: every adapter's last one may be short (the rows without one count as an adapter).
inline int64_t tiles_bound(int64_t T, int L, int rows_per_tile) {
    const int64_t n = T / rows_per_tile + L + 1;
    return n < T ? n : T;
}

// Terms that h is taken as by the second product.
template <typename T>
__host__ __device__ constexpr int terms_of(int y_type) {
    return std::is_same<T, __nv_bfloat16>::value && y_type == NVFP4_TYPE_F32 ? 3 : 2;
}

template <typename F>
cudaError_t by_rank(int R, F&& f) {
    if (R <= 16) return f(std::integral_constant<int, 16>());
    if (R <= 32) return f(std::integral_constant<int, 32>());
    if (R <= 64) return f(std::integral_constant<int, 64>());
    return f(std::integral_constant<int, 128>());
}

// Lets a kernel ask for up to `bytes` of dynamic shared memory, once per device (`ready` is the kernel's own).
struct Ready {
    std::mutex mutex;
    bool on[kMaxDevices] = {};
    int clusters[kMaxDevices][3][kMaxRank / 8 + 1] = {};   // that run at once, by size (2, 4, 8) and rank (0: not asked yet)
};
inline cudaError_t allow_shared(const void* kernel, int bytes, Ready& ready) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(ready.mutex);
    if (!ready.on[dev]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        ready.on[dev] = true;
    }
    return cudaSuccess;
}

// Clusters of `split` CTAs of a kernel that run at once on the current device.
template <typename... A>
cudaError_t clusters_at_once(void (*kernel)(A...), int threads, int smem, int R, int split, Ready& ready, int64_t& clusters) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(ready.mutex);
    int& known = ready.clusters[dev][split / 4][R / 8];
    if (known == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(split);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = split;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorInvalidConfiguration;
        known = n;
    }
    clusters = known;
    return cudaSuccess;
}

constexpr int kManyShared = 225 * 1024;   // 227 KB to a CTA, less the static variables
constexpr int kMaxStages = 6;
// Shared memory of the kernel for many rows: a ring of stages (128 bytes of 128 rows of x, or of y, and the adapter's part
// that goes with them), and beside it the CTA's sums and the terms of h.
struct ManyLayout {
    int blocks;                           // of 64 ranks, or of fewer in shorter rows
    int down_bytes, up_bytes;             // the adapter's part
    int stage, stages;                    // bytes of a stage; how many
    int sum_pitch, sum, h, total;         // floats of a row of the sums; offsets; all bytes
    int cols;                             // outputs of a stage
    bool fits, two;                       // two CTAs to an SM
    __host__ __device__ ManyLayout(int R, int terms, bool trans, int y_type) {
        cols = y_type == NVFP4_TYPE_F32 ? 32 : 64;
        blocks = (R + 63) / 64;
        down_bytes = trans ? 64 * rank_bytes(R) * blocks : rank_up(R) * 128;
        up_bytes = trans ? rank_up(R) * 128 : cols * rank_bytes(R) * blocks;
        stage = (kManyRows * 128 + (down_bytes > up_bytes ? down_bytes : up_bytes) + 1023) / 1024 * 1024;
        sum_pitch = R + 4;
        const int rest = kManyRows * sum_pitch * 4 + terms * kManyRows * padded_pitch(rank_up(R)) + 1024;
        // two CTAs to an SM where that leaves three stages, otherwise one with what there is
        constexpr int kHalf = 112 * 1024, kWhole = kManyShared;
        stages = (kHalf - rest) / stage;
        two = R <= 32 && stages >= 3;
        if (!two) stages = (kWhole - rest) / stage;
        if (stages > kMaxStages) stages = kMaxStages;
        fits = rest < kWhole && stages >= 2;
        sum = stages * stage;
        h = sum + kManyRows * sum_pitch * 4;
        total = sum + rest;
    }
};
inline bool many_fits(int R, int terms, bool trans) {
    return ManyLayout(R, terms, trans, NVFP4_TYPE_BF16).fits && ManyLayout(R, terms, trans, NVFP4_TYPE_F32).fits;
}

// Map of [slices][rows][cols] 16-bit units, rows `ld` units apart and slices `slice` (multiples of 8): boxes of box_rows rows
// in shared-memory rows of `bytes` (32, 64 or 128), swizzled as wide; what lies outside reads as zero.
bool make_units_map(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t ld, int64_t slices, int64_t slice, int box_rows,
                    int bytes = 128);

size_t sort_bytes(int64_t T, int L);
Tiles sort_layout(void* ws, int64_t T, int L);
cudaError_t launch_sort(const int32_t* ids, int64_t T, int L, int rows_per_tile, const Tiles& t, int* err, cudaStream_t st);

// Copies rows that start on no 16-byte boundary to out [rows][ld_out] that do, ld_out a multiple of 8 (zeros behind cols); a
// programmatic dependent of the sort, which it has no use for but to end behind it.
cudaError_t launch_align_rows(const uint16_t* rows, int64_t T, int cols, int64_t ld, uint16_t* out, int64_t ld_out, cudaStream_t st);

// The kernels, each compiled in a file of its own; tiles: clusters to launch.
cudaError_t launch_few_forward_bf16(const Params& p, int64_t tiles, bool pdl, cudaStream_t st);
cudaError_t launch_few_forward_f16(const Params& p, int64_t tiles, bool pdl, cudaStream_t st);
cudaError_t launch_few_backward(const Params& p, int64_t tiles, bool pdl, cudaStream_t st);
template <typename T, bool kTrans, int kType>
cudaError_t launch_many(const Params& p, int64_t tiles, bool pdl, cudaStream_t st);
template <typename T, bool kTrans>
cudaError_t launch_many_any(const Params& p, int64_t tiles, bool pdl, cudaStream_t st) {
    return p.y_type == NVFP4_TYPE_BF16  ? launch_many<T, kTrans, NVFP4_TYPE_BF16>(p, tiles, pdl, st)
           : p.y_type == NVFP4_TYPE_F16 ? launch_many<T, kTrans, NVFP4_TYPE_F16>(p, tiles, pdl, st)
                                        : launch_many<T, kTrans, NVFP4_TYPE_F32>(p, tiles, pdl, st);
}

// Gradients of the adapters.
struct GradParams {
    const uint16_t* x;          // [T][ldx], K columns; rows on 16-byte boundaries
    const uint16_t* dy;         // [T][lddy], N columns; the same
    int64_t ldx, lddy;
    const float* h;             // [T][R]
    const float* dh;            // [T][R], with the scale
    const float* scale;
    Tiles tiles;
    int L, R, K, N;
    float* ddown;               // [L][R][K]
    float* dup;                 // [L][N][R]
    int ddown_wide;             // pairs of its columns on 8-byte boundaries
    float* parts;               // grad_bytes(T, L, R, K, N) bytes
    int* err;
};
size_t grad_bytes(int64_t T, int L, int R, int64_t K, int64_t N);
cudaError_t launch_grad(const GradParams& p, int64_t T, cudaStream_t st);

}  // namespace lora
}  // namespace nvfp4
