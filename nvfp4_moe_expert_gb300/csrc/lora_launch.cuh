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
int terms_of(int y_type) {
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

size_t sort_bytes(int64_t T, int L);
Tiles sort_layout(void* ws, int64_t T, int L);
cudaError_t launch_sort(const int32_t* ids, int64_t T, int L, int rows_per_tile, const Tiles& t, int* err, cudaStream_t st);

// The kernels, each compiled in a file of its own; tiles: clusters to launch.
cudaError_t launch_few_forward_bf16(const Params& p, int64_t tiles, bool pdl, cudaStream_t st);
cudaError_t launch_few_forward_f16(const Params& p, int64_t tiles, bool pdl, cudaStream_t st);
cudaError_t launch_few_backward(const Params& p, int64_t tiles, bool pdl, cudaStream_t st);
cudaError_t launch_many_forward_bf16(const Params& p, int64_t tiles, bool pdl, cudaStream_t st);
cudaError_t launch_many_forward_f16(const Params& p, int64_t tiles, bool pdl, cudaStream_t st);
cudaError_t launch_many_backward(const Params& p, int64_t tiles, bool pdl, cudaStream_t st);

// Gradients of the adapters.
struct GradParams {
    const uint16_t* x;          // [T][ldx], K columns
    const uint16_t* dy;         // [T][lddy], N columns
    int64_t ldx, lddy;
    int x_wide, dy_wide;
    const float* h;             // [T][R]
    const float* dh;            // [T][R], with the scale
    const float* scale;
    Tiles tiles;
    int L, R, K, N;
    float* ddown;               // [L][R][K]
    float* dup;                 // [L][N][R]
};
cudaError_t launch_grad(const GradParams& p, cudaStream_t st);

}  // namespace lora
}  // namespace nvfp4
