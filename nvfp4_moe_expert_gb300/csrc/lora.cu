// Low-rank adapters: the sort of the tokens by adapter, and the kernel for tiles of 16 rows (lora.cuh says what is computed).
#include "lora_launch.cuh"

namespace nvfp4 {
namespace lora {
namespace {

constexpr int kSortThreads = 1024, kSortWarps = 32;

// Rows put in order by adapter (each adapter's in their own order), then cut into tiles of `rows_per_tile`.  One block: a
// warp takes a stretch of the rows, counts its adapters, and after the sums over adapters and warps puts its rows in place,
// 32 at a time (match_any gives a row its place among them).  ids are read twice.
__global__ void __launch_bounds__(kSortThreads)
    sort_kernel(const int32_t* __restrict__ ids, int T, int L, int rows_per_tile, int32_t* __restrict__ perm,
                int32_t* __restrict__ offsets, int32_t* __restrict__ tile_adapter, int32_t* __restrict__ tile_start,
                int32_t* __restrict__ tile_count, int* err) {
    extern __shared__ int s_at[];                           // [kSortWarps][L + 1], first counts, then places
    __shared__ int s_scan[kSortWarps], s_rows, s_tiles;
    const int bins = L + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int* mine = s_at + warp * bins;
    for (int i = threadIdx.x; i < kSortWarps * bins; i += kSortThreads) s_at[i] = 0;
    if (threadIdx.x == 0) s_rows = s_tiles = 0;
    __syncthreads();
    const int stretch = ((T + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
    const int64_t begin = static_cast<int64_t>(warp) * stretch, end = min(begin + stretch, static_cast<int64_t>(T));
    bool bad = false;
    for (int64_t t = begin + lane; t < end; t += 32) {
        const int id = ids[t];
        bad |= id >= L;
        atomicAdd(mine + (id < 0 || id >= L ? L : id), 1);
    }
    if (bad) set_device_error(err, NVFP4_ERR_BAD_EXPERT_ID);
    __syncthreads();
    // an adapter's rows over the warps, then the adapters one behind the other, 1024 at a time
    for (int base = 0; base < bins; base += kSortThreads) {
        const int a = base + static_cast<int>(threadIdx.x);
        int rows = 0;
        if (a < bins) {
            for (int w = 0; w < kSortWarps; ++w) {
                const int c = s_at[w * bins + a];
                s_at[w * bins + a] = rows;
                rows += c;
            }
        }
        const int tiles = (rows + rows_per_tile - 1) / rows_per_tile;
        const int first_row = s_rows, first_tile = s_tiles;
        int sums[2] = {rows, tiles}, before[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {                       // sums over the adapters in front, in the block
            int v = sums[k];
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(kAll, v, o);
                if (lane >= o) v += u;
            }
            __syncthreads();
            if (lane == 31) s_scan[warp] = v;
            __syncthreads();
            int front = 0;
            for (int w = 0; w < warp; ++w) front += s_scan[w];
            before[k] = front + v - sums[k];
        }
        const int row = first_row + before[0], tile = first_tile + before[1];
        if (a < bins) {
            offsets[a] = row;
            for (int w = 0; w < kSortWarps; ++w) s_at[w * bins + a] += row;
            for (int i = 0; i < tiles; ++i) {
                tile_adapter[tile + i] = a < L ? a : -1;
                tile_start[tile + i] = row + i * rows_per_tile;
            }
        }
        __syncthreads();
        if (threadIdx.x == kSortThreads - 1) {
            s_rows = row + rows;
            s_tiles = tile + tiles;
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        offsets[bins] = T;
        *tile_count = s_tiles;
    }
    for (int64_t base = begin; base < end; base += 32) {
        const int64_t t = base + lane;
        const unsigned active = __ballot_sync(kAll, t < end);
        if (t < end) {
            const int id = ids[t], a = id < 0 || id >= L ? L : id;
            const unsigned same = __match_any_sync(active, a);
            const int place = mine[a] + __popc(same & ((1u << lane) - 1));
            perm[place] = static_cast<int32_t>(t);
            __syncwarp(active);
            if ((same >> lane) == 1) mine[a] += __popc(same);   // the last of them
        }
        __syncwarp();
    }
}

}  // namespace

size_t sort_bytes(int64_t T, int L) {
    const size_t tiles = static_cast<size_t>(tiles_bound(T, L, kFewRows));
    return align_256(static_cast<size_t>(T) * 4) + align_256((L + 2) * 4) + 2 * align_256(tiles * 4) + 256;
}

Tiles sort_layout(void* ws, int64_t T, int L) {
    const size_t tiles = static_cast<size_t>(tiles_bound(T, L, kFewRows));
    uint8_t* p = static_cast<uint8_t*>(ws);
    Tiles t;
    t.perm = reinterpret_cast<int32_t*>(p);
    p += align_256(static_cast<size_t>(T) * 4);
    t.offsets = reinterpret_cast<int32_t*>(p);
    p += align_256((L + 2) * 4);
    t.adapter = reinterpret_cast<int32_t*>(p);
    p += align_256(tiles * 4);
    t.start = reinterpret_cast<int32_t*>(p);
    p += align_256(tiles * 4);
    t.count = reinterpret_cast<int32_t*>(p);
    return t;
}

cudaError_t launch_sort(const int32_t* ids, int64_t T, int L, int rows_per_tile, const Tiles& t, int* err, cudaStream_t st) {
    const size_t smem = static_cast<size_t>(kSortWarps) * (L + 1) * sizeof(int);
    static Ready ready;
    const cudaError_t e = allow_shared(reinterpret_cast<const void*>(sort_kernel),
                                       kSortWarps * (kMaxAdapters + 1) * static_cast<int>(sizeof(int)), ready);
    if (e != cudaSuccess) return e;
    return launch_pdl(false, sort_kernel, dim3(1), dim3(kSortThreads), smem, st, ids, static_cast<int>(T), L, rows_per_tile,
                      const_cast<int32_t*>(t.perm), const_cast<int32_t*>(t.offsets), const_cast<int32_t*>(t.adapter),
                      const_cast<int32_t*>(t.start), const_cast<int32_t*>(t.count), err);
}

}  // namespace lora

namespace {

bool wide(const void* p, int64_t ld, int type) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld * (type == NVFP4_TYPE_F32 ? 4 : 2) % 16 == 0;
}

// Tiles of 16 rows while the tiles of 128 are too few to fill the GPU.
constexpr int64_t kFewTokens = 1024;

}  // namespace

bool lora_sorts(int64_t T) { return T > lora::kInCta; }
size_t lora_workspace(int64_t T, int L) { return lora_sorts(T) ? lora::sort_bytes(T, L) : 0; }
size_t lora_backward_workspace(int64_t T, int L, int R) {
    return lora::align_256(lora::sort_bytes(T, L)) + lora::align_256(static_cast<size_t>(T) * R * sizeof(float));
}

cudaError_t launch_lora_add(const LoraArgs& a, cudaStream_t st) {
    using namespace lora;
    Params p = {};
    p.x = a.x;
    p.ldx = a.ldx;
    p.x_wide = 1;
    p.down = a.down;
    p.up = a.up;
    p.scale = a.scale;
    p.ids = a.ids;
    p.y = a.y;
    p.out = a.out;
    p.h = a.h;
    p.ldy = a.ldy;
    p.ldo = a.ldo;
    p.y_type = a.y_type;
    p.out_wide = wide(a.y, a.ldy, a.y_type) && wide(a.out, a.ldo, a.y_type);
    p.skip_none = a.y == a.out && a.h == nullptr;
    p.T = static_cast<int>(a.T);
    p.L = a.L;
    p.R = a.R;
    p.C = static_cast<int>(a.K);
    p.D = static_cast<int>(a.N);
    p.err = a.err;
    const bool bf16 = a.type == NVFP4_TYPE_BF16;
    if (!lora_sorts(a.T)) {
        const int64_t tiles = tiles_bound(a.T, a.L, kFewRows);
        return bf16 ? launch_few_forward_bf16(p, tiles, false, st) : launch_few_forward_f16(p, tiles, false, st);
    }
    const int rows = a.T <= kFewTokens ? kFewRows : kManyRows;
    p.tiles = sort_layout(a.ws, a.T, a.L);
    const cudaError_t e = launch_sort(a.ids, a.T, a.L, rows, p.tiles, a.err, st);
    if (e != cudaSuccess) return e;
    const int64_t tiles = tiles_bound(a.T, a.L, rows);
    if (rows == kFewRows) return bf16 ? launch_few_forward_bf16(p, tiles, true, st) : launch_few_forward_f16(p, tiles, true, st);
    return bf16 ? launch_many_forward_bf16(p, tiles, true, st) : launch_many_forward_f16(p, tiles, true, st);
}

cudaError_t launch_lora_add_backward(const LoraBackwardArgs& a, cudaStream_t st) {
    using namespace lora;
    const Tiles tiles = sort_layout(a.ws, a.T, a.L);
    float* dh = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + align_256(sort_bytes(a.T, a.L)));
    const int rows = a.T <= kFewTokens ? kFewRows : kManyRows;
    cudaError_t e = launch_sort(a.ids, a.T, a.L, rows, tiles, a.err, st);
    if (e != cudaSuccess) return e;
    Params p = {};
    p.x = a.dy;
    p.ldx = a.lddy;
    p.x_wide = wide(a.dy, a.lddy, NVFP4_TYPE_BF16);
    p.down = a.up;                        // dh = s dy B: B is [N][R]
    p.up = a.down;                        // dx = dh A: A is [R][K]
    p.scale = a.scale;
    p.ids = a.ids;
    p.y = a.accumulate ? a.dx : nullptr;
    p.out = a.dx;
    p.h = dh;
    p.ldy = p.ldo = a.lddx;
    p.y_type = a.dx_type;
    p.out_wide = wide(a.dx, a.lddx, a.dx_type);
    p.h_scaled = 1;
    p.skip_none = a.accumulate;           // nobody reads the dh of rows without an adapter
    p.T = static_cast<int>(a.T);
    p.L = a.L;
    p.R = a.R;
    p.C = static_cast<int>(a.N);
    p.D = static_cast<int>(a.K);
    p.tiles = tiles;
    p.err = a.err;
    const int64_t bound = tiles_bound(a.T, a.L, rows);
    e = rows == kFewRows ? launch_few_backward(p, bound, true, st) : launch_many_backward(p, bound, true, st);
    if (e != cudaSuccess) return e;
    GradParams g = {};
    g.x = static_cast<const uint16_t*>(a.x);
    g.dy = static_cast<const uint16_t*>(a.dy);
    g.ldx = a.ldx;
    g.lddy = a.lddy;
    g.x_wide = 1;
    g.dy_wide = p.x_wide;
    g.h = a.h;
    g.dh = dh;
    g.scale = a.scale;
    g.tiles = tiles;
    g.L = a.L;
    g.R = a.R;
    g.K = static_cast<int>(a.K);
    g.N = static_cast<int>(a.N);
    g.ddown = a.ddown;
    g.dup = a.dup;
    return launch_grad(g, st);
}

}  // namespace nvfp4
