// Low-rank adapters: the sort of the tokens by adapter, and the kernel for tiles of 16 rows (lora.cuh says what is computed).
#include <algorithm>

#include "lora_launch.cuh"

namespace nvfp4 {
namespace lora {
namespace {

constexpr int kSortThreads = 1024, kSortWarps = 32;

// Rows put in order by adapter (each adapter's in their own order), then cut into tiles of `rows_per_tile`.  One cluster of
// 8 CTAs: a warp takes a stretch of the rows, counts its adapters, and after the sums over warps, CTAs and adapters puts
// its rows in place, 32 at a time (match_any gives a row its place among them).  The counts need no global memory, so
// nothing has to be cleared in front.  2000 to 16384 rows in 5.1 to 5.9 us: the start, two cluster barriers and four trips to
// memory; one CTA, bound by the instructions of each warp, took 9 us for 8192 rows and 10.4 for 16384.
constexpr int kAhead = 4;                 // loads of ids at a time

__global__ void __cluster_dims__(kGroups, 1, 1) __launch_bounds__(kSortThreads, 1)
    sort_kernel(const int32_t* __restrict__ ids, int T, int L, int rows_per_tile, int32_t* __restrict__ perm,
                int32_t* __restrict__ offsets, int32_t* __restrict__ tile_adapter, int32_t* __restrict__ tile_start,
                int32_t* __restrict__ tile_count, int32_t* __restrict__ prefix,
                int32_t* __restrict__ pieces, int* err) {
    pdl_launch_dependents();                                // what reads this kernel's results waits for its end
    extern __shared__ int s_at[];                           // [kSortWarps][bins] rows of a warp, then those in front of it
    __shared__ int s_scan[3][kSortWarps];
    const int bins = L + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_rank());
    int* mine = s_at + warp * bins;
    int *s_own = s_at + kSortWarps * bins, *s_first = s_own + bins;   // [bins] the CTA's rows; its first place
    for (int i = threadIdx.x; i < kSortWarps * bins; i += kSortThreads) s_at[i] = 0;
    __syncthreads();
    constexpr unsigned kAllWarps = kSortWarps * kGroups;
    const unsigned rows = T, stretch = ((rows + kAllWarps - 1) / kAllWarps + 31) / 32 * 32;   // T < 2^31 - 256: no overflow below
    const unsigned begin = (rank * kSortWarps + warp) * stretch, end = min(begin + stretch, rows);
    int id[kAhead];
    const auto fetch = [&](unsigned base) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const unsigned t = base + 32 * j + lane;
            id[j] = t < end ? ids[t] : -1;
        }
    };
    bool bad = false;
#pragma unroll 1
    for (unsigned base = begin; base < end; base += 32 * kAhead) {
        fetch(base);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (base + 32 * j + lane >= end) continue;
            bad |= id[j] >= L;
            atomicAdd(mine + (id[j] < 0 || id[j] >= L ? L : id[j]), 1);
        }
    }
    if (bad) set_device_error(err, NVFP4_ERR_BAD_EXPERT_ID);
    __syncthreads();
    for (int a = warp; a < bins; a += kSortWarps) {         // an adapter's rows over the warps
        const int c = s_at[lane * bins + a];
        int v = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(kAll, v, o);
            if (lane >= o) v += u;
        }
        s_at[lane * bins + a] = v - c;
        if (lane == 31) s_own[a] = v;
    }
    cluster_barrier();
    // the adapters one behind the other, 1024 at a time (L is at most that, and one for the rows without); every CTA
    // does all of it, each writes the tiles of every eighth adapter
    int first_row = 0, first_tile = 0, first_stage = 0;
    for (int base = 0; base < bins; base += kSortThreads) {
        const int a = base + static_cast<int>(threadIdx.x);
        int own = 0, front = 0;
        if (a < bins) {
#pragma unroll
            for (int c = 0; c < kGroups; ++c) {
                const int v = cluster_load_s32(cluster_addr(s_own + a, c));
                own += v;
                if (c < rank) front += v;
            }
        }
        const int tiles = (own + rows_per_tile - 1) / rows_per_tile;
        const int stages = a >= L ? 0 : max((own + kStageRows - 1) / kStageRows, 1);
        int r = own, n = tiles, g = stages;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int ur = __shfl_up_sync(kAll, r, o), un = __shfl_up_sync(kAll, n, o), ug = __shfl_up_sync(kAll, g, o);
            if (lane >= o) r += ur, n += un, g += ug;
        }
        if (lane == 31) s_scan[0][warp] = r, s_scan[1][warp] = n, s_scan[2][warp] = g;
        __syncthreads();
        int wr = s_scan[0][lane], wn = s_scan[1][lane], wg = s_scan[2][lane];   // every warp: the warps in front
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int ur = __shfl_up_sync(kAll, wr, o), un = __shfl_up_sync(kAll, wn, o), ug = __shfl_up_sync(kAll, wg, o);
            if (lane >= o) wr += ur, wn += un, wg += ug;
        }
        const int row = first_row + r - own + (warp ? __shfl_sync(kAll, wr, (warp - 1) & 31) : 0);
        const int tile = first_tile + n - tiles + (warp ? __shfl_sync(kAll, wn, (warp - 1) & 31) : 0);
        const int stage = first_stage + g - stages + (warp ? __shfl_sync(kAll, wg, (warp - 1) & 31) : 0);
        first_stage += __shfl_sync(kAll, wg, 31);
        first_row += __shfl_sync(kAll, wr, 31);
        first_tile += __shfl_sync(kAll, wn, 31);
        if (a < bins) {
            s_first[a] = row + front;
            if (a % kGroups == rank) {
                offsets[a] = row;
                prefix[a] = stage;                          // at L: all
                for (int i = 0; i < tiles; ++i) {
                    tile_adapter[tile + i] = a < L ? a : -1;
                    tile_start[tile + i] = row + i * rows_per_tile;
                }
            }
        }
        __syncthreads();
    }
    if (rank == 0 && threadIdx.x < kMaxCtas) pieces[threadIdx.x] = 0;
    if (threadIdx.x == 0 && rank == 0) {
        offsets[bins] = T;
        *tile_count = first_tile;
    }
#pragma unroll 1
    for (unsigned base = begin; base < end; base += 32 * kAhead) {
        if (end - begin > 32 * kAhead) fetch(base);         // otherwise they are still here
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const unsigned t = base + 32 * j + lane;
            if (base + 32 * j >= end) continue;
            const int a = t >= end ? -1 : id[j] < 0 || id[j] >= L ? L : id[j];
            const unsigned same = __match_any_sync(kAll, a);
            if (a >= 0) perm[s_first[a] + mine[a] + __popc(same & ((1u << lane) - 1))] = t;
            __syncwarp();
            if (a >= 0 && (same >> lane) == 1) mine[a] += __popc(same);   // the last of them
            __syncwarp();
        }
    }
    cluster_barrier();                                      // no CTA leaves while another reads its counts
}

// A thread to 8 elements.  8191 x 1999 take 14 us, 65 MB at 4.6 TB/s, most of it beside the sort; with dy as it came the gradients
// took 125 us instead of 79 and dx 88 instead of 77.
__global__ void __launch_bounds__(256) align_rows_kernel(const uint16_t* __restrict__ rows, int64_t T, int cols, int64_t ld,
                                                         uint16_t* __restrict__ out, int64_t ld_out) {
    const unsigned chunks = static_cast<unsigned>(ld_out / 8);
    const int64_t all = T * chunks, step = static_cast<int64_t>(gridDim.x) * 256;
    constexpr int kMine = 4;
    for (int64_t base = blockIdx.x * 256 + threadIdx.x; base < all; base += kMine * step) {
        Straddle w[kMine];
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int64_t at = base + i * step, t = at / chunks;
            if (at < all) w[i].load(rows + t * ld, 8 * static_cast<int>(at - t * chunks), cols);
        }
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int64_t at = base + i * step;
            if (at < all) *reinterpret_cast<uint4*>(out + 8 * at) = w[i].value();
        }
    }
    pdl_wait();
}

}  // namespace

cudaError_t launch_align_rows(const uint16_t* rows, int64_t T, int cols, int64_t ld, uint16_t* out, int64_t ld_out, cudaStream_t st) {
    const int64_t blocks = (T * (ld_out / 8) + 1023) / 1024, most = 8 * device_sm_count();
    return launch_pdl(true, align_rows_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(256), 0, st, rows, T, cols, ld,
                      out, ld_out);
}

namespace {
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}
}  // namespace

bool make_units_map(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t ld, int64_t slices, int64_t slice, int box_rows,
                    int bytes) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(slices)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(slice) * 2};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(bytes / 2), static_cast<cuuint32_t>(box_rows), 1}, estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, slices ? 3 : 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t sort_bytes(int64_t T, int L) {
    const size_t tiles = static_cast<size_t>(tiles_bound(T, L, kFewRows));
    return align_256(static_cast<size_t>(T) * 4) + 2 * align_256((L + 2) * 4) + 2 * align_256(tiles * 4) + 256 + align_256(kMaxCtas * 4);
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
    p += 256;
    t.prefix = reinterpret_cast<int32_t*>(p);
    p += align_256((L + 2) * 4);
    t.pieces = reinterpret_cast<int32_t*>(p);
    return t;
}

cudaError_t launch_sort(const int32_t* ids, int64_t T, int L, int rows_per_tile, const Tiles& t, int* err, cudaStream_t st) {
    const size_t smem = static_cast<size_t>(kSortWarps + 2) * (L + 1) * sizeof(int);
    static Ready ready;
    const cudaError_t e = allow_shared(reinterpret_cast<const void*>(sort_kernel),
                                       (kSortWarps + 2) * (kMaxAdapters + 1) * static_cast<int>(sizeof(int)), ready);
    if (e != cudaSuccess) return e;
    return launch_pdl(false, sort_kernel, dim3(kGroups), dim3(kSortThreads), smem, st, ids, static_cast<int>(T), L, rows_per_tile,
                      const_cast<int32_t*>(t.perm), const_cast<int32_t*>(t.offsets), const_cast<int32_t*>(t.adapter),
                      const_cast<int32_t*>(t.start), const_cast<int32_t*>(t.count),
                      const_cast<int32_t*>(t.prefix), t.pieces, err);
}

}  // namespace lora

namespace {

bool wide(const void* p, int64_t ld, int type) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld * (type == NVFP4_TYPE_F32 ? 4 : 2) % 16 == 0;
}

// Whether tiles of 16 rows take less time than tiles of 128: 6 us and a time for each of the one, a longer start and a time for
// each of the other, both with the columns.  The host does not know the ids: each adapter is taken to have tokens, its last tile half full on
// average, so a batch of 12 requests is slower beside a large pool (8192 x 2048 -> 2048 of rank 16 37 us with 12 adapters or 128, 80
// with 512, 88 with 1024; of rank 64 53, 55, 57 and 61).  BF16 adapters of rank 120 and 128 with FP32 outputs have no room for two
// stages of 128 rows (8192 x 2048 -> 2048 127 us of rank 112, 377 of rank 120).  us of
// 2048 -> 2048, tiles of 16 and of 128, with 1 adapter, 32, 64 and 256 (* what the rule takes):
//                    1             32            64            256
//   rank 16   512   10 * 15      10 * 15      16 * 25      40 * 62
//            1024   18 * 16      18 * 16      19 * 25      40 * 62
//            2048   25 19 *      25 18 *      24 27 *      41 * 63
//            8192   78 30 *      75 31 *      75 32 *      78 68 *
//   rank 32   512   11 * 20      14 * 20      20 * 36      62 * 92
//            1024   21 * 21      21 * 22      21 * 36      63 * 93
//            2048   35 26 *      35 24 *      36 39 *      64 * 94
//   rank 64   512   28 20 *      28 24 *      43 * 44     138 140 *
//            2048   76 28 *      75 25 *      76 45 *     140 140 *
//   rank 128  512   38 37 *      39 * 48      61 * 92     202 * 311
//            1024   62 35 *      62 52 *      63 * 91     203 * 316
//            2048  108 57 *     108 55 *     108 97 *     204 * 321
bool few_rows(int64_t T, int L, int R, int64_t K, int64_t N, int terms, bool trans) {
    using namespace lora;
    if (!many_fits(R, terms, trans)) return true;
    const int i = R <= 16 ? 0 : R <= 32 ? 1 : R <= 64 ? 2 : 3;
    constexpr double kTile16[] = {0.137, 0.216, 0.525, 0.766}, kStart[] = {13.5, 17.5, 14, 22}, kTile128[] = {0.195, 0.292, 0.485, 1.12};
    const double columns = static_cast<double>(K + N) / 4096, used = static_cast<double>(L < T ? L : T);
    const double tiles16 = std::max(used, T / 16.0 + used / 2), tiles128 = std::max(used, T / 128.0 + used / 2);
    return 6 + kTile16[i] * columns * tiles16 <= 10 + ((kStart[i] - 10) + kTile128[i] * tiles128) * columns;
}

}  // namespace

bool lora_sorts(int64_t T) { return T > lora::kInCta; }
size_t lora_workspace(int64_t T, int L) { return lora_sorts(T) ? lora::sort_bytes(T, L) : 0; }
namespace {
// The sort, dh, the parts of the adapters' gradients, and room for dy in aligned rows.
struct BackwardLayout {
    size_t dh, parts, dy, total;
    int64_t lddy;
    BackwardLayout(int64_t T, int L, int R, int64_t K, int64_t N) {
        using namespace lora;
        dh = align_256(sort_bytes(T, L));
        parts = dh + align_256(static_cast<size_t>(T) * R * sizeof(float));
        dy = parts + align_256(grad_bytes(T, L, R, K, N));
        lddy = (N + 7) / 8 * 8;
        total = dy + align_256(static_cast<size_t>(T) * lddy * 2);
    }
};
}  // namespace

size_t lora_backward_workspace(int64_t T, int L, int R, int64_t K, int64_t N) { return BackwardLayout(T, L, R, K, N).total; }

cudaError_t launch_lora_add(const LoraArgs& a, cudaStream_t st) {
    using namespace lora;
    Params p = {};
    p.x = a.x;
    p.ldx = a.ldx;
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
    p.y_wide = wide(a.y, a.ldy, a.y_type);
    p.out_wide = wide(a.out, a.ldo, a.y_type);
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
    const int rows = few_rows(a.T, a.L, a.R, a.K, a.N, bf16 && a.y_type == NVFP4_TYPE_F32 ? 3 : 2, false) ? kFewRows : kManyRows;
    p.tiles = sort_layout(a.ws, a.T, a.L);
    const cudaError_t e = launch_sort(a.ids, a.T, a.L, rows, p.tiles, a.err, st);
    if (e != cudaSuccess) return e;
    const int64_t tiles = tiles_bound(a.T, a.L, rows);
    if (rows == kFewRows) return bf16 ? launch_few_forward_bf16(p, tiles, true, st) : launch_few_forward_f16(p, tiles, true, st);
    return bf16 ? launch_many_any<__nv_bfloat16, false>(p, tiles, true, st) : launch_many_any<__half, false>(p, tiles, true, st);
}

cudaError_t launch_lora_add_backward(const LoraBackwardArgs& a, cudaStream_t st) {
    using namespace lora;
    const Tiles tiles = sort_layout(a.ws, a.T, a.L);
    const BackwardLayout lay(a.T, a.L, a.R, a.K, a.N);
    float* dh = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + lay.dh);
    const int rows = few_rows(a.T, a.L, a.R, a.K, a.N, a.dx_type == NVFP4_TYPE_F32 ? 3 : 2, true) ? kFewRows : kManyRows;
    cudaError_t e = launch_sort(a.ids, a.T, a.L, rows, tiles, a.err, st);
    if (e != cudaSuccess) return e;
    Params p = {};
    p.x = a.dy;
    p.ldx = a.lddy;
    if (!wide(a.dy, a.lddy, NVFP4_TYPE_BF16)) {
        uint16_t* dy = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(a.ws) + lay.dy);
        e = launch_align_rows(static_cast<const uint16_t*>(a.dy), a.T, static_cast<int>(a.N), a.lddy, dy, lay.lddy, st);
        if (e != cudaSuccess) return e;
        p.x = dy;
        p.ldx = lay.lddy;
    }
    p.down = a.up;                        // dh = s dy B: B is [N][R]
    p.up = a.down;                        // dx = dh A: A is [R][K]
    p.scale = a.scale;
    p.ids = a.ids;
    p.y = a.accumulate ? a.dx : nullptr;
    p.out = a.dx;
    p.h = dh;
    p.ldy = p.ldo = a.lddx;
    p.y_type = a.dx_type;
    p.y_wide = p.out_wide = wide(a.dx, a.lddx, a.dx_type);
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
    e = rows == kFewRows ? launch_few_backward(p, bound, true, st) : launch_many_any<__nv_bfloat16, true>(p, bound, true, st);
    if (e != cudaSuccess) return e;
    GradParams g = {};
    g.x = static_cast<const uint16_t*>(a.x);
    g.dy = static_cast<const uint16_t*>(p.x);
    g.ldx = a.ldx;
    g.lddy = p.ldx;
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
    g.ddown_wide = a.K % 2 == 0 && (reinterpret_cast<uintptr_t>(a.ddown) & 7) == 0;
    g.err = a.err;
    g.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + lay.parts);
    return launch_grad(g, a.T, st);
}

}  // namespace nvfp4
