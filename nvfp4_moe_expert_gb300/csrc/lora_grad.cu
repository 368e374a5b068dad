// Gradients of low-rank adapters:  dA_a = sum_t dh_t x_t^T  [R][K],  dB_a = sum_t s_a dy_t h_t^T  [N][R],  over the tokens of
// adapter a in their order.
//
// Both are sums over tokens of a column of R values (dh, or s h) times a row of x, or dy.  The work is units (an adapter, up
// to 32 of its ranks, a slab of 256 columns of x or dy) of stages (32 tokens), one behind the other, cut into as many equal
// stretches as CTAs run at once: requests are uneven, and with CTAs of a cluster sharing a unit's tokens the longest adapter's
// took twice the mean, and 1.7 waves two (93 us for 16384 x (4096 + 4096), rank 16).  A unit that lies in one stretch is written by
// its CTA; of the others each CTA leaves its part in the workspace (at most two: where its stretch begins and where it
// ends), and the last to do so adds the unit's parts in order, whoever that is: the same bits every time.  (A second kernel
// for that took 8 to 11 us.)  More than 32 ranks read a slab again, out of L2.
//
// Two loader warps keep a ring of stages full, x or dy by TMA (16 rows to an instruction where they lie in a row, four of any
// place otherwise) and the terms of h, which they make of copies that were started two stages before; the 8 others multiply, 32
// columns each.  With loads and products in the same warps a stage was 336 instructions of each, 24 of them products.
// 16384 x (4096 + 4096) of rank 16 take 72 us (83 with cp.async in the warps that multiply; 84 with h one stage ahead), 268 MB at
// 3.7 TB/s of the 4.5 that a kernel which only reads such an array gets; 512 x (2048 + 1536) 11 us (15); 8191 x (4096 + 1999) of
// rank 64 75 us, 19 GFLOP with the three terms, 250 TFLOP/s of 600: there the products and their operands out of shared memory
// count, the loads no more.
//
// A stage of x or dy is only read by ldmatrix, and each register that was loaded goes into a product in front of the warp's arrival:
// it goes back to TMA without a proxy fence.
//
// dh and h are FP32; they are taken as sums of three BF16 terms (2^-24 of them is left), as x and dy are BF16 and the sums
// FP32.  The tensor cores cut an accumulator's low bits off at each step: one chain over 2048 tokens was 6e-6 of the
// result low, so every 8 stages (48 steps) the chain is added to FP32 sums beside it and starts anew.
#include <algorithm>

#include "lora_launch.cuh"

namespace nvfp4 {
namespace lora {
namespace {

constexpr int kCols = 256, kTokens = kStageRows, kTerms = 3, kRanks = 32;
constexpr int kLoaders = 2;               // warps that load, 16 tokens of a stage each
constexpr int kStages = 4, kChain = 8;    // stages of the ring; of a chain of products
constexpr int kPart = kRanks * kCols;     // floats of a part
constexpr int kAhead = 2, kHeld = kAhead + 1, kLists = 8;   // stages that a loader's copies are ahead; buffers for h, and for rows

template <int kM>
struct GradLayout {
    static constexpr int pitch = padded_pitch(16 * kM);
    static constexpr int tile = kTokens * 128;                       // 64 columns
    static constexpr int x = tile * (kCols / 64), h = kTerms * kTokens * pitch;   // bytes of a stage
    static constexpr int raw = 16 * 16 * kM * 4;                     // h as it is, of a loader's tokens
    static constexpr int total = kStages * (x + h) + kLoaders * kHeld * raw + 1024;
    static constexpr int bytes(int L) { return total + (2 * L + 3) * 4; }   // with prefix and offsets
    static_assert(x % 1024 == 0 && h % 16 == 0, "swizzled tiles; 16-byte chunks");
};

struct GradMaps {
    CUtensorMap x, dy, x16, dy16;         // boxes of one row, for gathers, and of 16
};

// The next BF16 terms of two values, which keep what is left of them (0 where a term is infinite).
__device__ __forceinline__ uint32_t next_terms(float& a, float& b) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    const uint32_t w = *reinterpret_cast<const uint32_t*>(&t);
    a -= __uint_as_float(w << 16);
    b -= __uint_as_float(w & 0xFFFF0000u);
    if (!(a == a)) a = 0.0f;
    if (!(b == b)) b = 0.0f;
    return w;
}

// The units' shape: slabs of K in front of those of N, `rank_parts` units to a slab.
struct Shape {
    int slabs_k, rank_parts, units;       // units of an adapter
};
// A unit, and what a stretch holds of it.
struct Segment {
    int adapter, unit;
    int64_t begin, end;                   // the unit's stages in the whole
};
// The unit that stage `at` of the whole belongs to (at < all).  prefix[a]: stages of a unit of the adapters in front of a.
__device__ __forceinline__ Segment find_unit(const int32_t* prefix, int L, int units, int64_t at) {
    int lo = 0, hi = L;                   // prefix[lo] units <= at < prefix[hi] units
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (static_cast<int64_t>(prefix[mid]) * units <= at) lo = mid;
        else hi = mid;
    }
    const int64_t first = static_cast<int64_t>(prefix[lo]) * units;
    const int stages = prefix[lo + 1] - prefix[lo], unit = static_cast<int>((at - first) / stages);
    return {lo, unit, first + static_cast<int64_t>(unit) * stages, first + static_cast<int64_t>(unit + 1) * stages};
}
// The whole's stages over the CTAs: the first `more` take one more than `each`.
struct Stretches {
    int64_t each, more;
    __device__ __forceinline__ Stretches(int64_t all, int ctas) : each(all / ctas), more(all - each * ctas) {}
    __device__ __forceinline__ int64_t begin(int cta) const { return each * cta + min(static_cast<int64_t>(cta), more); }
    __device__ __forceinline__ int owner(int64_t stage) const {
        const int64_t large = more * (each + 1);
        return static_cast<int>(stage < large ? stage / (each + 1) : more + (stage - large) / each);
    }
};

// What is known of a unit's slab.
struct Slab {
    bool is_down;
    int rank0, ranks, col0, width;
    __device__ __forceinline__ Slab(const GradParams& p, const Shape& sh, int unit) {
        const int slab = unit / sh.rank_parts;
        rank0 = unit % sh.rank_parts * kRanks;
        ranks = min(kRanks, p.R - rank0);
        is_down = slab < sh.slabs_k;
        col0 = (is_down ? slab : slab - sh.slabs_k) * kCols;
        width = is_down ? p.K : p.N;
    }
    // two sums of rank r (of those of the unit), columns c and c + 1
    __device__ __forceinline__ void store(const GradParams& p, int adapter, int r, int c, float lo, float hi) const {
        const int left = width - col0 - c;
        if (r >= ranks || left <= 0) return;
        if (is_down) {
            float* at = p.ddown + (static_cast<int64_t>(adapter) * p.R + rank0 + r) * p.K + col0 + c;
            if (p.ddown_wide) {
                *reinterpret_cast<float2*>(at) = make_float2(lo, hi);
                return;
            }
            at[0] = lo;
            if (left > 1) at[1] = hi;
        } else {
            float* at = p.dup + (static_cast<int64_t>(adapter) * p.N + col0 + c) * p.R + rank0 + r;
            at[0] = lo;
            if (left > 1) at[p.R] = hi;
        }
    }
};

// The stages of a stretch, one by one, over its units.
struct Walk {
    const GradParams& p;
    const Shape& sh;
    const int *prefix, *offsets;
    int64_t at, end;
    Segment seg;
    Slab slab;
    __device__ __forceinline__ Walk(const GradParams& p_, const Shape& sh_, const int* prefix_, const int* offsets_, int64_t begin, int64_t end_)
        : p(p_), sh(sh_), prefix(prefix_), offsets(offsets_), at(begin), end(end_), seg(), slab(p_, sh_, 0) {
        if (at < end) enter();
    }
    __device__ __forceinline__ void enter() {
        seg = find_unit(prefix, p.L, sh.units, at);
        slab = Slab(p, sh, seg.unit);
    }
    __device__ __forceinline__ int row0() const { return offsets[seg.adapter] + static_cast<int>(at - seg.begin) * kTokens; }
    __device__ __forceinline__ int last() const { return offsets[seg.adapter + 1]; }
    __device__ __forceinline__ void next() {
        if (++at < end && at == seg.end) enter();
    }
};

// What a loader warp knows of a stage, 32 words in shared memory: the rows of its 16 tokens (behind the adapter's last token
// that one's row again), the scale, how many of the 16 are there, the first column and rank, whether it is of dA.
enum { kScaleAt = 16, kRowsAt, kColAt, kRankAt, kDownAt };

template <int kM>
__global__ void __launch_bounds__(kThreads + 32 * kLoaders, 2)
    grad_kernel(const __grid_constant__ GradMaps maps, const GradParams p, const Shape sh) {
    using Lay = GradLayout<kM>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ __align__(16) int s_list[kLoaders][kLists][32];
    __shared__ int s_last, abort_word;
    volatile int* abort_flag = &abort_word;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* smem_h = smem + kStages * Lay::x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 2 * kLoaders);
            mbar_init(&empty[s], kWarps);
        }
        abort_word = 0;
        fence_barrier_init();
    }
    if (threadIdx.x == kThreads) {
        prefetch_tensormap(&maps.x16);
        prefetch_tensormap(&maps.dy16);
    }
    pdl_wait();
    int *s_prefix = reinterpret_cast<int*>(smem_raw + Lay::total), *s_offsets = s_prefix + p.L + 1;
    for (int a = threadIdx.x; a < 2 * p.L + 3; a += blockDim.x) s_prefix[a] = a <= p.L ? p.tiles.prefix[a] : p.tiles.offsets[a - p.L - 1];
    __syncthreads();
    const Stretches cut(static_cast<int64_t>(s_prefix[p.L]) * sh.units, gridDim.x);
    const int64_t begin = cut.begin(blockIdx.x), end = cut.begin(blockIdx.x + 1);
    bool failed = false;
    int buffer = 0;
    uint32_t phase = 0;
    const auto next_buffer = [&]() {
        if (++buffer == kStages) {
            buffer = 0;
            phase ^= 1;
        }
    };

    if (warp >= kWarps) {
        // ------------------------------------------------------------ loaders
        // h comes kAhead stages ahead of its use, the rows' numbers as many ahead of that: each is a trip to memory
        const int loader = warp - kWarps;
        Walk walk(p, sh, s_prefix, s_offsets, begin, end);
        uint8_t* raw = smem_h + kStages * Lay::h + loader * kHeld * Lay::raw;
        const auto list = [&](int i) { return s_list[loader][i % kLists]; };
        const auto get_rows = [&](int i) {
            if (walk.at >= end) return;
            const int row0 = walk.row0() + 16 * loader, rows = max(min(16, walk.last() - row0), 0);
            int* to = list(i);
            if (lane < 16) {
                if (rows > 0) cp_async4(smem_u32(to + lane), p.tiles.perm + row0 + min(lane, rows - 1));
            } else if (lane == kScaleAt) {
                if (walk.slab.is_down || p.scale == nullptr) to[lane] = __float_as_int(1.0f);
                else cp_async4(smem_u32(to + lane), p.scale + walk.seg.adapter);
            } else if (lane <= kDownAt) {
                to[lane] = lane == kRowsAt ? rows : lane == kColAt ? walk.slab.col0 : lane == kRankAt ? walk.slab.rank0 : walk.slab.is_down;
            }
            walk.next();
        };
        const auto get_h = [&](int i) {
            if (i >= end - begin) return;
            const int* of = list(i);
            const int rank0 = of[kRankAt], rows = of[kRowsAt], ranks = min(kRanks, p.R - rank0);
            const float* h = (of[kDownAt] ? p.dh : p.h) + rank0;
#pragma unroll
            for (int j = 0; j < 2 * kM; ++j) {
                const int e = lane + 32 * j, token = e / (4 * kM), rank = e % (4 * kM) * 4;
                if (token < rows && rank < ranks)
                    cp_async16(smem_u32(raw + i % kHeld * Lay::raw + 16 * e), h + static_cast<int64_t>(of[token]) * p.R + rank);
            }
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) get_rows(i);
        cp_commit();
        cp_wait<0>();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            get_h(i);
            get_rows(kAhead + i);
            cp_commit();
        }
        const int stages = static_cast<int>(end - begin);
        int i = 0;
#pragma unroll 1
        for (; i < stages; ++i) {
            cp_wait<kAhead - 1>();                          // this stage's h and the rows of stage i + kAhead
            __syncwarp();
            get_h(i + kAhead);
            get_rows(i + 2 * kAhead);
            cp_commit();
            const int* of = list(i);
            const int rows = of[kRowsAt], col0 = of[kColAt], rank0 = of[kRankAt], ranks = min(kRanks, p.R - rank0), first_row = of[0];
            const bool is_down = of[kDownAt] != 0;
            const int blocks = min(kCols / 64, ((is_down ? p.K : p.N) - col0 + 63) / 64);
            if (!mbar_wait_bounded(&empty[buffer], phase ^ 1u, abort_flag, kWaitBudgetCycles)) failed = true;
            if (__any_sync(kAll, failed)) break;
            if (lane == 0) mbar_arrive_expect_tx(&full[buffer], rows > 0 ? 2048 * blocks : 0);
            __syncwarp();
            if (rows > 0) {
                const bool box = __all_sync(kAll, of[lane & 15] == first_row + (lane & 15));
                const uint32_t to = smem_u32(smem) + buffer * Lay::x + 2048 * loader, bar = smem_u32(&full[buffer]);
                if (box) {
                    if (lane < blocks) load_rows16(to + lane * Lay::tile, is_down ? &maps.x16 : &maps.dy16, bar, col0 + 64 * lane, first_row);
                } else if (lane < 4 * blocks) {
                    const int4 r = reinterpret_cast<const int4*>(of)[lane & 3];
                    const int four[4] = {r.x, r.y, r.z, r.w};
                    gather4(to + (lane >> 2) * Lay::tile + 512 * (lane & 3), is_down ? &maps.x : &maps.dy, bar, col0 + 64 * (lane >> 2), four);
                }
                const float scale = __int_as_float(of[kScaleAt]);
#pragma unroll
                for (int j = 0; j < 2 * kM; ++j) {
                    const int e = lane + 32 * j, token = e / (4 * kM), rank = e % (4 * kM) * 4;
                    const float4 h = *reinterpret_cast<const float4*>(raw + i % kHeld * Lay::raw + 16 * e);
                    const bool there = token < rows && rank < ranks;
                    float v[4] = {there ? h.x * scale : 0.0f, there ? h.y * scale : 0.0f, there ? h.z * scale : 0.0f, there ? h.w * scale : 0.0f};
                    uint8_t* to_h = smem_h + buffer * Lay::h + (16 * loader + token) * Lay::pitch + 2 * rank;
#pragma unroll
                    for (int t = 0; t < kTerms; ++t) {
                        const uint32_t lo = next_terms(v[0], v[1]), hi = next_terms(v[2], v[3]);
                        *reinterpret_cast<uint2*>(to_h + t * kTokens * Lay::pitch) = make_uint2(lo, hi);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[buffer]);
            next_buffer();
        }
        cp_wait<0>();
        if (__any_sync(kAll, failed)) {                     // copies under way land before the CTA leaves
            if (lane == 0) set_device_error(p.err, NVFP4_ERR_DEVICE_TIMEOUT);
            *abort_flag = 1;
            for (int s = 0; s < min(i, kStages); ++s) {
                if (--buffer < 0) {
                    buffer = kStages - 1;
                    phase ^= 1;
                }
                mbar_wait_bounded(&full[buffer], phase, nullptr, kWaitBudgetCycles);
            }
        }
        return;
    }

    // ------------------------------------------------------------ products: all ranks with 32 columns to a warp
    const uint32_t sx0 = smem_u32(smem) + (warp >> 1) * Lay::tile, sh0 = smem_u32(smem_h) + ((lane & 7) + (lane >> 4) * 8) * Lay::pitch + 16 * ((lane >> 3) & 1);
    for (int64_t at = begin; at < end;) {
        const Segment seg = find_unit(s_prefix, p.L, sh.units, at);
        const int64_t stop = min(end, seg.end);
        const Slab slab(p, sh, seg.unit);
        const int stages = static_cast<int>(stop - at);
        int left = s_offsets[seg.adapter + 1] - s_offsets[seg.adapter] - static_cast<int>(at - seg.begin) * kTokens;   // tokens
        float acc[kM][4][4], total[kM][4][4];
#pragma unroll
        for (int m = 0; m < kM; ++m) {
#pragma unroll
            for (int n = 0; n < 4; ++n) {
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][n][i] = total[m][n][i] = 0.0f;
            }
        }
#pragma unroll 1
        for (int s = 0; s < stages; ++s, left -= kTokens) {
            if (!failed && !mbar_wait_bounded(&full[buffer], phase, abort_flag, kWaitBudgetCycles)) failed = true;
            const uint32_t sx = sx0 + buffer * Lay::x, shh = sh0 + buffer * Lay::h;
#pragma unroll
            for (int k = 0; k < kTokens / 16; ++k) {
                if (left <= 16 * k) break;                  // nothing was loaded
                uint32_t b[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
                    ldsm4_trans(sx + swizzled(16 * k + (lane & 7) + ((lane >> 3) & 1) * 8, 4 * (warp & 1) + 2 * n + (lane >> 4)), b[n]);
#pragma unroll
                for (int m = 0; m < kM; ++m) {
#pragma unroll
                    for (int t = 0; t < kTerms; ++t) {
                        uint32_t a[4];
                        ldsm4_trans(shh + (t * kTokens + 16 * k) * Lay::pitch + 32 * m, a);
#pragma unroll
                        for (int n = 0; n < 4; ++n) mma(__nv_bfloat16(), acc[m][n], a, b[n >> 1][2 * (n & 1)], b[n >> 1][2 * (n & 1) + 1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[buffer]);
            next_buffer();
            if ((s + 1) % kChain == 0 || s + 1 == stages) {
#pragma unroll
                for (int m = 0; m < kM; ++m) {
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            total[m][n][i] += acc[m][n][i];
                            acc[m][n][i] = 0.0f;
                        }
                    }
                }
            }
        }
        // a lane's sums of tile (m, n): ranks 16 m + lane / 4 and 8 more, columns 32 warp + 8 n + 2 (lane % 4) and the next
        const int r = lane >> 2, c = 32 * warp + 2 * (lane & 3);
        bool write = at == seg.begin && stop == seg.end;
        if (!write) {
            // parts as the lanes hold them; the last CTA to leave one adds the unit's in order
            const int first_cta = cut.owner(seg.begin), last_cta = cut.owner(seg.end - 1);
            float4* part = reinterpret_cast<float4*>(p.parts + (2 * static_cast<int64_t>(blockIdx.x) + (at != begin)) * kPart) + threadIdx.x;
#pragma unroll
            for (int i = 0; i < 4 * kM; ++i) {
                const float (&v)[4] = total[i >> 2][i & 3];
                part[i * kThreads] = make_float4(v[0], v[1], v[2], v[3]);
            }
            __threadfence();
            consumer_barrier();
            if (threadIdx.x == 0) s_last = atomicAdd(p.tiles.pieces + first_cta, 1) == last_cta - first_cta;
            consumer_barrier();
            write = s_last;
            if (write) {
                __threadfence();
#pragma unroll
                for (int m = 0; m < kM; ++m) {
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) total[m][n][i] = 0.0f;
                    }
                }
                for (int k = first_cta; k <= last_cta; ++k) {
                    const float4* from = reinterpret_cast<const float4*>(p.parts + (2 * static_cast<int64_t>(k) + (cut.begin(k) < seg.begin)) * kPart) + threadIdx.x;
#pragma unroll
                    for (int i = 0; i < 4 * kM; ++i) {
                        const float4 w = __ldcg(from + i * kThreads);
                        float (&v)[4] = total[i >> 2][i & 3];
                        v[0] += w.x, v[1] += w.y, v[2] += w.z, v[3] += w.w;
                    }
                }
            }
        }
        if (write) {
#pragma unroll
            for (int m = 0; m < kM; ++m) {
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    slab.store(p, seg.adapter, 16 * m + r, c + 8 * n, total[m][n][0], total[m][n][1]);
                    slab.store(p, seg.adapter, 16 * m + r + 8, c + 8 * n, total[m][n][2], total[m][n][3]);
                }
            }
        }
        at = stop;
    }
    if (failed) {
        if (lane == 0) set_device_error(p.err, NVFP4_ERR_DEVICE_TIMEOUT);
        *abort_flag = 1;
    }
}

Shape shape_of(int64_t K, int64_t N, int R) {
    Shape sh;
    sh.slabs_k = static_cast<int>((K + kCols - 1) / kCols);
    sh.rank_parts = (R + kRanks - 1) / kRanks;
    sh.units = (sh.slabs_k + static_cast<int>((N + kCols - 1) / kCols)) * sh.rank_parts;
    return sh;
}
// CTAs: two to an SM, with four stages each at least.
int ctas_of(int64_t T, int L, const Shape& sh) {
    const int64_t all = (T / kTokens + L) * sh.units, most = 2 * std::min(device_sm_count(), kMaxCtas / 2), few = (all + 3) / 4;
    return static_cast<int>(few < most ? few : most);
}

template <int kM>
cudaError_t launch(const GradParams& p, int64_t T, cudaStream_t st) {
    const Shape sh = shape_of(p.K, p.N, p.R);
    const unsigned ctas = static_cast<unsigned>(ctas_of(T, p.L, sh));
    static Ready ready;
    const cudaError_t e = allow_shared(reinterpret_cast<const void*>(grad_kernel<kM>), GradLayout<kM>::bytes(kMaxAdapters), ready);
    if (e != cudaSuccess) return e;
    GradMaps maps;
    if (!make_units_map(&maps.x, p.x, p.K, T, p.ldx, 0, 0, 1) || !make_units_map(&maps.x16, p.x, p.K, T, p.ldx, 0, 0, 16) ||
        !make_units_map(&maps.dy, p.dy, p.N, T, p.lddy, 0, 0, 1) || !make_units_map(&maps.dy16, p.dy, p.N, T, p.lddy, 0, 0, 16))
        return cudaErrorInvalidValue;
    return launch_pdl(true, grad_kernel<kM>, dim3(ctas), dim3(kThreads + 32 * kLoaders), static_cast<size_t>(GradLayout<kM>::bytes(p.L)), st, maps, p, sh);
}

}  // namespace

size_t grad_bytes(int64_t T, int L, int R, int64_t K, int64_t N) {
    return 2 * static_cast<size_t>(ctas_of(T, L, shape_of(K, N, R))) * kRanks * kCols * sizeof(float);
}

cudaError_t launch_grad(const GradParams& p, int64_t T, cudaStream_t st) { return p.R <= 16 ? launch<1>(p, T, st) : launch<2>(p, T, st); }

}  // namespace lora
}  // namespace nvfp4
