// Gradients of low-rank adapters:  dA_a = sum_t dh_t x_t^T  [R][K],  dB_a = sum_t s_a dy_t h_t^T  [N][R],  over the tokens of
// adapter a in their order.
//
// Both are sums over tokens of a column of R values (dh, or s h) times a row of x, or dy.  The work is units (an adapter, up
// to 32 of its ranks, a slab of 256 columns of x or dy) of stages (32 tokens), one behind the other, cut into as many equal
// stretches as CTAs run at once: requests are uneven, and with CTAs of a cluster sharing a unit's tokens the longest adapter's
// took twice the mean, and 1.7 waves two (93 us for 16384 x (4096 + 4096), rank 16).  A unit that lies in one stretch is written by
// its CTA; of the others each CTA leaves its part in the workspace (at most two: where its stretch begins and where it
// ends), and the last to do so adds the unit's parts in order, whoever that is: the same bits every time.  (A second kernel
// for that took 8 to 11 us.)  More than 32 ranks read
// a slab again, out of L2.
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
constexpr int kStages = 4, kChain = 8;    // stages of the ring; of a chain of products
constexpr int kIndexed = 16;              // stages whose rows are listed at a time
constexpr int kPitch = kCols + 4;         // floats of a row of the sums in shared memory

template <int kM>
struct GradLayout {
    static constexpr int pitch = padded_pitch(16 * kM);
    static constexpr int tile = kTokens * 128;                       // 64 columns
    static constexpr int h_at = tile * (kCols / 64);
    static constexpr int stage = h_at + kTerms * kTokens * pitch;    // a multiple of 128
    static constexpr int sums = 16 * kM * kPitch * 4;
    static constexpr int total = kStages * stage > sums ? kStages * stage : sums;
    static_assert(h_at % 128 == 0 && stage % 16 == 0, "16-byte chunks");
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
    // rank and column of element i, in the order in which they lie in the gradient (ranks and kCols are multiples of 4)
    __device__ __forceinline__ void place(int i, int& r, int& c) const {
        c = is_down ? i % kCols : static_cast<unsigned>(i) / static_cast<unsigned>(ranks);
        r = is_down ? i / kCols : i - c * ranks;
    }
    // elements i to i + 3, which lie side by side
    __device__ __forceinline__ void store(const GradParams& p, int adapter, int i, const float4& v) const {
        int r, c;
        place(i, r, c);
        const int there = is_down ? width - col0 - c : col0 + c < width ? 4 : 0;
        float* at = is_down ? p.ddown + (static_cast<int64_t>(adapter) * p.R + rank0 + r) * p.K + col0 + c
                            : p.dup + (static_cast<int64_t>(adapter) * p.N + col0 + c) * p.R + rank0 + r;
        const float w[4] = {v.x, v.y, v.z, v.w};
        if (there >= 4 && p.grads_wide) {
            *reinterpret_cast<float4*>(at) = v;
            return;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j < there) at[j] = w[j];
        }
    }
};

template <int kM>
__device__ __forceinline__ void add_stages(const GradParams& p, const Slab& slab, int adapter, int skip, int stages, uint8_t* smem,
                                           int (&s_rows)[2][kIndexed * kTokens], float (&total)[kM][4][4]) {
    using Lay = GradLayout<kM>;
    const uint32_t base = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool is_down = slab.is_down;
    const int col0 = slab.col0, width = slab.width, ranks = slab.ranks;
    const uint16_t* x = is_down ? p.x : p.dy;
    const int64_t ldx = is_down ? p.ldx : p.lddy;
    const float* h = (is_down ? p.dh : p.h) + slab.rank0;
    const float scale = is_down || p.scale == nullptr ? 1.0f : p.scale[adapter];
    const int begin = p.tiles.offsets[adapter], first = skip * kTokens, last = p.tiles.offsets[adapter + 1] - begin;
    const int32_t* perm = p.tiles.perm + begin + first;

    const bool full_slab = col0 + kCols <= width;
    // rows of kIndexed stages, block by block; -1 behind the last
    static_assert(kIndexed * kTokens == 2 * kThreads, "two rows to a thread");
    const auto get_rows = [&](int block, int (&to)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = block * kIndexed * kTokens + i * kThreads + static_cast<int>(threadIdx.x);
            to[i] = at < last - first ? perm[at] : -1;
        }
    };
    const auto put_rows = [&](int block, const int (&from)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) s_rows[block & 1][i * kThreads + threadIdx.x] = from[i];
    };
    const auto row_at = [&](int s, int r) { return s_rows[(s / kIndexed) & 1][s % kIndexed * kTokens + r]; };
    const auto load_x = [&](int s) {
        if (s < stages) {
            const uint32_t at = base + s % kStages * Lay::stage;
            const int r = threadIdx.x >> 3, t = row_at(s, r);
            const uint16_t* row = t < 0 ? x : x + t * ldx;
            if (full_slab && (s + 1) * kTokens <= last - first) {
                const uint32_t to = at + swizzled(r, threadIdx.x & 7);
                const uint16_t* from = row + col0 + 8 * (threadIdx.x & 7);
#pragma unroll
                for (int i = 0; i < kCols / 64; ++i) cp_async16(to + i * Lay::tile, from + 64 * i);
            } else {
#pragma unroll
                for (int i = 0; i < kCols / 64; ++i) {
                    const int c = col0 + 64 * i + 8 * (threadIdx.x & 7), left = t < 0 ? 0 : min(max(width - c, 0), 8);
                    cp_async16(at + i * Lay::tile + swizzled(r, threadIdx.x & 7), left ? row + c : row, 2 * left);
                }
            }
        }
        cp_commit();
    };
    // h: 32 tokens x up to 32 ranks, 4 values to a thread
    const int h_row = threadIdx.x >> 3, h_col = 4 * (threadIdx.x & 7);
    const auto load_h = [&](int s) {
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (s < stages && h_col < ranks) {
            const int t = row_at(s, h_row);
            if (t >= 0) v = *reinterpret_cast<const float4*>(h + static_cast<int64_t>(t) * p.R + h_col);
        }
        return v;
    };
    const auto store_h = [&](int s, const float4& held) {
        if (h_col >= 16 * kM) return;
        float v[4] = {held.x * scale, held.y * scale, held.z * scale, held.w * scale};
        uint8_t* to = smem + s % kStages * Lay::stage + Lay::h_at + h_row * Lay::pitch + 2 * h_col;
#pragma unroll
        for (int t = 0; t < kTerms; ++t)
            *reinterpret_cast<uint2*>(to + t * kTokens * Lay::pitch) = make_uint2(next_terms(v[0], v[1]), next_terms(v[2], v[3]));
    };

    float acc[kM][4][4];
#pragma unroll
    for (int m = 0; m < kM; ++m) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][n][i] = total[m][n][i] = 0.0f;
        }
    }
    int first_rows[2];
    get_rows(0, first_rows);
    put_rows(0, first_rows);
    __syncthreads();
    for (int s = 0; s < kStages - 1; ++s) load_x(s);
    float4 held[kStages - 1];             // of the stages that are under way
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) held[s] = load_h(s);
    int listed[2] = {-1, -1};
#pragma unroll 1
    for (int s = 0; s < stages; ++s) {
        store_h(s, held[0]);
        cp_wait<kStages - 2>();
        // the rows of the block that loads reach from the next stage on; its place was last read a block ago
        const int ahead = s % kIndexed;
        if (ahead == kIndexed - kStages) put_rows(s / kIndexed + 1, listed);
        __syncthreads();                                    // the stage is there, the one before is used up
        if (ahead == kIndexed - kStages - 4) get_rows(s / kIndexed + 1, listed);
        load_x(s + kStages - 1);
#pragma unroll
        for (int i = 0; i + 2 < kStages; ++i) held[i] = held[i + 1];
        held[kStages - 2] = load_h(s + kStages - 1);
        const uint32_t sx = base + s % kStages * Lay::stage + (warp >> 1) * Lay::tile, sh = base + s % kStages * Lay::stage + Lay::h_at;
#pragma unroll
        for (int k = 0; k < kTokens / 16; ++k) {
            uint32_t b[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n)
                ldsm4_trans(sx + swizzled(16 * k + (lane & 7) + ((lane >> 3) & 1) * 8, 4 * (warp & 1) + 2 * n + (lane >> 4)), b[n]);
#pragma unroll
            for (int m = 0; m < kM; ++m) {
#pragma unroll
                for (int t = 0; t < kTerms; ++t) {
                    uint32_t a[4];
                    ldsm4_trans(sh + t * kTokens * Lay::pitch + (16 * k + (lane & 7) + (lane >> 4) * 8) * Lay::pitch + 32 * m +
                                    16 * ((lane >> 3) & 1), a);
#pragma unroll
                    for (int n = 0; n < 4; ++n) mma(__nv_bfloat16(), acc[m][n], a, b[n >> 1][2 * (n & 1)], b[n >> 1][2 * (n & 1) + 1]);
                }
            }
        }
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

    cp_wait<0>();
    __syncthreads();
}

// Adds the parts of a unit that lies in the stretches first_cta to last_cta (the first one's begins with it or not).
__device__ __forceinline__ void join_parts(const GradParams& p, const Slab& slab, const Segment& seg, const Stretches& cut, int first_cta, int last_cta) {
    // four elements at a time and all of a thread's at once: the parts' latency once for each, not for each element too
    constexpr int kMine = kRanks * kCols / 4 / kThreads;
    const int count = slab.ranks * kCols / 4;
    float4 v[kMine];
#pragma unroll
    for (int j = 0; j < kMine; ++j) v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int k = first_cta; k <= last_cta; ++k) {
        const float* part = p.parts + (2 * static_cast<int64_t>(k) + (cut.begin(k) < seg.begin)) * (kRanks * kCols);
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            const int i = threadIdx.x + j * kThreads;
            if (i >= count) break;
            const float4 w = __ldcg(reinterpret_cast<const float4*>(part + 4 * i));
            v[j] = make_float4(v[j].x + w.x, v[j].y + w.y, v[j].z + w.z, v[j].w + w.w);
        }
    }
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        const int i = threadIdx.x + j * kThreads;
        if (i < count) slab.store(p, seg.adapter, 4 * i, v[j]);
    }
}

template <int kM>
__global__ void __launch_bounds__(kThreads, 2) grad_kernel(const GradParams p, const Shape sh) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_rows[2][kIndexed * kTokens];
    __shared__ int s_last, s_prefix[kMaxAdapters + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    for (int a = threadIdx.x; a <= p.L; a += kThreads) s_prefix[a] = p.tiles.prefix[a];
    __syncthreads();
    const Stretches cut(static_cast<int64_t>(s_prefix[p.L]) * sh.units, gridDim.x);
    const int64_t begin = cut.begin(blockIdx.x), end = cut.begin(blockIdx.x + 1);
    for (int64_t at = begin; at < end;) {
        const Segment seg = find_unit(s_prefix, p.L, sh.units, at);
        const int64_t stop = min(end, seg.end);
        const Slab slab(p, sh, seg.unit);
        float total[kM][4][4];
        add_stages<kM>(p, slab, seg.adapter, static_cast<int>(at - seg.begin), static_cast<int>(stop - at), smem, s_rows, total);
        float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int m = 0; m < kM; ++m) {
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                float* to = sums + (16 * m + (lane >> 2)) * kPitch + 32 * warp + 8 * n + 2 * (lane & 3);
                *reinterpret_cast<float2*>(to) = make_float2(total[m][n][0], total[m][n][1]);
                *reinterpret_cast<float2*>(to + 8 * kPitch) = make_float2(total[m][n][2], total[m][n][3]);
            }
        }
        __syncthreads();
        const bool whole = at == seg.begin && stop == seg.end;
        float* part = p.parts + (2 * static_cast<int64_t>(blockIdx.x) + (at != begin)) * (kRanks * kCols);
        for (int i = threadIdx.x; i < slab.ranks * kCols / 4; i += kThreads) {
            int r, c;
            slab.place(4 * i, r, c);
            const float* from = sums + r * kPitch + c;
            const int step = slab.is_down ? 1 : kPitch;
            const float4 v = make_float4(from[0], from[step], from[2 * step], from[3 * step]);
            if (whole) slab.store(p, seg.adapter, 4 * i, v);
            else *reinterpret_cast<float4*>(part + 4 * i) = v;
        }
        if (!whole) {
            const int first_cta = cut.owner(seg.begin), last_cta = cut.owner(seg.end - 1);
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) s_last = atomicAdd(p.tiles.pieces + first_cta, 1) == last_cta - first_cta;
            __syncthreads();
            if (s_last) {
                __threadfence();
                join_parts(p, slab, seg, cut, first_cta, last_cta);
            }
        }
        __syncthreads();
        at = stop;
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
    const cudaError_t e = allow_shared(reinterpret_cast<const void*>(grad_kernel<kM>), GradLayout<kM>::total, ready);
    if (e != cudaSuccess) return e;
    return launch_pdl(true, grad_kernel<kM>, dim3(ctas), dim3(kThreads), static_cast<size_t>(GradLayout<kM>::total), st, p, sh);
}

}  // namespace

size_t grad_bytes(int64_t T, int L, int R, int64_t K, int64_t N) {
    return 2 * static_cast<size_t>(ctas_of(T, L, shape_of(K, N, R))) * kRanks * kCols * sizeof(float);
}

cudaError_t launch_grad(const GradParams& p, int64_t T, cudaStream_t st) { return p.R <= 16 ? launch<1>(p, T, st) : launch<2>(p, T, st); }

}  // namespace lora
}  // namespace nvfp4
