// Low-rank adapters, tiles of up to 128 rows: prompts and training batches.  lora.cuh says what is computed.
//
// Bound by memory, so the loads are not to pause: loader warps keep a ring of stages full, first its share of C (64
// columns of x and of the adapter a stage), then its share of D (128 bytes a row of y and the adapter's part), then the next
// tile's, whatever the 8 other warps are at.  Those take 16 rows each: products of the first phase into registers; the
// CTAs' sums meet in shared memory over the cluster, each CTA adding its share of the rows and handing their terms to all; products of the
// second phase are added to y where it lies in shared memory, which goes out from there in whole rows of 128 bytes.
//
// x and y come by TMA, 16 rows to an instruction where they lie in a row, four rows of any place otherwise.  Where rows of y
// start on no 16-byte boundary four loader warps read aligned words of them and shift those together, a stage's on
// their way while the last one's are put in place.  (With the loads
// and the products in the same warps, cp.async and a barrier for each stage, 16384 x 4096 -> 4096 of rank 16 took 145 to 199 us:
// 500 instructions a stage and warp, half of them addresses.)
//
// 16384 x 4096 -> 4096 of rank 16 take 88 us, 403 MB at 4.6 TB/s, and its dx without the sum 79, 268 MB at 3.4 TB/s; a kernel
// that only copies 268 MB 128 bytes at a time from row to row takes 61, 4.4 TB/s (52 in longer pieces, 5.1).  Issue slots are 47% full, of a stage
// 320 instructions a warp, and with 18 warps an SM the products' and shared memory's latency shows.  At rank 64 registers and shared
// memory leave one CTA, 9 warps, to an SM: 2000 x 2048 -> 1536 27 us, 8191 rows of dx (1999 -> 4096) 60; issue slots 35% and tensor pipe
// 27% full, each instruction waits for the last.  (Two warps to the same 16 rows, ranks and outputs shared out, were within 4%.)
//
// A stage goes back to TMA without a proxy fence where it was only read by ldmatrix: each register that was loaded goes into a product in
// front of the warp's arrival, so the read is over.  Where a stage was written to (sums beside y, shifted words) or read by ordinary
// loads (rows on their way out) a fence stands in front of the arrival, or of the copy.
#pragma once

#include "lora_launch.cuh"

namespace nvfp4 {
namespace lora {

struct ManyMaps {
    CUtensorMap x, y, x16, y16, down, up;   // of x and y: boxes of one row, for gathers, and of 16
};

// Step kk of the second product of a warp's 16 rows (`a`: their terms) with a group of 32 outputs (`up`: the group's rows, or
// columns): acc[i] gets outputs 8 i to 8 i + 7.
template <typename T, bool kTrans, int kTerms, int kRowBytes>
__device__ __forceinline__ void multiply_outputs(float (&acc)[4][4], const uint32_t (&a)[kTerms][4], uint32_t up, int block_bytes,
                                                 int first_chunk, int kk, int lane) {
    constexpr int kPer = kRowBytes / 32;  // steps of 16 ranks to a row
    uint32_t b[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {         // two tiles of 8 outputs at once
        if (!kTrans)                      // rows of ranks
            ldsm4(up + kk / kPer * block_bytes + swizzled_rows<kRowBytes>(8 * (2 * i + (lane >> 4)) + (lane & 7), 2 * (kk % kPer) + ((lane >> 3) & 1)), b[i]);
        else                              // rows of 64 outputs
            ldsm4_trans(up + swizzled(16 * kk + ((lane >> 3) & 1) * 8 + (lane & 7), first_chunk + 2 * i + (lane >> 4)), b[i]);
    }
#pragma unroll
    for (int t = 0; t < kTerms; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) mma(T(), acc[i], a[t], b[i >> 1][2 * (i & 1)], b[i >> 1][2 * (i & 1) + 1]);
    }
}

// 16 bytes of out.  dx is not to push dy out of L2, which the adapters' gradients read next.
template <bool kTrans>
__device__ __forceinline__ void store_chunk(uint8_t* to, const uint4& v) {
    if (kTrans) __stcs(reinterpret_cast<uint4*>(to), v);
    else *reinterpret_cast<uint4*>(to) = v;
}
// The first `left` of 8 units.
__device__ __forceinline__ void store_units(uint8_t* to, const uint4& v, int left, int units) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (units == 2) {
            if (2 * j < left) reinterpret_cast<uint32_t*>(to)[j] = w[j];
        } else {
            if (2 * j < left) reinterpret_cast<uint16_t*>(to)[2 * j] = static_cast<uint16_t>(w[j]);
            if (2 * j + 1 < left) reinterpret_cast<uint16_t*>(to)[2 * j + 1] = static_cast<uint16_t>(w[j] >> 16);
        }
    }
}
// `there` units of a row by 8 lanes that hold 8 each (`to`: the lane's, nullptr: no row), where they start on no 16-byte
// boundary: each lane shifts its own and its left neighbour's into the aligned word between them, and the units in front of
// the first and behind the last whole word go one to a lane.
template <int kUnits>
__device__ __forceinline__ void store_unaligned(uint8_t* to, const uint4& v, int there, int lane) {
    const int k = lane & 7, off = static_cast<int>(reinterpret_cast<uintptr_t>(to) & 15), first = off ? (16 - off) / 2 : 0;
    Straddle w;                           // the word that ends inside the lane's units: from unit 8 k - off / 2 on
    w.lo = make_uint4(__shfl_up_sync(kAll, v.x, 1), __shfl_up_sync(kAll, v.y, 1), __shfl_up_sync(kAll, v.z, 1), __shfl_up_sync(kAll, v.w, 1));
    w.hi = v;
    w.left = 8;
    w.off = (16 - off) & 15;
    if (off == 0) w.lo = v;
    const uint4 word = w.value();
    if (to != nullptr && (off == 0 || k > 0) && 8 * k - off / 2 + 8 <= there) *reinterpret_cast<uint4*>(to - off) = word;
    // what is left: units [0, first) and [last, there), at most 14
    const int last = first + (there > first ? (there - first) / 8 * 8 : 0), head = min(first, there), tail = max(last, head), rest = head + max(there - tail, 0);
    for (int j = k * kUnits;; j += 8 * kUnits) {
        if (!__any_sync(kAll, to != nullptr && j < rest)) break;
        const int unit = j < head ? j : tail + j - head;
        uint32_t w[4] = {v.x, v.y, v.z, v.w}, got = 0;
        const int from = (lane & ~7) + (min(unit, 63) >> 3), word = (unit & 7) >> 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = __shfl_sync(kAll, w[i], from);
            if (word == i) got = x;
        }
        if (to == nullptr || j >= rest) continue;
        uint8_t* at = to + 2 * (unit - 8 * k);
        if (kUnits == 2) *reinterpret_cast<uint32_t*>(at) = got;
        else *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(unit & 1 ? got >> 16 : got);
    }
}

// kLoaders: warps that load, 1 (where rows of y and out start on 16-byte boundaries: all by TMA) or 4 (y by shifted words).
// kType: y's and out's (branches by it for every value took 3000 cycles a stage).
template <typename T, bool kTrans, int kType, int kRank, int kLoaders>
__global__ void __launch_bounds__(kThreads + 32 * kLoaders, kRank <= 32 && kLoaders == 1 ? 2 : 1)
    many_kernel(const __grid_constant__ ManyMaps maps, const Params p, const ManyLayout lay) {
    constexpr int kTiles = kRank / 8;
    constexpr bool kWide = kType == NVFP4_TYPE_F32;
    constexpr int kCols = kWide ? 32 : 64, kUnits = kWide ? 2 : 1;   // outputs of a stage; 16-bit units of an output
    constexpr int kTerms = terms_of<T>(kType), kRankBytes = rank_bytes(kRank);
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], sums_ready, h_ready;
    __shared__ float s_undo[kManyRows];
    __shared__ int abort_word;
    volatile int* abort_flag = &abort_word;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t base = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_rank()), split = static_cast<int>(cluster_size());
    const int groups = kGroups / split, steps = sub_steps(p.C), group_cols = kWarps * sub_rounds(p.C) * steps * 16;   // a multiple of 64
    const int c0 = min(rank * groups * group_cols, p.C), c1 = min(c0 + groups * group_cols, p.C);
    const int chunks = (p.D + kCols - 1) / kCols, per_cta = (chunks + split - 1) / split;
    const int chunk0 = min(rank * per_cta, chunks), chunk1 = min(chunk0 + per_cta, chunks);
    if (threadIdx.x == 0) {
        for (int s = 0; s < lay.stages; ++s) {
            mbar_init(&full[s], kLoaders == 1 ? 1 : 32 * kLoaders);
            mbar_init(&empty[s], kWarps);
        }
        mbar_init(&sums_ready, split);
        mbar_init(&h_ready, split);
        abort_word = 0;
        fence_barrier_init();
    }
    if (threadIdx.x == kThreads) {
        prefetch_tensormap(&maps.x16);
        prefetch_tensormap(&maps.y16);
        prefetch_tensormap(&maps.down);
        prefetch_tensormap(&maps.up);
    }
    __syncthreads();
    cluster_barrier();                                      // every CTA's barriers are there
    pdl_wait();
    const int count = *p.tiles.count;
    bool failed = false;
    int buffer = 0;
    uint32_t phase = 0;
    const auto next_buffer = [&]() {
        if (++buffer == lay.stages) {
            buffer = 0;
            phase ^= 1;
        }
    };

    if (warp >= kWarps) {
        // ------------------------------------------------------------ loaders
        const int thread = threadIdx.x - kThreads;
        int issued = 0;
        for (int q = blockIdx.x / split; q < count; q += gridDim.x / split) {
            const int adapter = p.tiles.adapter[q], start = p.tiles.start[q];
            const int rows = min(kManyRows, p.tiles.offsets[(adapter < 0 ? p.L : adapter) + 1] - start);
            if (adapter < 0 && p.skip_none) continue;
            const int x_stages = adapter < 0 ? 0 : (c1 - c0 + 63) / 64, all = x_stages + chunk1 - chunk0;
            // TMA: a lane's four rows (behind the last: outside the tensor, zeros); otherwise a thread's chunk of every 16th row
            int four[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) four[i] = 4 * lane + i < rows ? p.tiles.perm[start + 4 * lane + i] : p.T;
            // 16 rows in a row, as those of one request are, are one box (the rows behind the tile's last are read along)
            const int group_row = __shfl_sync(kAll, four[0], lane & ~3);
            bool apart = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) apart |= 4 * lane + i < rows && four[i] != group_row + 4 * (lane & 3) + i;
            const bool box = (__ballot_sync(kAll, apart) >> (lane & ~3) & 15) == 0;
            const bool group = 16 * (lane >> 2) < rows && warp == kWarps && (!box || (lane & 3) == 0);
            constexpr int kMine = kLoaders == 1 ? 1 : 8;
            int row[kMine];
            Straddle words[kMine];                              // of y's next stage
            const auto fetch = [&](int s) {
                if (s < x_stages || s >= all || p.y == nullptr) return;
                const uint16_t* from = static_cast<const uint16_t*>(p.y);
                const int64_t ld = p.ldy * kUnits;
                const int unit = (chunk0 + s - x_stages) * kCols * kUnits + 8 * (thread & 7);
#pragma unroll
                for (int i = 0; i < kMine; ++i) {
                    if (row[i] >= 0) words[i].load(from + row[i] * ld, unit, p.D * kUnits);
                }
            };
            if (kLoaders > 1) {
#pragma unroll
                for (int i = 0; i < kMine; ++i) {
                    const int r = (thread >> 3) + 16 * i;
                    row[i] = r < rows ? p.tiles.perm[start + r] : -1;
                }
                fetch(0);
            }
            for (int s = 0; s < all; ++s, ++issued) {
                if (!mbar_wait_bounded(&empty[buffer], phase ^ 1u, abort_flag, kWaitBudgetCycles)) failed = true;
                if (__any_sync(kAll, failed)) break;
                const uint32_t at = base + buffer * lay.stage, part = at + kManyRows * 128, bar = smem_u32(&full[buffer]);
                const bool is_x = s < x_stages, tma = is_x || kLoaders == 1, none = !is_x && p.y == nullptr;
                const int c = is_x ? c0 + 64 * s : (chunk0 + s - x_stages) * kCols;
                if (kLoaders > 1) fence_proxy_async_shared();
                if (thread == 0) {
                    const int bytes = (adapter < 0 ? 0 : is_x ? lay.down_bytes : lay.up_bytes) + (tma && !none ? (rows + 15) / 16 * 2048 : 0);
                    mbar_arrive_expect_tx(&full[buffer], bytes);
                    if (adapter >= 0 && is_x) {
                        if (!kTrans) load_box(part, &maps.down, bar, c, 0, adapter);
                        else for (int b = 0; b < lay.blocks; ++b) load_box(part + b * 64 * kRankBytes, &maps.down, bar, 64 * b, c, adapter);
                    } else if (adapter >= 0) {
                        if (kTrans) load_box(part, &maps.up, bar, c, 0, adapter);
                        else for (int b = 0; b < lay.blocks; ++b) load_box(part + b * kCols * kRankBytes, &maps.up, bar, 64 * b, c, adapter);
                    }
                }
                __syncwarp();
                if (tma && !none && group) {
                    if (box) load_rows16(at + 512 * lane, is_x ? &maps.x16 : &maps.y16, bar, is_x ? c : c * kUnits, group_row);
                    else gather4(at + 512 * lane, is_x ? &maps.x : &maps.y, bar, is_x ? c : c * kUnits, four);
                }
                if (kLoaders > 1) {
                    if (!tma && !none) {
#pragma unroll
                        for (int i = 0; i < kMine; ++i) {
                            if (row[i] >= 0) words[i].store(at + swizzled((thread >> 3) + 16 * i, thread & 7));
                        }
                    }
                    fetch(s + 1);
                    if (thread != 0) mbar_arrive(&full[buffer]);
                }
                next_buffer();
            }
            if (failed) break;
        }
        if (__any_sync(kAll, failed)) {                     // copies under way land before the CTA leaves
            if (lane == 0) set_device_error(p.err, NVFP4_ERR_DEVICE_TIMEOUT);
            *abort_flag = 1;
            for (int s = 0; s < min(issued, lay.stages); ++s) {
                if (--buffer < 0) {
                    buffer = lay.stages - 1;
                    phase ^= 1;
                }
                mbar_wait_bounded(&full[buffer], phase, nullptr, kWaitBudgetCycles);
            }
        }
    } else {
        // ------------------------------------------------------------ products and outputs
        const int quad = lane >> 2, my_row = 16 * warp + quad, pitch = padded_pitch(rank_up(p.R));
        const uint32_t ha = base + lay.h + (16 * warp + (lane & 7) + ((lane >> 3) & 1) * 8) * pitch + 16 * (lane >> 4);
        uint32_t tile_phase = 0;
        for (int q = blockIdx.x / split; q < count; q += gridDim.x / split) {
            const int adapter = p.tiles.adapter[q], start = p.tiles.start[q];
            const int rows = min(kManyRows, p.tiles.offsets[(adapter < 0 ? p.L : adapter) + 1] - start);
            if (adapter < 0 && p.skip_none) continue;
            const int x_stages = adapter < 0 ? 0 : (c1 - c0 + 63) / 64;
            const bool busy = 16 * warp < rows;
            // a lane's 16 bytes of every fourth of the warp's rows of out
            uint8_t* out[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 16 * warp + (lane >> 3) + 4 * i;
                out[i] = r < rows ? static_cast<uint8_t*>(p.out) + (p.tiles.perm[start + r] * p.ldo + chunk0 * kCols) * (2 * kUnits) + 16 * (lane & 7)
                                  : nullptr;
            }
            if (adapter >= 0) {
                float acc[kTiles][4], total[kTiles][4];
#pragma unroll
                for (int j = 0; j < kTiles; ++j) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[j][i] = total[j][i] = 0.0f;
                }
                // sums of the groups, a pair's in one place (the sums'), the other pair's in another, h's.  Only the ring holds the warps
                // together, and sums2's rows lie over other warps' h: all of them are to be behind the second product of the tile in
                // front (16384 x 4096 -> 4096 of rank 16 took as long without the barrier; with one where sums2 is first written, in
                // the loop, rank 96 to FP32 on odd rows spilled and took 195 us instead of 174)
                consumer_barrier();
                float* const sums = reinterpret_cast<float*>(smem + lay.sum) + my_row * lay.sum_pitch + 2 * (lane & 3);
                float* const sums2 = sums + (lay.h - lay.sum) / 4;
                const auto close_group = [&](int group) {
                    float* const to = group & 2 ? sums2 : sums;
#pragma unroll
                    for (int j = 0; j < kTiles; ++j) {
                        if (8 * j >= p.R) break;
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            float2* const at = reinterpret_cast<float2*>(to + 8 * r * lay.sum_pitch + 8 * j);
                            float2 v = make_float2(total[j][2 * r] + acc[j][2 * r], total[j][2 * r + 1] + acc[j][2 * r + 1]);
                            if (group & 1) {
                                const float2 was = *at;
                                v = make_float2(was.x + v.x, was.y + v.y);
                            }
                            *at = v;
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) total[j][i] = acc[j][i] = 0.0f;
                    }
                };
                int left = steps, group = 0;                // steps of the sub-slice
                for (int s = 0, next = group_cols; s < x_stages; ++s) {
                    if (64 * s == next) {
                        close_group(group++);
                        next += group_cols;
                    }
                    if (!failed && !mbar_wait_bounded(&full[buffer], phase, abort_flag, kWaitBudgetCycles)) failed = true;
                    if (busy) {
                        const uint32_t at = base + buffer * lay.stage, sx = at + 2048 * warp + lane_rows(lane);
                        const uint32_t sd = at + kManyRows * 128 +
                                            (kTrans ? swizzled_rows<kRankBytes>(((lane >> 3) & 1) * 8 + (lane & 7), lane >> 4) : lane_down<false>(lane, p.R));
                        // the whole stage: behind C lie zeros, and a CTA's share ends with a stage or with C
                        uint32_t a[4][4];
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) ldsm4(sx ^ (kk << 5), a[kk]);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            // all of kRank: what lies behind R is zeros, or anything, and goes nowhere
#pragma unroll
                            for (int j = 0; j < kTiles; j += 2) {
                                uint32_t b[4];
                                if (!kTrans) ldsm4((sd ^ (kk << 5)) + 1024 * j, b);   // rows of 64 columns
                                else ldsm4_trans((sd ^ ((j & 7) << 4)) + (j >> 3) * 64 * 128 + 16 * kRankBytes * kk, b);   // of ranks
                                mma(T(), acc[j], a[kk], b[0], b[1]);
                                mma(T(), acc[j + 1], a[kk], b[2], b[3]);
                            }
                            if (--left == 0) {
                                left = steps;
#pragma unroll
                                for (int j = 0; j < kTiles; ++j) {
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        total[j][i] += acc[j][i];
                                        acc[j][i] = 0.0f;
                                    }
                                }
                            }
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty[buffer]);
                    next_buffer();
                }
                close_group(group);                         // C may end inside it, or in front of others, which are 0
                if (group & 2) {
#pragma unroll
                    for (int j = 0; j < kTiles; ++j) {
                        if (8 * j >= p.R) break;
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            float2* const at = reinterpret_cast<float2*>(sums + 8 * r * lay.sum_pitch + 8 * j);
                            const float2 v = *at, w = *reinterpret_cast<const float2*>(sums2 + 8 * r * lay.sum_pitch + 8 * j);
                            *at = make_float2(v.x + w.x, v.y + w.y);
                        }
                    }
                }
                asm volatile("fence.acq_rel.cluster;" ::: "memory");
                consumer_barrier();
                if (threadIdx.x < split) cluster_arrive(cluster_addr(&sums_ready, threadIdx.x));
                // the CTA's share of the rows, 32 at a time, 8 lanes to one; where their h goes is read while the sums come (16 at a
                // time, and read then, 16384 x 4096 -> 4096 took 91 us instead of 88)
                const int share = kManyRows / split, row0 = share * rank, end_row = row0 + share;
                int h_row = 0;
                if (p.h != nullptr && lane < 8) {
                    const int r = row0 + 32 * (lane >> 2) + 4 * warp + (lane & 3);
                    if (r < min(end_row, rows)) h_row = p.tiles.perm[start + r];
                }
                if (!failed && !cluster_wait_bounded(&sums_ready, tile_phase, abort_flag, kWaitBudgetCycles)) failed = true;
#pragma unroll 1
                for (int pass = 0; row0 + 32 * pass < min(end_row, rows); ++pass) {
                    const int at_row = row0 + 32 * pass + 4 * warp + (lane >> 3);
                    const bool mine = at_row < end_row;
                    const int r = mine ? at_row : row0, to_row = __shfl_sync(kAll, h_row, 4 * pass + (lane >> 3));
                    const uint32_t to = smem_u32(smem) + lay.h + r * pitch;
                    const bool keep = p.h != nullptr && mine && r < rows;
                    float row_undo;
                    finish_row<T, kRank, 8>(reinterpret_cast<const float*>(smem + lay.sum), split, r, lay.sum_pitch, p.R,
                                            p.scale == nullptr ? 1.0f : p.scale[adapter], kTerms, kManyRows * pitch,
                                            keep ? p.h + static_cast<int64_t>(to_row) * p.R : nullptr, p.h_scaled != 0,
                                            lane & 7,
                                            [&](int at, uint32_t v) {
                                                if (!mine) return;
#pragma unroll
                                                for (int c = 0; c < kGroups; ++c) {
                                                    if (c >= split) break;
                                                    uint32_t there;
                                                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(to + at), "r"(c));
                                                    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(there), "r"(v) : "memory");
                                                }
                                            },
                                            row_undo);
                    if (mine && (lane & 7) < split)
                        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr(s_undo + r, lane & 7)), "f"(row_undo) : "memory");
                }
                asm volatile("fence.acq_rel.cluster;" ::: "memory");
                consumer_barrier();
                if (threadIdx.x < split) cluster_arrive(cluster_addr(&h_ready, threadIdx.x));
                if (!failed && !cluster_wait_bounded(&h_ready, tile_phase, abort_flag, kWaitBudgetCycles)) failed = true;
                tile_phase ^= 1;
            } else if (p.h != nullptr && rank == 0) {
                for (int i = threadIdx.x; i < rows * p.R; i += kThreads)
                    p.h[static_cast<int64_t>(p.tiles.perm[start + i / p.R]) * p.R + i % p.R] = 0.0f;
            }

            float undo[2] = {1.0f, 1.0f};
            if (std::is_same<T, __half>::value && adapter >= 0) {
                undo[0] = s_undo[my_row];
                undo[1] = s_undo[my_row + 8];
            }
            {
                // a lane's 2 outputs of 4 tiles of 8, in its two rows
                const int mine = my_row * 128 + (kWide ? (((lane >> 1) & 1) ^ quad) << 4 | 8 * (lane & 1) : quad << 4 | 4 * (lane & 3));
                const int line = swizzled(16 * warp + (lane >> 3), lane & 7);
                const int full_rows = kLoaders == 1 || p.out_wide ? min(max(rows - 16 * warp, 0), 16) : 0;
                for (int chunk = chunk0; chunk < chunk1; ++chunk) {
                    if (!failed && !mbar_wait_bounded(&full[buffer], phase, abort_flag, kWaitBudgetCycles)) failed = true;
                    uint4 v[4];
                    if (busy && !failed) {
                        uint8_t* y = smem + buffer * lay.stage;
                        const uint32_t part = smem_u32(y) + kManyRows * 128;
#pragma unroll
                        for (int g = 0; g < kCols / 32; ++g) {
                            if (adapter < 0 && p.y != nullptr) break;   // a row without one keeps its bits (-0 + 0 is +0)
                            // y where it lies; all read before any is written, which the compiler cannot do by itself
                            const auto at = [&](int i, int r) { return y + 1024 * r + (mine ^ (kWide ? i << 5 : (4 * g + i) << 4)); };
                            float2 was[4][2];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
#pragma unroll
                                for (int r = 0; r < 2; ++r) {
                                    if (kWide) was[i][r] = *reinterpret_cast<const float2*>(at(i, r));
                                    else was[i][r] = unpack2(*reinterpret_cast<const uint32_t*>(at(i, r)), kType);
                                    if (p.y == nullptr) was[i][r] = make_float2(0.0f, 0.0f);
                                }
                            }
                            float acc[4][4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
#pragma unroll
                                for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
                            }
                            if (adapter >= 0) {
#pragma unroll
                                for (int kk = 0; kk < kRank / 16; ++kk) {
                                    if (16 * kk >= p.R) break;
                                    // the rows' terms again for each stage: held over them they took the registers of the rest
                                    // (8191 rows of dx of rank 64 75 us instead of 62, 8192 rows of dx of 4096 -> 4096 of rank 32 73 instead of 63)
                                    uint32_t h_of[kTerms][4];
#pragma unroll
                                    for (int t = 0; t < kTerms; ++t) ldsm4(ha + t * kManyRows * pitch + 32 * kk, h_of[t]);
                                    multiply_outputs<T, kTrans, kTerms, kRankBytes>(acc, h_of, part + (kTrans ? 0 : 32 * kRankBytes * g), kCols * kRankBytes,
                                                                        4 * g, kk, lane);
                                }
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
#pragma unroll
                                for (int r = 0; r < 2; ++r) {
                                    float lo = acc[i][2 * r], hi = acc[i][2 * r + 1];
                                    if (std::is_same<T, __half>::value) lo *= undo[r], hi *= undo[r];
                                    lo += was[i][r].x, hi += was[i][r].y;
                                    if (kWide) *reinterpret_cast<float2*>(at(i, r)) = make_float2(lo, hi);
                                    else *reinterpret_cast<uint32_t*>(at(i, r)) = pack2(lo, hi, kType);
                                }
                            }
                        }
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint4*>(y + (line ^ (i & 1) << 6) + 512 * i);
                        fence_proxy_async_shared();         // this stage was written to; TMA writes it next
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty[buffer]);   // in front of the stores, which it would wait for
                    next_buffer();
                    const int there = busy && !failed ? min((p.D - chunk * kCols) * kUnits, 64) : 0, left = there - 8 * (lane & 7);   // units
                    if (full_rows == 16 && left >= 8) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) store_chunk<kTrans>(out[i], v[i]);
                    } else if (kLoaders == 1 || p.out_wide) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (out[i] == nullptr) continue;
                            if (left >= 8) store_chunk<kTrans>(out[i], v[i]);
                            else store_units(out[i], v[i], left, kUnits);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) store_unaligned<kUnits>(out[i], v[i], there, lane);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (out[i] != nullptr) out[i] += 128;
                    }
                }
            }
        }
        if (failed) {
            if (lane == 0) set_device_error(p.err, NVFP4_ERR_DEVICE_TIMEOUT);
            *abort_flag = 1;
        }
    }
    cluster_barrier();                                      // no CTA leaves while another may reach into it
}

template <typename T, bool kTrans, int kType, int kRank, int kLoaders>
cudaError_t launch_many_kernel(const ManyMaps& maps, const Params& p, const ManyLayout& lay, int64_t tiles, bool pdl, cudaStream_t st) {
    static Ready ready;
    auto* kernel = many_kernel<T, kTrans, kType, kRank, kLoaders>;
    cudaError_t e = allow_shared(reinterpret_cast<const void*>(kernel), kManyShared, ready);
    if (e != cudaSuccess) return e;
    // CTAs to a tile: rounds over the GPU (every other adapter taken to have a tile of its own) times a CTA's stages of a tile and
    // the pause between its two products (about as long as 4).  With 2, 4 and 8 16384 x 4096 -> 4096 of rank 16 took 98, 105 and
    // 117 us, 2000 x 2048 -> 1536 of rank 64 and 8 adapters 51, 33 and 40 (before the products were made shorter).
    int64_t clusters = 0, best = 0;                         // that run at once
    int split = 0;
    const int64_t half = (p.L < p.T ? p.L : p.T) / 2, full = (p.T / kManyRows > half ? p.T / kManyRows : half) + 1, stages = (p.C + 63) / 64 + (p.D + lay.cols - 1) / lay.cols;
    for (int n = 2; n <= kGroups; n *= 2) {
        int64_t at_once = 0;
        e = clusters_at_once(kernel, kThreads + 32 * kLoaders, lay.total, p.R, n, ready, at_once);
        if (e != cudaSuccess) return e;
        const int64_t cost = (full + at_once - 1) / at_once * ((stages + n - 1) / n + 4);
        if (split == 0 || cost < best) {
            split = n;
            best = cost;
            clusters = at_once;
        }
    }
    if (tiles < clusters) clusters = tiles;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * split));
    cfg.blockDim = dim3(kThreads + 32 * kLoaders);
    cfg.dynamicSmemBytes = static_cast<size_t>(lay.total);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(split);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, maps, p, lay);
}

template <typename T, bool kTrans, int kType>
cudaError_t launch_many(const Params& p, int64_t tiles, bool pdl, cudaStream_t st) {
    const int units = kType == NVFP4_TYPE_F32 ? 2 : 1, Rp = rank_up(p.R);
    const ManyLayout lay(p.R, terms_of<T>(kType), kTrans, kType);
    ManyMaps maps;
    const int rank_row = rank_bytes(p.R);
    bool ok = kTrans ? make_units_map(&maps.down, p.down, p.R, p.C, p.R, p.L, static_cast<int64_t>(p.C) * p.R, 64, rank_row)
                     : make_units_map(&maps.down, p.down, p.C, p.R, p.C, p.L, static_cast<int64_t>(p.C) * p.R, Rp);
    ok = ok && (kTrans ? make_units_map(&maps.up, p.up, p.D, p.R, p.D, p.L, static_cast<int64_t>(p.D) * p.R, Rp)
                       : make_units_map(&maps.up, p.up, p.R, p.D, p.R, p.L, static_cast<int64_t>(p.D) * p.R, lay.cols, rank_row));
    maps.y = maps.y16 = maps.up;        // what is not used is another's
    ok = ok && make_units_map(&maps.x, p.x, p.C, p.T, p.ldx, 0, 0, 1) && make_units_map(&maps.x16, p.x, p.C, p.T, p.ldx, 0, 0, 16);
    const int64_t row = static_cast<int64_t>(p.D) * units;
    if (ok && p.y != nullptr && p.y_wide)
        ok = make_units_map(&maps.y, p.y, row, p.T, p.ldy * units, 0, 0, 1) && make_units_map(&maps.y16, p.y, row, p.T, p.ldy * units, 0, 0, 16);
    if (!ok) return cudaErrorInvalidValue;
    return by_rank(p.R, [&](auto rank) {
        constexpr int kRank = decltype(rank)::value;
        return p.y_wide && p.out_wide ? launch_many_kernel<T, kTrans, kType, kRank, 1>(maps, p, lay, tiles, pdl, st)
                                      : launch_many_kernel<T, kTrans, kType, kRank, 4>(maps, p, lay, tiles, pdl, st);
    });
}

}  // namespace lora
}  // namespace nvfp4
