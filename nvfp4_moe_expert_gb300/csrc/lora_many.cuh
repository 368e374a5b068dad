// Low-rank adapters, tiles of up to 128 rows: prompts and training batches.  lora.cuh says what is computed.
//
// Bound by memory, so the loads are not to pause: loader warps keep a ring of stages full, first a tile's eighth of C (64
// columns of x and of the adapter a stage), then its eighth of D (128 bytes a row of y and the adapter's part), then the next
// tile's, whatever the 8 other warps are at.  Those take 16 rows each: products of the first phase into registers; the
// 8 CTAs' sums meet in shared memory over the cluster, each CTA adding 16 rows and handing their terms to all; products of the
// second phase are added to y where it lies in shared memory, which goes out from there in whole rows of 128 bytes.
//
// x and y come by TMA, 16 rows to an instruction where they lie in a row, four rows of any place otherwise, where
// rows start on 16-byte boundaries; otherwise four loader warps read aligned words and shift them together.  (With the loads
// and the products in the same warps, cp.async and a barrier for each stage, 16384 x 4096 -> 4096 of rank 16 took 145 to 199 us:
// 500 instructions a stage and warp, half of them addresses.)
#pragma once

#include "lora_launch.cuh"

namespace nvfp4 {
namespace lora {

// Four rows (`at[i]`) of 64 units from column c on, one behind the other in shared memory.
__device__ __forceinline__ void gather4(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c, const int (&at)[4]) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c), "r"(at[0]), "r"(at[1]), "r"(at[2]), "r"(at[3]), "r"(bar)
        : "memory");
}
// Sixteen rows from `row` on.
__device__ __forceinline__ void load_rows16(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c, int row) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(c), "r"(row), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c, int row, int slice) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(c), "r"(row), "r"(slice), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void consumer_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

struct ManyMaps {
    CUtensorMap x, y, x16, y16, down, up;   // of x and y: boxes of one row, for gathers, and of 16
};

// The second product of a warp's 16 rows with a group of 32 outputs (`up`: the group's rows, or columns): acc[i] gets
// outputs 8 i to 8 i + 7.
template <typename T, bool kTrans, int kTerms>
__device__ __forceinline__ void multiply_outputs(float (&acc)[4][4], uint32_t h, int term_bytes, uint32_t up, int block_bytes,
                                                 int first_chunk, int Rp, int lane) {
#pragma unroll 1
    for (int kk = 0; kk < Rp / 16; ++kk) {
        uint32_t a[kTerms][4], b[2][4];
#pragma unroll
        for (int t = 0; t < kTerms; ++t) ldsm4(h + t * term_bytes + 32 * kk, a[t]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {     // two tiles of 8 outputs at once
            if (!kTrans)                  // rows of 64 ranks
                ldsm4(up + (kk >> 2) * block_bytes + swizzled(8 * (2 * i + (lane >> 4)) + (lane & 7), 2 * (kk & 3) + ((lane >> 3) & 1)), b[i]);
            else                          // rows of 64 outputs
                ldsm4_trans(up + swizzled(16 * kk + ((lane >> 3) & 1) * 8 + (lane & 7), first_chunk + 2 * i + (lane >> 4)), b[i]);
        }
#pragma unroll
        for (int t = 0; t < kTerms; ++t) {
#pragma unroll
            for (int i = 0; i < 4; ++i) mma(T(), acc[i], a[t], b[i >> 1][2 * (i & 1)], b[i >> 1][2 * (i & 1) + 1]);
        }
    }
}

// kLoaders: warps that load, 1 (x and y by TMA) or 4.  kType: y's and out's (branches by it for every value took 3000 cycles a stage).
template <typename T, bool kTrans, int kType, int kRank, int kLoaders>
__global__ void __cluster_dims__(kSplit, 1, 1) __launch_bounds__(kThreads + 32 * kLoaders, kRank <= 32 && kLoaders == 1 ? 2 : 1)
    many_kernel(const __grid_constant__ ManyMaps maps, const Params p, const ManyLayout lay) {
    constexpr int kTiles = kRank / 8;
    constexpr bool kWide = kType == NVFP4_TYPE_F32;
    constexpr int kCols = kWide ? 32 : 64, kUnits = kWide ? 2 : 1;   // outputs of a stage; 16-bit units of an output
    constexpr int kTerms = terms_of<T>(kType);
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], sums_ready, h_ready;
    __shared__ float s_undo[kManyRows];
    __shared__ int abort_word;
    volatile int* abort_flag = &abort_word;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t base = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_rank());
    const int steps = sub_steps(p.C), c0 = min(rank * kWarps * steps * 16, p.C), c1 = min(c0 + kWarps * steps * 16, p.C);
    const int chunks = (p.D + kCols - 1) / kCols, per_cta = (chunks + kSplit - 1) / kSplit;
    const int chunk0 = min(rank * per_cta, chunks), chunk1 = min(chunk0 + per_cta, chunks);
    if (threadIdx.x == 0) {
        for (int s = 0; s < lay.stages; ++s) {
            mbar_init(&full[s], kLoaders == 1 ? 1 : 32 * kLoaders);
            mbar_init(&empty[s], kWarps);
        }
        mbar_init(&sums_ready, kSplit);
        mbar_init(&h_ready, kSplit);
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
        const bool x_tma = kLoaders == 1 || p.x_wide, y_tma = kLoaders == 1 || p.out_wide;
        int issued = 0;
        for (int q = blockIdx.x / kSplit; q < count; q += gridDim.x / kSplit) {
            const int adapter = p.tiles.adapter[q], start = p.tiles.start[q];
            const int rows = min(kManyRows, p.tiles.offsets[(adapter < 0 ? p.L : adapter) + 1] - start);
            if (adapter < 0 && p.skip_none) continue;
            const int x_stages = adapter < 0 ? 0 : (c1 - c0 + 63) / 64, all = x_stages + chunk1 - chunk0;
            // TMA: a lane's four rows (behind the last: outside the tensor, zeros); otherwise a thread's chunk of every 16th row
            constexpr int kMine = kLoaders == 1 ? 4 : 8;
            int row[kMine];
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
            if (kLoaders > 1) {
#pragma unroll
                for (int i = 0; i < kMine; ++i) {
                    const int r = (thread >> 3) + 16 * i;
                    row[i] = r < rows ? p.tiles.perm[start + r] : -1;
                }
            }
            for (int s = 0; s < all; ++s, ++issued) {
                if (!mbar_wait_bounded(&empty[buffer], phase ^ 1u, abort_flag, kWaitBudgetCycles)) failed = true;
                if (__any_sync(kAll, failed)) break;
                const uint32_t at = base + buffer * lay.stage, part = at + kManyRows * 128, bar = smem_u32(&full[buffer]);
                const bool is_x = s < x_stages, tma = is_x ? x_tma : y_tma, none = !is_x && p.y == nullptr;
                const int c = is_x ? c0 + 64 * s : (chunk0 + s - x_stages) * kCols;
                if (kLoaders > 1) fence_proxy_async_shared();
                if (thread == 0) {
                    const int bytes = (adapter < 0 ? 0 : is_x ? lay.down_bytes : lay.up_bytes) + (tma && !none ? (rows + 15) / 16 * 2048 : 0);
                    mbar_arrive_expect_tx(&full[buffer], bytes);
                    if (adapter >= 0 && is_x) {
                        if (!kTrans) load_box(part, &maps.down, bar, c, 0, adapter);
                        else for (int b = 0; b < lay.blocks; ++b) load_box(part + b * 64 * 128, &maps.down, bar, 64 * b, c, adapter);
                    } else if (adapter >= 0) {
                        if (kTrans) load_box(part, &maps.up, bar, c, 0, adapter);
                        else for (int b = 0; b < lay.blocks; ++b) load_box(part + b * kCols * 128, &maps.up, bar, 64 * b, c, adapter);
                    }
                }
                __syncwarp();
                if (tma && !none && group) {
                    if (box) load_rows16(at + 512 * lane, is_x ? &maps.x16 : &maps.y16, bar, is_x ? c : c * kUnits, group_row);
                    else gather4(at + 512 * lane, is_x ? &maps.x : &maps.y, bar, is_x ? c : c * kUnits, four);
                }
                if (kLoaders > 1) {
                    if (!tma && !none) {
                        const uint16_t* from = static_cast<const uint16_t*>(is_x ? p.x : p.y);
                        const int64_t ld = is_x ? p.ldx : p.ldy * kUnits;
                        const int unit = (is_x ? c : c * kUnits) + 8 * (thread & 7), there = is_x ? p.C : p.D * kUnits;
#pragma unroll
                        for (int i = 0; i < kMine; i += 4) {
                            Straddle w[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                if (row[i + j] >= 0) w[j].load(from + row[i + j] * ld, unit, there);
                            }
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                if (row[i + j] >= 0) w[j].store(at + swizzled((thread >> 3) + 16 * (i + j), thread & 7));
                            }
                        }
                    }
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
        for (int q = blockIdx.x / kSplit; q < count; q += gridDim.x / kSplit) {
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
                int left = steps;                           // of the sub-slice
                for (int s = 0; s < x_stages; ++s) {
                    if (!failed && !mbar_wait_bounded(&full[buffer], phase, abort_flag, kWaitBudgetCycles)) failed = true;
                    if (busy) {
                        const uint32_t at = base + buffer * lay.stage, sx = at + 2048 * warp + lane_rows(lane);
                        const uint32_t sd = at + kManyRows * 128 +
                                            (kTrans ? swizzled(((lane >> 3) & 1) * 8 + (lane & 7), lane >> 4) : lane_down<false>(lane, p.R));
                        const int n = min(4, (c1 - c0 - 64 * s + 15) / 16);
                        uint32_t a[4][4];
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) ldsm4(sx ^ (kk << 5), a[kk]);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            if (kk >= n) break;
                            if (!kTrans) {
                                multiply_down<T, false, kTiles>(acc, a[kk], sd, kk, p.R);
                            } else {                        // rows of 64 ranks, 16 to a step
#pragma unroll
                                for (int j = 0; j < kTiles; j += 2) {
                                    if (8 * j >= p.R) break;
                                    uint32_t b[4];
                                    ldsm4_trans((sd ^ ((j & 7) << 4)) + (j >> 3) * 64 * 128 + 2048 * kk, b);
                                    mma(T(), acc[j], a[kk], b[0], b[1]);
                                    if (8 * (j + 1) < p.R) mma(T(), acc[j + 1], a[kk], b[2], b[3]);
                                }
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
                float* sum = reinterpret_cast<float*>(smem + lay.sum) + my_row * lay.sum_pitch + 2 * (lane & 3);
#pragma unroll
                for (int j = 0; j < kTiles; ++j) {
                    if (8 * j >= p.R) break;
#pragma unroll
                    for (int i = 0; i < 4; ++i) total[j][i] += acc[j][i];   // C ends inside a sub-slice, or 0
                    *reinterpret_cast<float2*>(sum + 8 * j) = make_float2(total[j][0], total[j][1]);
                    *reinterpret_cast<float2*>(sum + 8 * j + 8 * lay.sum_pitch) = make_float2(total[j][2], total[j][3]);
                }
                asm volatile("fence.acq_rel.cluster;" ::: "memory");
                consumer_barrier();
                if (threadIdx.x < kSplit) cluster_arrive(cluster_addr(&sums_ready, threadIdx.x));
                if (!failed && !cluster_wait_bounded(&sums_ready, tile_phase, abort_flag, kWaitBudgetCycles)) failed = true;
                if (16 * rank < rows) {
                    const int r = 16 * rank + 2 * warp + (lane >> 4);
                    const uint32_t to = smem_u32(smem) + lay.h + r * pitch;
                    const bool keep = p.h != nullptr && r < rows;
                    float row_undo;
                    finish_row<T, kRank>(reinterpret_cast<const float*>(smem + lay.sum), r, lay.sum_pitch, p.R,
                                         p.scale == nullptr ? 1.0f : p.scale[adapter], kTerms, kManyRows * pitch,
                                         keep ? p.h + static_cast<int64_t>(p.tiles.perm[start + r]) * p.R : nullptr, p.h_scaled != 0,
                                         lane & 15,
                                         [&](int at, uint32_t v) {
#pragma unroll
                                             for (int c = 0; c < kSplit; ++c) {
                                                 uint32_t there;
                                                 asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(to + at), "r"(c));
                                                 asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(there), "r"(v) : "memory");
                                             }
                                         },
                                         row_undo);
                    if ((lane & 15) < kSplit)
                        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr(s_undo + r, lane & 15)), "f"(row_undo) : "memory");
                }
                asm volatile("fence.acq_rel.cluster;" ::: "memory");
                consumer_barrier();
                if (threadIdx.x < kSplit) cluster_arrive(cluster_addr(&h_ready, threadIdx.x));
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
                const int full_rows = p.out_wide ? min(max(rows - 16 * warp, 0), 16) : 0;
                for (int chunk = chunk0; chunk < chunk1; ++chunk) {
                    if (!failed && !mbar_wait_bounded(&full[buffer], phase, abort_flag, kWaitBudgetCycles)) failed = true;
                    uint4 v[4];
                    if (busy && !failed) {
                        uint8_t* y = smem + buffer * lay.stage;
                        const uint32_t part = smem_u32(y) + kManyRows * 128;
#pragma unroll
                        for (int g = 0; g < kCols / 32; ++g) {
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
                            if (adapter >= 0)
                                multiply_outputs<T, kTrans, kTerms>(acc, ha, kManyRows * pitch, part + (kTrans ? 0 : 4096 * g), kCols * 128, 4 * g,
                                                                    rank_up(p.R), lane);
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
                    const int left = busy && !failed ? (p.D - chunk * kCols) * kUnits - 8 * (lane & 7) : 0;   // units of the row from the lane's on
                    if (full_rows == 16 && left >= 8) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(out[i]) = v[i];
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (out[i] == nullptr || left <= 0) continue;
                            if (p.out_wide && left >= 8) {
                                *reinterpret_cast<uint4*>(out[i]) = v[i];
                                continue;
                            }
                            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                if (kWide) {
                                    if (2 * j < left) reinterpret_cast<uint32_t*>(out[i])[j] = w[j];
                                } else {
                                    if (2 * j < left) reinterpret_cast<uint16_t*>(out[i])[2 * j] = static_cast<uint16_t>(w[j]);
                                    if (2 * j + 1 < left) reinterpret_cast<uint16_t*>(out[i])[2 * j + 1] = static_cast<uint16_t>(w[j] >> 16);
                                }
                            }
                        }
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
    __syncwarp();
    cluster_barrier();                                      // no CTA leaves while another may reach into it
}

template <typename T, bool kTrans, int kType, int kRank, int kLoaders>
cudaError_t launch_many_kernel(const ManyMaps& maps, const Params& p, const ManyLayout& lay, int64_t tiles, bool pdl, cudaStream_t st) {
    static Ready ready;
    auto* kernel = many_kernel<T, kTrans, kType, kRank, kLoaders>;
    cudaError_t e = allow_shared(reinterpret_cast<const void*>(kernel), kManyShared, ready);
    if (e != cudaSuccess) return e;
    int64_t clusters = 0;                                   // that run at once
    e = clusters_at_once(kernel, kThreads + 32 * kLoaders, lay.total, p.R, ready, clusters);
    if (e != cudaSuccess) return e;
    if (tiles < clusters) clusters = tiles;
    return launch_pdl(pdl, kernel, dim3(static_cast<unsigned>(clusters * kSplit)), dim3(kThreads + 32 * kLoaders),
                      static_cast<size_t>(lay.total), st, maps, p, lay);
}

template <typename T, bool kTrans, int kType>
cudaError_t launch_many(const Params& p, int64_t tiles, bool pdl, cudaStream_t st) {
    const int units = kType == NVFP4_TYPE_F32 ? 2 : 1, Rp = rank_up(p.R);
    const ManyLayout lay(p.R, terms_of<T>(kType), kTrans, kType);
    const bool tma_y = p.y != nullptr && p.out_wide;
    ManyMaps maps;
    bool ok = kTrans ? make_units_map(&maps.down, p.down, p.R, p.C, p.R, p.L, static_cast<int64_t>(p.C) * p.R, 64)
                     : make_units_map(&maps.down, p.down, p.C, p.R, p.C, p.L, static_cast<int64_t>(p.C) * p.R, Rp);
    ok = ok && (kTrans ? make_units_map(&maps.up, p.up, p.D, p.R, p.D, p.L, static_cast<int64_t>(p.D) * p.R, Rp)
                       : make_units_map(&maps.up, p.up, p.R, p.D, p.R, p.L, static_cast<int64_t>(p.D) * p.R, lay.cols));
    maps.x = maps.y = maps.x16 = maps.y16 = maps.up;        // what is not used is another's
    if (ok && p.x_wide)
        ok = make_units_map(&maps.x, p.x, p.C, p.T, p.ldx, 0, 0, 1) && make_units_map(&maps.x16, p.x, p.C, p.T, p.ldx, 0, 0, 16);
    const int64_t row = static_cast<int64_t>(p.D) * units;
    if (ok && tma_y)
        ok = make_units_map(&maps.y, p.y, row, p.T, p.ldy * units, 0, 0, 1) && make_units_map(&maps.y16, p.y, row, p.T, p.ldy * units, 0, 0, 16);
    if (!ok) return cudaErrorInvalidValue;
    const bool one = p.x_wide && (tma_y || p.y == nullptr);
    return by_rank(p.R, [&](auto rank) {
        constexpr int kRank = decltype(rank)::value;
        return one ? launch_many_kernel<T, kTrans, kType, kRank, 1>(maps, p, lay, tiles, pdl, st)
                   : launch_many_kernel<T, kTrans, kType, kRank, 4>(maps, p, lay, tiles, pdl, st);
    });
}

}  // namespace lora
}  // namespace nvfp4
