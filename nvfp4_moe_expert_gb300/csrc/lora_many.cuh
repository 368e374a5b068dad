// Low-rank adapters, tiles of up to 128 rows: prompts and training batches.  lora.cuh says what is computed.
//
// Bound by memory, so the loads are not to pause: loader warps keep a ring of stages full, first a tile's eighth of C (64
// columns of x and of the adapter a stage), then its eighth of D (128 bytes a row of y and the adapter's part), then the next
// tile's, whatever the 8 other warps are at.  Those take 16 rows each: products of the first phase into registers; the
// 8 CTAs' sums meet in shared memory over the cluster, each CTA adding 16 rows and handing their terms to all; products of the
// second phase are added to y where it lies in shared memory, which goes out from there in whole rows of 128 bytes.
//
// x and y come by TMA, four rows of any place to an instruction (their tile's rows lie where the sort found them), where
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
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c, int row, int slice) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(c), "r"(row), "r"(slice), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void consumer_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

struct ManyMaps {
    CUtensorMap x, y, down, up;
};

// The second product of a warp's 16 rows with a group of 32 outputs (`up`: the group's rows, or columns): acc[i] gets
// outputs 8 i to 8 i + 7.
template <typename T, bool kTrans>
__device__ __forceinline__ void multiply_outputs(float (&acc)[4][4], uint32_t h, int term_bytes, int terms, uint32_t up, int block_bytes,
                                                 int first_chunk, int Rp, int lane) {
    for (int kk = 0; kk < Rp / 16; ++kk) {
        uint32_t b[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {     // two tiles of 8 outputs at once
            if (!kTrans)                  // rows of 64 ranks
                ldsm4(up + (kk >> 2) * block_bytes + swizzled(8 * (2 * i + (lane >> 4)) + (lane & 7), 2 * (kk & 3) + ((lane >> 3) & 1)), b[i]);
            else                          // rows of 64 outputs
                ldsm4_trans(up + swizzled(16 * kk + ((lane >> 3) & 1) * 8 + (lane & 7), first_chunk + 2 * i + (lane >> 4)), b[i]);
        }
        for (int t = 0; t < terms; ++t) {
            uint32_t a[4];
            ldsm4(h + t * term_bytes + 32 * kk, a);
#pragma unroll
            for (int i = 0; i < 4; ++i) mma(T(), acc[i], a, b[i >> 1][2 * (i & 1)], b[i >> 1][2 * (i & 1) + 1]);
        }
    }
}

// kLoaders: warps that load, 1 (x and y by TMA) or 4.
template <typename T, bool kTrans, int kRank, int kLoaders>
__global__ void __cluster_dims__(kSplit, 1, 1) __launch_bounds__(kThreads + 32 * kLoaders, kRank <= 32 && kLoaders == 1 ? 2 : 1)
    many_kernel(const __grid_constant__ ManyMaps maps, const Params p, const ManyLayout lay, const int terms) {
    constexpr int kTiles = kRank / 8;
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
    const int chunks = (p.D + lay.cols - 1) / lay.cols, per_cta = (chunks + kSplit - 1) / kSplit;
    const int chunk0 = min(rank * per_cta, chunks), chunk1 = min(chunk0 + per_cta, chunks);
    const int units = p.y_type == NVFP4_TYPE_F32 ? 2 : 1;   // 16-bit units of an output
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
        prefetch_tensormap(&maps.x);
        prefetch_tensormap(&maps.y);
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
            const bool group = 4 * lane < rows && warp == kWarps;
            int four[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) four[i] = 4 * lane + i < rows ? p.tiles.perm[start + 4 * lane + i] : p.T;
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
                const int c = is_x ? c0 + 64 * s : (chunk0 + s - x_stages) * lay.cols;
                if (kLoaders > 1) fence_proxy_async_shared();
                if (thread == 0) {
                    const int bytes = (adapter < 0 ? 0 : is_x ? lay.down_bytes : lay.up_bytes) + (tma && !none ? (rows + 3) / 4 * 512 : 0);
                    mbar_arrive_expect_tx(&full[buffer], bytes);
                    if (adapter >= 0 && is_x) {
                        if (!kTrans) load_box(part, &maps.down, bar, c, 0, adapter);
                        else for (int b = 0; b < lay.blocks; ++b) load_box(part + b * 64 * 128, &maps.down, bar, 64 * b, c, adapter);
                    } else if (adapter >= 0) {
                        if (kTrans) load_box(part, &maps.up, bar, c, 0, adapter);
                        else for (int b = 0; b < lay.blocks; ++b) load_box(part + b * lay.cols * 128, &maps.up, bar, 64 * b, c, adapter);
                    }
                }
                __syncwarp();
                if (tma && !none && group) gather4(at + 512 * lane, is_x ? &maps.x : &maps.y, bar, is_x ? c : c * units, four);
                if (kLoaders > 1) {
                    if (!tma && !none) {
                        const uint16_t* from = static_cast<const uint16_t*>(is_x ? p.x : p.y);
                        const int64_t ld = is_x ? p.ldx : p.ldy * units;
                        const int unit = (is_x ? c : c * units) + 8 * (thread & 7), there = is_x ? p.C : p.D * units;
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
                out[i] = r < rows ? static_cast<uint8_t*>(p.out) + (p.tiles.perm[start + r] * p.ldo + chunk0 * lay.cols) * (2 * units) + 16 * (lane & 7)
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
#pragma unroll 1
                        for (int kk = 0; kk < n; ++kk) {
                            uint32_t a[4];
                            ldsm4(sx ^ (kk << 5), a);
                            if (!kTrans) {
                                multiply_down<T, false, kTiles>(acc, a, sd, kk, p.R);
                            } else {                        // rows of 64 ranks, 16 to a step
#pragma unroll
                                for (int j = 0; j < kTiles; j += 2) {
                                    if (8 * j >= p.R) break;
                                    uint32_t b[4];
                                    ldsm4_trans((sd ^ ((j & 7) << 4)) + (j >> 3) * 64 * 128 + 2048 * kk, b);
                                    mma(T(), acc[j], a, b[0], b[1]);
                                    if (8 * (j + 1) < p.R) mma(T(), acc[j + 1], a, b[2], b[3]);
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
                                         p.scale == nullptr ? 1.0f : p.scale[adapter], terms, kManyRows * pitch,
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
            for (int chunk = chunk0; chunk < chunk1; ++chunk) {
                if (!failed && !mbar_wait_bounded(&full[buffer], phase, abort_flag, kWaitBudgetCycles)) failed = true;
                if (busy && !failed) {
                    const uint32_t at = base + buffer * lay.stage, part = at + kManyRows * 128;
#pragma unroll 1
                    for (int g = 0; 32 * g < lay.cols; ++g) {
                        float acc[4][4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
                        }
                        if (adapter >= 0)
                            multiply_outputs<T, kTrans>(acc, ha, kManyRows * pitch, terms, part + (kTrans ? 0 : 4096 * g), lay.cols * 128, 4 * g,
                                                        rank_up(p.R), lane);
                        // y where it lies: a lane's 2 outputs of 4 tiles of 8, in its two rows
                        uint8_t* y = smem + buffer * lay.stage + my_row * 128;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                float lo = acc[i][2 * r], hi = acc[i][2 * r + 1];
                                if (std::is_same<T, __half>::value) lo *= undo[r], hi *= undo[r];
                                if (units == 2) {
                                    float2* to = reinterpret_cast<float2*>(y + 1024 * r + (((2 * i + ((lane >> 1) & 1)) ^ quad) << 4) + 8 * (lane & 1));
                                    const float2 was = p.y == nullptr ? make_float2(0.0f, 0.0f) : *to;
                                    *to = make_float2(was.x + lo, was.y + hi);
                                } else {
                                    uint32_t* to = reinterpret_cast<uint32_t*>(y + 1024 * r + (((4 * g + i) ^ quad) << 4) + 4 * (lane & 3));
                                    const uint32_t was = p.y == nullptr ? 0u : *to;
                                    *to = p.y_type == NVFP4_TYPE_BF16 ? add2_bf16(was, lo, hi) : add2_f16(was, lo, hi);
                                }
                            }
                        }
                    }
                    __syncwarp();
                    const int left = (p.D - chunk * lay.cols) * units - 8 * (lane & 7);   // units of the row from the lane's on
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (out[i] == nullptr || left <= 0) continue;
                        const uint4 v = *reinterpret_cast<const uint4*>(smem + buffer * lay.stage + swizzled(16 * warp + (lane >> 3) + 4 * i, lane & 7));
                        if (p.out_wide && left >= 8) {
                            *reinterpret_cast<uint4*>(out[i]) = v;
                        } else {
                            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                if (units == 2) {
                                    if (2 * j < left) reinterpret_cast<uint32_t*>(out[i])[j] = w[j];
                                } else {
                                    if (2 * j < left) reinterpret_cast<uint16_t*>(out[i])[2 * j] = static_cast<uint16_t>(w[j]);
                                    if (2 * j + 1 < left) reinterpret_cast<uint16_t*>(out[i])[2 * j + 1] = static_cast<uint16_t>(w[j] >> 16);
                                }
                            }
                        }
                    }
                    fence_proxy_async_shared();             // this stage was written to; TMA writes it next
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (out[i] != nullptr) out[i] += 128;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[buffer]);
                next_buffer();
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

template <typename T, bool kTrans, int kRank, int kLoaders>
cudaError_t launch_many(const ManyMaps& maps, const Params& p, const ManyLayout& lay, int terms, int64_t tiles, bool pdl, cudaStream_t st) {
    static Ready ready;
    auto* kernel = many_kernel<T, kTrans, kRank, kLoaders>;
    cudaError_t e = allow_shared(reinterpret_cast<const void*>(kernel), kManyShared, ready);
    if (e != cudaSuccess) return e;
    int64_t clusters = 0;                                   // that run at once
    e = clusters_at_once(kernel, kThreads + 32 * kLoaders, lay.total, p.R, p.y_type == NVFP4_TYPE_F32, ready, clusters);
    if (e != cudaSuccess) return e;
    if (tiles < clusters) clusters = tiles;
    return launch_pdl(pdl, kernel, dim3(static_cast<unsigned>(clusters * kSplit)), dim3(kThreads + 32 * kLoaders),
                      static_cast<size_t>(lay.total), st, maps, p, lay, terms);
}

template <typename T, bool kTrans>
cudaError_t launch_many(const Params& p, int64_t tiles, bool pdl, cudaStream_t st) {
    const int terms = terms_of<T>(p.y_type), units = p.y_type == NVFP4_TYPE_F32 ? 2 : 1, Rp = rank_up(p.R);
    const ManyLayout lay(p.R, terms, kTrans, p.y_type);
    const bool tma_y = p.y != nullptr && p.out_wide;
    ManyMaps maps;
    // what is not used is x's map again
    bool ok = kTrans ? make_units_map(&maps.down, p.down, p.R, p.C, p.R, p.L, static_cast<int64_t>(p.C) * p.R, 64)
                     : make_units_map(&maps.down, p.down, p.C, p.R, p.C, p.L, static_cast<int64_t>(p.C) * p.R, Rp);
    ok = ok && (kTrans ? make_units_map(&maps.up, p.up, p.D, p.R, p.D, p.L, static_cast<int64_t>(p.D) * p.R, Rp)
                       : make_units_map(&maps.up, p.up, p.R, p.D, p.R, p.L, static_cast<int64_t>(p.D) * p.R, lay.cols));
    maps.x = maps.y = maps.up;
    if (ok && p.x_wide) ok = make_units_map(&maps.x, p.x, p.C, p.T, p.ldx, 0, 0, 1);
    if (ok && tma_y) ok = make_units_map(&maps.y, p.y, static_cast<int64_t>(p.D) * units, p.T, p.ldy * units, 0, 0, 1);
    if (!ok) return cudaErrorInvalidValue;
    const bool one = p.x_wide && (tma_y || p.y == nullptr);
    return by_rank(p.R, [&](auto rank) {
        constexpr int kRank = decltype(rank)::value;
        return one ? launch_many<T, kTrans, kRank, 1>(maps, p, lay, terms, tiles, pdl, st)
                   : launch_many<T, kTrans, kRank, 4>(maps, p, lay, terms, tiles, pdl, st);
    });
}

}  // namespace lora
}  // namespace nvfp4
