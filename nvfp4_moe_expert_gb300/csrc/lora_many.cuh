// Low-rank adapters, tiles of up to 128 rows: prompts and training batches.  lora.cuh says what is computed.
//
// A CTA streams its eighth of C (128 rows x 64 columns and the adapter's columns a stage) through shared memory, a warp
// taking 16 rows; the 8 CTAs' sums meet in shared memory over the cluster (each CTA adds 16 rows and hands their terms to
// all), and each CTA adds its eighth of D to y, read and written straight from the accumulators' lanes, 64 bytes and more
// of a row at a time.
#pragma once

#include "lora_launch.cuh"

namespace nvfp4 {
namespace lora {

constexpr int kStages = 3;

template <bool kTrans>
struct ManyLayout {
    int down_at, stage;                   // of a stage: the adapter's columns behind x's, all bytes
    int pitch, h, up, total;              // floats of a row of the sums; offsets of h's terms and of the second operand
    int up_size;
    __host__ __device__ explicit ManyLayout(int R, int terms) {
        down_at = kManyRows * 128;
        stage = down_at + (down_bytes<kTrans>(R, 64) + 127) / 128 * 128;
        pitch = R + 4;
        h = kManyRows * pitch * 4;        // the sums and h's terms lie over the stages, which are used up then
        const int end = h + terms * kManyRows * padded_pitch(rank_up(R));
        up = ((end > kStages * stage ? end : kStages * stage) + 127) / 128 * 128;
        up_size = (up_bytes<kTrans, 64>(R) + 127) / 128 * 128;
        total = up + 2 * up_size;
    }
};

template <typename T, bool kTrans, int kRank>
__global__ void __cluster_dims__(kSplit, 1, 1) __launch_bounds__(kThreads, kRank <= 64 ? 2 : 1)
    many_kernel(const Params p, const int terms) {
    constexpr int kTiles = kRank / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_row[kManyRows];
    __shared__ float s_undo[kManyRows];
    const ManyLayout<kTrans> lay(p.R, terms);
    const uint32_t base = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane >> 2;
    const int rank = static_cast<int>(cluster_rank());
    const int steps = sub_steps(p.C), c0 = min(rank * kWarps * steps * 16, p.C), c1 = min(c0 + kWarps * steps * 16, p.C);
    const int chunks = (p.D + 63) / 64, per_cta = (chunks + kSplit - 1) / kSplit;
    const int chunk0 = rank * per_cta, chunk1 = min(chunk0 + per_cta, chunks);
    pdl_wait();
    const int count = *p.tiles.count;

    for (int q = blockIdx.x / kSplit; q < count; q += gridDim.x / kSplit) {
        const int adapter = p.tiles.adapter[q], start = p.tiles.start[q];
        const int rows = min(kManyRows, p.tiles.offsets[(adapter < 0 ? p.L : adapter) + 1] - start);
        if (adapter < 0 && p.skip_none) continue;
        __syncthreads();                                    // the last tile's buffers are used up
        if (threadIdx.x < kManyRows) s_row[threadIdx.x] = static_cast<int>(threadIdx.x) < rows ? p.tiles.perm[start + threadIdx.x] : -1;
        __syncthreads();
        const int row_of[2] = {s_row[16 * warp + quad], s_row[16 * warp + quad + 8]};
        const uint16_t* up = static_cast<const uint16_t*>(p.up) + static_cast<int64_t>(max(adapter, 0)) * p.D * p.R;
        const auto load_up_chunk = [&](int c) {
            if (c < chunk1) load_up<kTrans, 64>(base + lay.up + ((c - chunk0) & 1) * lay.up_size, up, p.R, p.D, 64 * c, threadIdx.x, kThreads);
            cp_commit();
        };
        float undo[2] = {1.0f, 1.0f};
        if (adapter >= 0) {
            const uint16_t* down = static_cast<const uint16_t*>(p.down) + static_cast<int64_t>(adapter) * p.C * p.R;
            const int stages = (c1 - c0 + 63) / 64, chunk = threadIdx.x & 7;
            const uint16_t* from[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = s_row[(threadIdx.x >> 3) + 32 * i];
                from[i] = t < 0 ? nullptr : static_cast<const uint16_t*>(p.x) + t * p.ldx;
            }
            const auto load_stage = [&](int s) {
                if (s < stages) {
                    const uint32_t at = base + s % kStages * lay.stage;
                    const int c = c0 + 64 * s;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (from[i] != nullptr) copy_chunk(at + swizzled((threadIdx.x >> 3) + 32 * i, chunk), from[i], c + 8 * chunk, p.C, p.x_wide);
                    }
                    load_down<kTrans>(at + lay.down_at, down, p.R, p.C, c, 64, threadIdx.x, kThreads);
                }
                cp_commit();
            };
            float acc[kTiles][4], total[kTiles][4];
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][i] = total[j][i] = 0.0f;
            }
            int left = steps;                               // of the sub-slice
            for (int s = 0; s < kStages - 1; ++s) load_stage(s);
            for (int s = 0; s < stages; ++s) {
                cp_wait<kStages - 2>();
                __syncthreads();
                load_stage(s + kStages - 1);
                if (16 * warp >= rows) continue;
                const uint32_t sx = base + s % kStages * lay.stage;
                const int n = min(4, (c1 - c0 - 64 * s + 15) / 16);
                for (int kk = 0; kk < n; ++kk) {
                    uint32_t a[4];
                    ldsm4(sx + swizzled(16 * warp + (lane & 7) + ((lane >> 3) & 1) * 8, 2 * kk + (lane >> 4)), a);
                    multiply_down<T, kTrans, kTiles>(acc, a, sx + lay.down_at, kk, p.R, lane);
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
            cp_wait<0>();
            __syncthreads();
            load_up_chunk(chunk0);
            load_up_chunk(chunk0 + 1);
            float* sum = reinterpret_cast<float*>(smem) + (16 * warp + quad) * lay.pitch + 2 * (lane & 3);
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
                if (8 * j >= p.R) break;
#pragma unroll
                for (int i = 0; i < 4; ++i) total[j][i] += acc[j][i];   // C ends inside a sub-slice, or 0
                *reinterpret_cast<float2*>(sum + 8 * j) = make_float2(total[j][0], total[j][1]);
                *reinterpret_cast<float2*>(sum + 8 * j + 8 * lay.pitch) = make_float2(total[j][2], total[j][3]);
            }
            cluster_barrier();
            {
                const int row = 16 * rank + 2 * warp + (lane >> 4), pitch = padded_pitch(rank_up(p.R));
                uint32_t to[kSplit];
#pragma unroll
                for (int c = 0; c < kSplit; ++c) to[c] = cluster_addr(smem, c) + lay.h + row * pitch;
                const bool keep = p.h != nullptr && row < rows;
                float row_undo;
                finish_row<T, kRank>(reinterpret_cast<const float*>(smem), row, lay.pitch, p.R,
                                     p.scale == nullptr ? 1.0f : p.scale[adapter], terms, kManyRows * pitch,
                                     keep ? p.h + static_cast<int64_t>(s_row[row]) * p.R : nullptr, p.h_scaled != 0, lane & 15,
                                     [&](int at, uint16_t v) {
#pragma unroll
                                         for (int c = 0; c < kSplit; ++c)
                                             asm volatile("st.shared::cluster.u16 [%0], %1;" ::"r"(to[c] + at), "h"(v) : "memory");
                                     },
                                     row_undo);
                if ((lane & 15) < kSplit)
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr(s_undo + row, lane & 15)), "f"(row_undo) : "memory");
            }
            cluster_barrier();
            undo[0] = s_undo[16 * warp + quad];
            undo[1] = s_undo[16 * warp + quad + 8];
        } else if (p.h != nullptr && rank == 0) {
            for (int i = threadIdx.x; i < rows * p.R; i += kThreads) p.h[static_cast<int64_t>(s_row[i / p.R]) * p.R + i % p.R] = 0.0f;
        }

        const int pitch = padded_pitch(rank_up(p.R));
        for (int c = chunk0; c < chunk1; ++c) {
            Eight y[2][2] = {};
            if (p.y != nullptr) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (row_of[i] >= 0)
                            y[g][i] = load_eight(p.y, p.y_type, row_of[i], p.ldy, 64 * c + 32 * g + 8 * (lane & 3), p.D, p.out_wide);
                    }
                }
            }
            if (adapter >= 0) {
                cp_wait<1>();
                __syncthreads();
            }
            if (16 * warp < rows) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    float o[2][8] = {};
                    if (adapter >= 0)
                        multiply_up<T, kTrans>(o, base + lay.h + 16 * warp * pitch, kManyRows * pitch, terms,
                                               base + lay.up + ((c - chunk0) & 1) * lay.up_size, g, p.R, lane);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) o[i][j] *= undo[i];
                        if (row_of[i] >= 0)
                            store_eight(p.out, p.y_type, row_of[i], p.ldo, 64 * c + 32 * g + 8 * (lane & 3), p.D, p.out_wide, y[g][i], o[i]);
                    }
                }
            }
            if (adapter >= 0) {
                __syncthreads();
                load_up_chunk(c + 2);
            }
        }
        cp_wait<0>();
    }
}

template <typename T, bool kTrans>
cudaError_t launch_many(const Params& p, int64_t tiles, bool pdl, cudaStream_t st) {
    const int terms = terms_of<T>(p.y_type);
    const ManyLayout<kTrans> lay(p.R, terms);
    // clusters that run at once, about: those a tile more than once take turns
    const int64_t resident = static_cast<int64_t>(device_sm_count()) * (lay.total <= 75 * 1024 ? 3 : lay.total <= 112 * 1024 ? 2 : 1) / kSplit;
    const int64_t clusters = tiles < resident ? tiles : resident;
    return by_rank(p.R, [&](auto rank) {
        constexpr int kRank = decltype(rank)::value;
        static Ready ready;
        auto* kernel = many_kernel<T, kTrans, kRank>;
        const cudaError_t e = allow_shared(reinterpret_cast<const void*>(kernel), ManyLayout<kTrans>(kRank, 3).total, ready);
        if (e != cudaSuccess) return e;
        return launch_pdl(pdl, kernel, dim3(static_cast<unsigned>(clusters * kSplit)), dim3(kThreads), static_cast<size_t>(lay.total), st,
                          p, terms);
    });
}

}  // namespace lora
}  // namespace nvfp4
