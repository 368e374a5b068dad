// Low-rank adapters, tiles of up to 16 rows: decode batches, and the adapters of few tokens each.  lora.cuh says what is
// computed.
//
// Each of a CTA's 8 warps takes one sub-slice of C by itself: its part of x and of the adapter's matrix come in by cp.async
// for this warp alone, without a barrier; the operand of the second product and y are on their way meanwhile, so the loads
// of both products are under way at once and the rest is the latency of one chain: load, products, sums in the CTA, sums
// over the cluster, products, store.  8 x 4096 -> 4096 of rank 16, each row its own adapter, take 7.7 us (a launch, and three trips
// to memory and over the cluster), 77 x 2080 -> 1999 of rank 8 to FP32 9.8, 512 rows of dx (1536 -> 2048, rank 16) 9.5.  A tile reads its
// adapter out of L2 again: from some hundred rows of an adapter on tiles of 128 take less (few_rows).
#pragma once

#include <algorithm>

#include "lora_launch.cuh"

namespace nvfp4 {
namespace lora {

template <bool kTrans>
struct FewLayout {
    int cols;                             // of C that a warp holds at once
    int x, down, up;                      // bytes of a warp's buffers
    int buffers;                          // for the second product's operand
    int part, sum, h, total;              // offsets: the warps' sums, the CTA's, the terms of h; all bytes
    __host__ __device__ explicit FewLayout(int R, int terms) {
        cols = R <= 64 ? 64 : 32;
        buffers = R <= 64 ? 2 : 1;
        x = kFewRows * 128;
        down = (down_bytes<kTrans>(R, cols) + 127) / 128 * 128;
        up = (up_bytes<kTrans>(R, 32) + 127) / 128 * 128;
        const int loads = kWarps * (x + down);
        part = 0;                         // over the loads, which are used up then
        sum = part + kWarps * kFewRows * R * 4;
        h = sum + kFewRows * R * 4;
        const int end = h + terms * kFewRows * padded_pitch(rank_up(R));
        total = (end > loads ? end : loads) + 127;
        total = total / 128 * 128 + kWarps * buffers * up;
    }
    __host__ __device__ int up_at() const { return total - kWarps * buffers * up; }
};

// Tile `q` of up to 256 tokens, found by the CTA from the ids: the tokens of an adapter in their order, 16 to a tile, the
// tiles by their first token.  Returns false if there are fewer tiles.
__device__ __forceinline__ bool find_tile(const int32_t* ids, int T, int L, int q, int* s_id, int* s_row, int* s_warp, int& adapter,
                                          int& rows, int* err) {
    __shared__ int s_tile[3];             // adapter, first rank, rows
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    int id = -2;                          // no token
    if (t < T) {
        id = ids[t];
        if (id >= L) {
            if (q == 0) set_device_error(err, NVFP4_ERR_BAD_EXPERT_ID);
            id = -1;
        }
        if (id < 0) id = -1;
    }
    s_id[t] = id;
    if (t == 0) s_tile[2] = 0;
    __syncthreads();
    int rank = 0, all = 0;
    for (int i = 0; i < T; i += 4) {
        const int4 v = *reinterpret_cast<const int4*>(s_id + i);
        const int e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int same = e[j] == id;
            all += same;
            rank += same && i + j < t;
        }
    }
    const bool first = t < T && rank % kFewRows == 0;
    const unsigned firsts = __ballot_sync(kAll, first);
    if (lane == 0) s_warp[warp] = __popc(firsts);
    __syncthreads();
    int tile = __popc(firsts & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) tile += s_warp[w];
    if (first && tile == q) {
        s_tile[0] = id;
        s_tile[1] = rank;
        s_tile[2] = min(kFewRows, all - rank);
    }
    __syncthreads();
    adapter = s_tile[0];
    rows = s_tile[2];
    if (rows == 0) return false;
    if (id == adapter && rank >= s_tile[1] && rank < s_tile[1] + rows) s_row[rank - s_tile[1]] = t;
    return true;
}

// kRounds: C has more than one round of sub-slices (with a loop over them the kernels of fewer columns took up to 39 registers more).
template <typename T, bool kTrans, int kRank, bool kRounds>
__global__ void __cluster_dims__(kGroups, 1, 1) __launch_bounds__(kThreads) few_kernel(const Params p, const int terms) {
    constexpr int kTiles = kRank / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(16) int s_id[kInCta];
    __shared__ int s_row[kFewRows], s_warp[kWarps];
    __shared__ float s_undo[kFewRows];
    const FewLayout<kTrans> lay(p.R, terms);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane >> 2;
    const int rank = static_cast<int>(cluster_rank()), q = blockIdx.x / kGroups;

    int adapter, rows;
    if (p.tiles.perm == nullptr) {
        if (!find_tile(p.ids, p.T, p.L, q, s_id, s_row, s_warp, adapter, rows, p.err)) return;
    } else {
        pdl_wait();
        if (q >= *p.tiles.count) return;
        adapter = p.tiles.adapter[q];
        const int start = p.tiles.start[q];
        rows = min(kFewRows, p.tiles.offsets[(adapter < 0 ? p.L : adapter) + 1] - start);
        if (static_cast<int>(threadIdx.x) < rows) s_row[threadIdx.x] = p.tiles.perm[start + threadIdx.x];
    }
    if (adapter < 0 && p.skip_none) return;
    __syncthreads();

    // outputs in groups of 32, an eighth of them to each CTA, one at a time to each warp
    const int groups = (p.D + 31) / 32, per_cta = (groups + kGroups - 1) / kGroups;
    const int last_group = min((rank + 1) * per_cta, groups), first_group = rank * per_cta + warp;
    const uint16_t* up = static_cast<const uint16_t*>(p.up) + static_cast<int64_t>(max(adapter, 0)) * p.D * p.R;
    const uint32_t my_up = smem_u32(smem) + lay.up_at() + warp * lay.buffers * lay.up;
    const int row_of[2] = {quad < rows ? s_row[quad] : -1, quad + 8 < rows ? s_row[quad + 8] : -1};
    Eight y[2] = {};
    const auto load_y = [&](int g) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (p.y != nullptr && row_of[i] >= 0) y[i] = load_eight(p.y, p.y_type, row_of[i], p.ldy, 32 * g + 8 * (lane & 3), p.D, p.y_wide);
        }
    };
    float undo[2] = {1.0f, 1.0f};

    if (adapter >= 0) {
        const uint16_t* down = static_cast<const uint16_t*>(p.down) + static_cast<int64_t>(adapter) * p.C * p.R;
        const int steps = sub_steps(p.C), rounds = kRounds ? sub_rounds(p.C) : 1;
        uint8_t* my = smem + warp * (lay.x + lay.down);
        const uint32_t sx = smem_u32(my), sd = sx + lay.x;
        float* sum = reinterpret_cast<float*>(smem + lay.sum);
        float mine[kRank / 16];           // of the CTA's sums, while there are rounds
        for (int round = 0; round < rounds; ++round) {
            const int c0 = ((rank * rounds + round) * kWarps + warp) * steps * 16, c1 = min(c0 + steps * 16, p.C);
            float acc[kTiles][4];
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
            }
            const auto load_piece = [&](int c) {
                const int cols = min(lay.cols, (c1 - c + 15) / 16 * 16);
                load_down<kTrans>(sd, down, p.R, p.C, c, cols, lane, 32);
                const int chunk = lane & 7;
                if (8 * chunk < cols) {
                    for (int r = lane >> 3; r < rows; r += 4)
                        copy_chunk(sx + swizzled(r, chunk), static_cast<const uint16_t*>(p.x) + s_row[r] * p.ldx, c + 8 * chunk, p.C);
                }
            };
            if (c0 < c1) load_piece(c0);
            cp_commit();
            if (round == 0) {
                for (int b = 0; b < lay.buffers; ++b) {
                    if (first_group + 8 * b < last_group)
                        load_up<kTrans>(my_up + b * lay.up, up, p.R, p.D, 32 * (first_group + 8 * b), 32, lane, 32);
                    cp_commit();
                }
                if (first_group < last_group) load_y(first_group);
                if (lay.buffers == 2) cp_wait<2>();
                else cp_wait<1>();
            } else {
                cp_wait<0>();
            }
            __syncwarp();
            for (int c = c0; c < c1; c += lay.cols) {
                if (c > c0) {
                    __syncwarp();
                    load_piece(c);
                    cp_commit();
                    cp_wait<0>();
                    __syncwarp();
                }
                const int n = min(lay.cols, c1 - c);
                for (int kk = 0; 16 * kk < n; ++kk) {
                    uint32_t a[4];
                    ldsm4((sx + lane_rows(lane)) ^ (kk << 5), a);
                    multiply_down<T, kTrans, kTiles>(acc, a, sd + lane_down<kTrans>(lane, p.R), kk, p.R);
                }
            }
            __syncthreads();                                // every warp's loads are used up
            float* part = reinterpret_cast<float*>(smem + lay.part) + warp * kFewRows * p.R;
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
                if (8 * j >= p.R) break;
                float* at = part + quad * p.R + 8 * j + 2 * (lane & 3);
                *reinterpret_cast<float2*>(at) = make_float2(acc[j][0], acc[j][1]);
                *reinterpret_cast<float2*>(at + 8 * p.R) = make_float2(acc[j][2], acc[j][3]);
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kRank / 16; ++j) {
                const int i = threadIdx.x + kThreads * j;
                if (i >= kFewRows * p.R) break;
                const float* from = reinterpret_cast<const float*>(smem + lay.part) + i;
                float v = round > 0 ? mine[j] + from[0] : from[0];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) v += from[w * kFewRows * p.R];
                mine[j] = v;
                if (round + 1 == rounds) sum[i] = v;
            }
            if (round + 1 < rounds) __syncthreads();        // the next round's loads lie over the parts
        }
        cluster_barrier();
        const int row = 2 * warp + (lane >> 4), pitch = padded_pitch(rank_up(p.R));
        const bool keep = p.h != nullptr && row < rows && (row >> 1) == rank;
        float row_undo;
        uint8_t* h = smem + lay.h + row * pitch;
        finish_row<T, kRank, 16>(sum, kGroups, row, p.R, p.R, p.scale == nullptr ? 1.0f : p.scale[adapter], terms, kFewRows * pitch,
                             keep ? p.h + static_cast<int64_t>(s_row[row]) * p.R : nullptr, p.h_scaled != 0, lane & 15,
                             [&](int at, uint32_t v) { *reinterpret_cast<uint32_t*>(h + at) = v; }, row_undo);
        if ((lane & 15) == 0) s_undo[row] = row_undo;
        cluster_barrier_arrive();                           // the other CTAs' sums are read
        __syncthreads();
        undo[0] = s_undo[quad];
        undo[1] = s_undo[quad + 8];
    } else {
        if (first_group < last_group) load_y(first_group);
        if (p.h != nullptr && rank == 0) {
            for (int i = threadIdx.x; i < rows * p.R; i += kThreads) p.h[static_cast<int64_t>(s_row[i / p.R]) * p.R + i % p.R] = 0.0f;
        }
    }

    int b = 0;
    for (int g = first_group; g < last_group; g += kWarps) {
        float o[2][8] = {};
        if (adapter >= 0) {
            if (lay.buffers == 2) cp_wait<1>();
            else cp_wait<0>();
            __syncwarp();
            multiply_up<T, kTrans>(o, smem_u32(smem) + lay.h, kFewRows * padded_pitch(rank_up(p.R)), terms, my_up + b * lay.up, 0, p.R, lane);
            __syncwarp();
            const int next = g + kWarps * lay.buffers;
            if (next < last_group) load_up<kTrans>(my_up + b * lay.up, up, p.R, p.D, 32 * next, 32, lane, 32);
            cp_commit();
            if (++b == lay.buffers) b = 0;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) o[i][j] *= undo[i];
            const int n = 32 * g + 8 * (lane & 3);
            if (row_of[i] < 0) continue;
            Eight v = y[i];               // where there is no y it stays zeros
            if (adapter >= 0) add_eight(v, o[i], p.y_type);   // a row without one keeps its bits (-0 + 0 is +0)
            store_eight(static_cast<uint8_t*>(p.out) + (row_of[i] * p.ldo + n) * (p.y_type == NVFP4_TYPE_F32 ? 4 : 2), p.y_type, n, p.D,
                        p.out_wide, v);
        }
        if (g + kWarps < last_group) load_y(g + kWarps);
    }
    if (adapter >= 0) cluster_barrier_wait();
}

template <typename T, bool kTrans>
cudaError_t launch_few(const Params& p, int64_t tiles, bool pdl, cudaStream_t st) {
    const int terms = terms_of<T>(p.y_type);
    const FewLayout<kTrans> lay(p.R, terms);
    const auto launch = [&](auto rank, auto rounds, int shared) {
        static Ready ready;
        auto* kernel = few_kernel<T, kTrans, decltype(rank)::value, decltype(rounds)::value>;
        const cudaError_t e = allow_shared(reinterpret_cast<const void*>(kernel), shared, ready);
        if (e != cudaSuccess) return e;
        return launch_pdl(pdl, kernel, dim3(static_cast<unsigned>(tiles * kGroups)), dim3(kThreads), static_cast<size_t>(lay.total), st,
                          p, terms);
    };
    if (sub_rounds(p.C) > 1)              // of any rank; up to 64 some layouts are larger
        return launch(std::integral_constant<int, 128>(), std::true_type(),
                      std::max(FewLayout<kTrans>(64, 3).total, FewLayout<kTrans>(128, 3).total));
    return by_rank(p.R, [&](auto rank) { return launch(rank, std::false_type(), FewLayout<kTrans>(decltype(rank)::value, 3).total); });
}

}  // namespace lora
}  // namespace nvfp4
