// Gradients of low-rank adapters:  dA_a = sum_t dh_t x_t^T  [R][K],  dB_a = sum_t s_a dy_t h_t^T  [N][R],  over the tokens of
// adapter a in their order.
//
// Both are sums over tokens of a column of R values (dh, or s h) times a row of x, or dy.  A CTA takes one adapter, up to 32
// of its ranks and a slab of 256 columns (a warp 32 of them), 32 tokens a stage, and keeps the sums in registers.  Few
// slabs of few adapters leave SMs idle, so up to 8 CTAs of a cluster share a slab's tokens and add their sums in order: no
// atomics, the same bits every time.  More than 32 ranks read the slab again, out of L2.
//
// dh and h are FP32; they are taken as sums of three BF16 terms (2^-24 of them is left), as x and dy are BF16 and the sums
// FP32.  The tensor cores cut an accumulator's low bits off at each step: one chain over 2048 tokens was 6e-6 of the
// result low, so every 8 stages (48 steps) the chain is added to FP32 sums beside it and starts anew.
#include "lora_launch.cuh"

namespace nvfp4 {
namespace lora {
namespace {

constexpr int kCols = 256, kTokens = 32, kTerms = 3, kRanks = 32;
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

template <int kM>
__global__ void __launch_bounds__(kThreads, 2) grad_kernel(const GradParams p, const int slabs_k, const int rank_parts) {
    using Lay = GradLayout<kM>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_rows[2][kIndexed * kTokens];
    const uint32_t base = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = static_cast<int>(cluster_rank()), parts = static_cast<int>(cluster_size());
    const int unit = blockIdx.x / parts, slab = unit / rank_parts, rank0 = unit % rank_parts * kRanks, adapter = blockIdx.y;
    const int ranks = min(kRanks, p.R - rank0);
    const bool is_down = slab < slabs_k;
    const int col0 = (is_down ? slab : slab - slabs_k) * kCols, width = is_down ? p.K : p.N;
    const uint16_t* x = is_down ? p.x : p.dy;
    const int64_t ldx = is_down ? p.ldx : p.lddy;
    const bool wide = is_down ? p.x_wide : p.dy_wide;
    const float* h = (is_down ? p.dh : p.h) + rank0;
    const float scale = is_down || p.scale == nullptr ? 1.0f : p.scale[adapter];
    pdl_wait();
    const int begin = p.tiles.offsets[adapter], all = p.tiles.offsets[adapter + 1] - begin;
    const int share = ((all + kTokens - 1) / kTokens + parts - 1) / parts * kTokens;
    const int first = min(part * share, all), last = min(first + share, all);
    const int stages = (last - first + kTokens - 1) / kTokens;
    const int32_t* perm = p.tiles.perm + begin + first;

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
            if (wide) {
#pragma unroll
                for (int i = 0; i < kCols / 64; ++i) {
                    const int c = col0 + 64 * i + 8 * (threadIdx.x & 7), left = t < 0 ? 0 : min(max(width - c, 0), 8);
                    cp_async16(at + i * Lay::tile + swizzled(r, threadIdx.x & 7), left ? row + c : row, 2 * left);
                }
            } else {
                Straddle s4[kCols / 64];
#pragma unroll
                for (int i = 0; i < kCols / 64; ++i) s4[i].load(row, t < 0 ? width : col0 + 64 * i + 8 * (threadIdx.x & 7), width);
#pragma unroll
                for (int i = 0; i < kCols / 64; ++i) s4[i].store(at + i * Lay::tile + swizzled(r, threadIdx.x & 7));
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
        for (int t = 0; t < kTerms; ++t) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = next_term<__nv_bfloat16>(v[k]);
            *reinterpret_cast<uint2*>(to + t * kTokens * Lay::pitch) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
        }
    };

    float acc[kM][4][4], total[kM][4][4];
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

    // the CTAs' sums in their order, a part of them each
    cp_wait<0>();
    __syncthreads();
    float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int m = 0; m < kM; ++m) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            float* at = sums + (16 * m + (lane >> 2)) * kPitch + 32 * warp + 8 * n + 2 * (lane & 3);
            *reinterpret_cast<float2*>(at) = make_float2(total[m][n][0], total[m][n][1]);
            *reinterpret_cast<float2*>(at + 8 * kPitch) = make_float2(total[m][n][2], total[m][n][3]);
        }
    }
    cluster_barrier();
    const int count = ranks * kCols, each = (count + parts - 1) / parts;
    float* out = is_down ? p.ddown + (static_cast<int64_t>(adapter) * p.R + rank0) * p.K : p.dup + static_cast<int64_t>(adapter) * p.N * p.R + rank0;
    for (int i = part * each + threadIdx.x; i < min((part + 1) * each, count); i += kThreads) {
        const int r = is_down ? i / kCols : i % ranks, c = is_down ? i % kCols : i / ranks;
        if (col0 + c >= width) continue;
        float v = cluster_load_f32(cluster_addr(sums + r * kPitch + c, 0));
        for (int k = 1; k < parts; ++k) v += cluster_load_f32(cluster_addr(sums + r * kPitch + c, k));
        out[is_down ? static_cast<int64_t>(r) * p.K + col0 + c : static_cast<int64_t>(col0 + c) * p.R + r] = v;
    }
    cluster_barrier();                                      // no CTA leaves while another reads its sums
}

template <int kM>
cudaError_t launch(const GradParams& p, cudaStream_t st) {
    const int slabs_k = (p.K + kCols - 1) / kCols, slabs_n = (p.N + kCols - 1) / kCols, rank_parts = (p.R + kRanks - 1) / kRanks;
    const int64_t units = static_cast<int64_t>(slabs_k + slabs_n) * rank_parts * p.L;
    int parts = 1;                        // CTAs to a slab: about four to an SM
    while (parts < 8 && units * parts * 2 <= 4 * device_sm_count()) parts *= 2;
    static Ready ready;
    const cudaError_t e = allow_shared(reinterpret_cast<const void*>(grad_kernel<kM>), GradLayout<kM>::total, ready);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((slabs_k + slabs_n) * rank_parts * parts), static_cast<unsigned>(p.L));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = GradLayout<kM>::total;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(parts);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, grad_kernel<kM>, p, slabs_k, rank_parts);
}

}  // namespace

cudaError_t launch_grad(const GradParams& p, cudaStream_t st) { return p.R <= 16 ? launch<1>(p, st) : launch<2>(p, st); }

}  // namespace lora
}  // namespace nvfp4
