// Gradients of low-rank adapters:  dA_a = sum_t dh_t x_t^T  [R][K],  dB_a = sum_t s_a dy_t h_t^T  [N][R],  over the tokens of
// adapter a in their order.
//
// Both are sums over tokens of a column of R values (dh, or s h) times a row of 128 columns (of x, or dy); a CTA takes one
// adapter and one slab of 128 columns, 64 tokens a stage, and keeps the R x 128 sums in registers.  Few slabs of few
// adapters leave SMs idle, so up to 8 CTAs of a cluster share a slab's tokens and add their sums in order: no atomics, the
// same bits every time.
//
// dh and h are FP32; they are taken as sums of three BF16 terms (2^-25 of them is left), as x and dy are BF16 and the
// sums FP32.
#include "lora_launch.cuh"

namespace nvfp4 {
namespace lora {
namespace {

constexpr int kCols = 128, kTokens = 64, kTerms = 3;
constexpr int kPitch = kCols + 4;         // floats of a row of the sums in shared memory

struct GradLayout {
    int h_at, stage, total;
    __host__ __device__ explicit GradLayout(int R) {
        h_at = kTokens * kCols * 2;
        stage = h_at + (kTerms * kTokens * padded_pitch(rank_up(R)) + 127) / 128 * 128;
        const int sums = rank_up(R) * kPitch * 4;
        total = 2 * stage > sums ? 2 * stage : sums;
    }
};

template <int kRank>
__global__ void __launch_bounds__(kThreads) grad_kernel(const GradParams p, const int slabs_k) {
    constexpr int kM = kRank / 16;        // tiles of 16 ranks
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_rows[2][kTokens];
    const GradLayout lay(p.R);
    const uint32_t base = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = static_cast<int>(cluster_rank()), parts = static_cast<int>(cluster_size());
    const int slab = blockIdx.x / parts, adapter = blockIdx.y;
    const bool is_down = slab < slabs_k;
    const int col0 = (is_down ? slab : slab - slabs_k) * kCols, width = is_down ? p.K : p.N;
    const uint16_t* x = is_down ? p.x : p.dy;
    const int64_t ldx = is_down ? p.ldx : p.lddy;
    const bool wide = is_down ? p.x_wide : p.dy_wide;
    const float* h = is_down ? p.dh : p.h;
    const float scale = is_down || p.scale == nullptr ? 1.0f : p.scale[adapter];
    pdl_wait();
    const int begin = p.tiles.offsets[adapter], all = p.tiles.offsets[adapter + 1] - begin;
    const int share = ((all + kTokens - 1) / kTokens + parts - 1) / parts * kTokens;
    const int first = min(part * share, all), last = min(first + share, all);
    const int stages = (last - first + kTokens - 1) / kTokens;

    const int pitch = padded_pitch(rank_up(p.R)), quads = p.R / 4;
    float4 held[kRank / 16];
    const auto list_rows = [&](int s) {
        if (threadIdx.x < kTokens) {
            const int i = first + s * kTokens + static_cast<int>(threadIdx.x);
            s_rows[s & 1][threadIdx.x] = i < last ? p.tiles.perm[begin + i] : -1;
        }
    };
    const auto load_x = [&](int s) {
        const uint32_t at = base + (s & 1) * lay.stage;
        const int q = threadIdx.x & 15;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = (threadIdx.x >> 4) + 16 * i, t = s_rows[s & 1][r];
            const uint32_t to = at + (q >> 3) * (kTokens * 128) + swizzled(r, q & 7);
            copy_chunk(to, x + (t < 0 ? 0 : t * ldx), t < 0 ? width : col0 + 8 * q, width, wide);
        }
        cp_commit();
    };
    const auto load_h = [&](int s) {
#pragma unroll
        for (int j = 0; j < kRank / 16; ++j) {
            const int i = threadIdx.x + kThreads * j, r = i / quads;
            const int t = r < kTokens ? s_rows[s & 1][r] : -1;
            held[j] = t < 0 ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                            : *reinterpret_cast<const float4*>(h + static_cast<int64_t>(t) * p.R + 4 * (i - r * quads));
        }
    };
    const auto store_h = [&](int s) {
#pragma unroll
        for (int j = 0; j < kRank / 16; ++j) {
            const int i = threadIdx.x + kThreads * j, r = i / quads;
            if (r >= kTokens) continue;
            float v[4] = {held[j].x * scale, held[j].y * scale, held[j].z * scale, held[j].w * scale};
            uint8_t* to = smem + (s & 1) * lay.stage + lay.h_at + r * pitch + 8 * (i - r * quads);
#pragma unroll
            for (int t = 0; t < kTerms; ++t) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = next_term<__nv_bfloat16>(v[k]);
                *reinterpret_cast<uint2*>(to + t * kTokens * pitch) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
            }
        }
    };

    float acc[kM][4][4];
#pragma unroll
    for (int m = 0; m < kM; ++m) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
        }
    }
    // warps 0-3 take 32 columns each of the even steps of 16 tokens, 4-7 of the odd ones
    const int cols = 32 * (warp & 3);
    list_rows(0);
    list_rows(1);
    __syncthreads();
    if (stages > 0) {
        load_x(0);
        load_h(0);
    }
    for (int s = 0; s < stages; ++s) {
        store_h(s);
        cp_wait<0>();
        __syncthreads();
        if (s + 1 < stages) {
            load_x(s + 1);
            load_h(s + 1);
        }
        // rows of the stage after the next, whose place is free since the last barrier but one
        if (s + 2 < stages) list_rows(s + 2);
        const uint32_t sx = base + (s & 1) * lay.stage + (cols >> 6) * (kTokens * 128), sh = base + (s & 1) * lay.stage + lay.h_at;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int token = 16 * (2 * k + (warp >> 2));
            uint32_t b[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n)
                ldsm4_trans(sx + swizzled(token + (lane & 7) + ((lane >> 3) & 1) * 8, ((cols & 63) >> 3) + 2 * n + (lane >> 4)), b[n]);
#pragma unroll
            for (int m = 0; m < kM; ++m) {
                if (16 * m >= p.R) break;
#pragma unroll
                for (int t = 0; t < kTerms; ++t) {
                    uint32_t a[4];
                    ldsm4_trans(sh + t * kTokens * pitch + (token + (lane & 7) + (lane >> 4) * 8) * pitch + 32 * m + 16 * ((lane >> 3) & 1), a);
#pragma unroll
                    for (int n = 0; n < 4; ++n) mma(__nv_bfloat16(), acc[m][n], a, b[n >> 1][2 * (n & 1)], b[n >> 1][2 * (n & 1) + 1]);
                }
            }
        }
    }

    // the two halves' sums, then the CTAs' in their order, a part of them each
    __syncthreads();
    float* sums = reinterpret_cast<float*>(smem);
    for (int half = 0; half < 2; ++half) {
        if ((warp >> 2) == half) {
#pragma unroll
            for (int m = 0; m < kM; ++m) {
                if (16 * m >= p.R) break;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float& to = sums[(16 * m + (lane >> 2) + 8 * (i >> 1)) * kPitch + cols + 8 * n + 2 * (lane & 3) + (i & 1)];
                        to = half == 0 ? acc[m][n][i] : to + acc[m][n][i];
                    }
                }
            }
        }
        __syncthreads();
    }
    cluster_barrier();
    const int total = p.R * kCols, each = (total + parts - 1) / parts;
    float* out = is_down ? p.ddown + static_cast<int64_t>(adapter) * p.R * p.K : p.dup + static_cast<int64_t>(adapter) * p.N * p.R;
    for (int i = part * each + threadIdx.x; i < min((part + 1) * each, total); i += kThreads) {
        const int r = is_down ? i / kCols : i % p.R, c = is_down ? i % kCols : i / p.R;
        if (col0 + c >= width) continue;
        float v = sums[r * kPitch + c];
        if (parts > 1) {
            v = 0.0f;
            for (int k = 0; k < parts; ++k) v += cluster_load_f32(cluster_addr(sums + r * kPitch + c, k));
        }
        out[is_down ? static_cast<int64_t>(r) * p.K + col0 + c : static_cast<int64_t>(col0 + c) * p.R + r] = v;
    }
    cluster_barrier();                                      // no CTA leaves while another reads its sums
}

}  // namespace

cudaError_t launch_grad(const GradParams& p, cudaStream_t st) {
    const GradLayout lay(p.R);
    const int slabs_k = (p.K + kCols - 1) / kCols, slabs_n = (p.N + kCols - 1) / kCols;
    const int64_t units = static_cast<int64_t>(slabs_k + slabs_n) * p.L;
    int parts = 1;                        // CTAs to a slab: about four to an SM
    while (parts < 8 && units * parts * 2 <= 4 * device_sm_count()) parts *= 2;
    return by_rank(p.R, [&](auto rank) {
        constexpr int kRank = decltype(rank)::value;
        static Ready ready;
        auto* kernel = grad_kernel<kRank>;
        const cudaError_t e = allow_shared(reinterpret_cast<const void*>(kernel), GradLayout(kRank).total, ready);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>((slabs_k + slabs_n) * parts), static_cast<unsigned>(p.L));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = static_cast<size_t>(lay.total);
        cfg.stream = st;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(parts);
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, kernel, p, slabs_k);
    });
}

}  // namespace lora
}  // namespace nvfp4
