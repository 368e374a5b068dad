// Dense 4-bit product out[t, n] = sum_k a[t, k] b[n, k] (+ bias[n]) of quantised rows on tcgen05.
//
//   NVFP4: acc = sum_k (qa*sa)[t,k] (qb*sb)[n,k] (E4M3 scales per 16), out = (acc*ga[t])*gb[n] + bias
//   MXFP4: acc = the same with E8M0 scales per 32 and no outer scales
//
// Kernel (sm_103a): one CTA per SM walks the (128 tokens x BN outputs) tiles.  Warp 0 loads a
// stage of 256 K-elements through TMA (128B swizzle) with its 512-byte scale tiles; warp 1 copies
// the scales to TMEM and issues the K=64 MMAs (M=128, N=BN) into an FP32 TMEM accumulator; warps
// 2-5 apply the outer scales and the bias and write their rows.  All waits are bounded
// (NVFP4_ERR_DEVICE_TIMEOUT, then a clean exit).
//
// K is walked 0..K-1 in 64-wide steps into one accumulator whatever the tile, so a token's output
// does not depend on how many tokens there are.
#include <mutex>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ops.cuh"
#include "ptx.cuh"

namespace nvfp4 {
namespace {

constexpr int kBM = 128;
constexpr int kRowBytes = 128;                       // bytes of K per row and stage: 256 elements
constexpr int kStageK = 256;
constexpr int kMaxStages = 12;
constexpr int kEpiWarps = 4;
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr uint32_t kTmemCols = 512;
constexpr int kSmemLimit = 227 * 1024;
constexpr int kFixedBytes = 4096;                    // column data, barriers, alignment slack

template <bool kMx>
struct Format {
    static constexpr int tiles = kMx ? 2 : 4;        // scale tiles of one 128-row set per stage
    static constexpr int tile_k = kStageK / tiles;   // K-elements of one
};

// Width of the MMA of a BN-wide tile.  The MMA's B scales have to start on an even TMEM column (32
// rows each) of their 128-row tile, so a tile of 32 outputs is the lower or upper half of an N=64
// MMA whose other half is not used.
__host__ __device__ constexpr int mma_n(int bn) { return bn < 64 ? 64 : bn; }

__host__ __device__ constexpr uint32_t idesc_fp4(bool mx, int M, int N) {
    return (1u << 7) | (1u << 10)                     // A, B: E2M1
           | (static_cast<uint32_t>(N >> 3) << 17)    // N / 8
           | ((mx ? 1u : 0u) << 23)                   // scale format: UE4M3 or UE8M0
           | (static_cast<uint32_t>(M >> 4) << 24);   // M / 16
}
// Scale-factor ids: which byte pair of a 4-byte scale word an MXFP4 MMA uses (0 or 2).
__host__ __device__ constexpr uint32_t idesc_sf_id(uint32_t id) { return (id << 4) | (id << 29); }

__device__ __forceinline__ void mma_fp4_elect(bool mx, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                              uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    if (mx)
        asm volatile(
            "{\n\t.reg .pred ep, acc;\n\t.reg .b32 er;\n\telect.sync er|ep, 0xffffffff;\n\t"
            "setp.ne.b32 acc, %4, 0;\n\t"
            "@ep tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], acc;\n\t}" ::"r"(
                d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
            : "memory");
    else
        tc_mma_nvf4_elect(d, a, b, idesc, sfa, sfb, accumulate);
}

struct Params {
    int64_t T;
    int N, K;
    const uint8_t* a_sf;
    const uint8_t* b_sf;
    const float* a_g;
    const float* b_g;
    const float* bias;
    void* out;
    int out_type;
    int64_t ldo;
    int vec;              // rows of out start and end on 16-byte boundaries
    int a_rows;           // rows of A loaded per tile (a multiple of 8, at most 128)
    int stages, stage_bytes;
    int n_tiles;
    int64_t tiles;
    int* err;
};

template <typename T>
__device__ __forceinline__ T to_out(float v);
template <>
__device__ __forceinline__ float to_out<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 to_out<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half to_out<__half>(float v) { return __float2half_rn(v); }

// 16 consecutive outputs of a row, of which the first `n` exist.
template <typename T>
__device__ __forceinline__ void store16(T* p, const float (&v)[16], int n, bool vec) {
    if (vec && n >= 16) {
        T o[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = to_out<T>(v[i]);
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)); ++i)
            reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(o)[i];
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (i < n) p[i] = to_out<T>(v[i]);
        }
    }
}

template <bool kMx, int BN>
__global__ void __launch_bounds__(kThreads, 1)
    linear_fp4_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const Params p) {
    using F = Format<kMx>;
    constexpr int kSfbSets = BN > 128 ? 2 : 1;                     // 128-row sets of B scale tiles
    constexpr int kSfSet = F::tiles * kSfAtomBytes;
    constexpr uint32_t kSfCols = 4 * F::tiles * (1 + kSfbSets);    // TMEM columns of a stage's scales
    constexpr int kAcc = BN <= 128 ? 2 : 1;                        // accumulators
    constexpr int kN = mma_n(BN);
    constexpr int kBBytes = kN * kRowBytes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], tmem_full[2], tmem_empty[2], drain;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word;
    __shared__ float s_col[kEpiWarps][2][32];
    volatile int* abort_flag = &abort_word;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int a_bytes = p.a_rows * kRowBytes;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tmem_full[i], 1);
            mbar_init(&tmem_empty[i], 32 * kEpiWarps);
        }
        mbar_init(&drain, 1);
        abort_word = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
    }
    if (warp == 1) {
        tmem_alloc(&tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    pdl_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const int num_ks = (p.K + kStageK - 1) / kStageK;
    const int sf_tiles = (p.K + F::tile_k - 1) / F::tile_k;        // scale tiles of a 128-row set, all of K
    bool failed = false;

    if (warp == 0) {
        const uint64_t pol_a = policy_evict_last(), pol_b = policy_evict_normal();
        int stage = 0;
        uint32_t phase = 0, issued = 0, issued_parity = 0;
        for (int64_t t = blockIdx.x; t < p.tiles && !failed; t += gridDim.x) {
            const int64_t mt = t / p.n_tiles;
            const int n0 = static_cast<int>(t % p.n_tiles) * BN;
            for (int ks = 0; ks < num_ks; ++ks) {
                const bool ok = mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, kWaitBudgetCycles);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    failed = true;
                    break;
                }
                uint8_t* st = smem + stage * p.stage_bytes;
                const int nt = min(F::tiles, sf_tiles - F::tiles * ks);
                const uint32_t sf_bytes = static_cast<uint32_t>(nt) * kSfAtomBytes;
                // the second set of a BN = 256 tile is past the end of B when N has none
                const int sets = kSfbSets == 2 && n0 + 128 < (p.N + 127) / 128 * 128 ? 2 : 1;
                mbar_arrive_expect_tx_elect(&full[stage], a_bytes + BN * kRowBytes + (1 + sets) * sf_bytes);
                tma_load_2d_elect(st, &tmA, &full[stage], ks * kRowBytes, static_cast<int>(mt * kBM), pol_a);
                uint8_t* b = st + a_bytes;
                tma_load_2d_elect(b + (n0 & (kN - BN)) * kRowBytes, &tmB, &full[stage], ks * kRowBytes, n0, pol_b);
                uint8_t* sf = b + kBBytes;
                bulk_load_elect(sf, p.a_sf + (mt * sf_tiles + F::tiles * ks) * kSfAtomBytes, sf_bytes, &full[stage],
                                pol_a);
                for (int i = 0; i < sets; ++i)
                    bulk_load_elect(sf + (1 + i) * kSfSet,
                                    p.b_sf + (static_cast<int64_t>(n0 / 128 + i) * sf_tiles + F::tiles * ks) *
                                                 kSfAtomBytes,
                                    sf_bytes, &full[stage], pol_b);
                issued |= 1u << stage;
                issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (failed) {
            if (lane == 0) set_device_error(p.err, NVFP4_ERR_DEVICE_TIMEOUT);
            *abort_flag = 1;
            for (int s = 0; s < p.stages; ++s) {
                if (issued & (1u << s)) mbar_wait_bounded(&full[s], (issued_parity >> s) & 1u, nullptr, kWaitBudgetCycles);
            }
        }
    } else if (warp == 1) {
        const uint32_t idesc = idesc_fp4(kMx, kBM, kN);
        const uint32_t sf0 = tmem + kAcc * kN;
        int stage = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool issued_any = false;
        for (int64_t t = blockIdx.x; t < p.tiles && !failed; t += gridDim.x) {
            const int n0 = static_cast<int>(t % p.n_tiles) * BN;
            // first scale column of the MMA's rows within their 128-row tile
            const uint32_t sfb_col = kN == 64 ? static_cast<uint32_t>(n0 & 64) / 32 : 0u;
            const bool ok = mbar_wait_bounded(&tmem_empty[acc], acc_phase ^ 1u, abort_flag, kWaitBudgetCycles);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                failed = true;
                break;
            }
            tc_fence_after();
            for (int ks = 0; ks < num_ks; ++ks) {
                const bool okf = mbar_wait_bounded(&full[stage], phase, abort_flag, kWaitBudgetCycles);
                if (!__all_sync(0xFFFFFFFFu, okf)) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                const uint32_t st = smem_u32(smem + stage * p.stage_bytes);
                const uint64_t ad = sdesc_k_swizzled<kRowBytes>(st);
                const uint64_t bd = sdesc_k_swizzled<kRowBytes>(st + a_bytes);
                const uint32_t sf = st + a_bytes + kBBytes;
                const uint32_t sfa = sf0 + stage * kSfCols, sfb = sfa + 4 * F::tiles;
                const int nk = min(kStageK / 64, (p.K - kStageK * ks + 63) / 64);
#pragma unroll
                for (int j = 0; j < kStageK / 64; ++j) {
                    if (j >= nk) break;
                    const int tile = kMx ? j >> 1 : j;
                    if (!kMx || (j & 1) == 0) {
                        tc_cp_32x128b_warpx4_elect(sfa + 4 * tile, sdesc_sf(sf + kSfAtomBytes * tile));
#pragma unroll
                        for (int i = 0; i < kSfbSets; ++i)
                            tc_cp_32x128b_warpx4_elect(sfb + 4 * (kSfbSets * tile + i),
                                                       sdesc_sf(sf + (1 + i) * kSfSet + kSfAtomBytes * tile));
                    }
                    mma_fp4_elect(kMx, tmem + acc * kN, ad + 2 * j, bd + 2 * j,
                                  kMx ? idesc | idesc_sf_id(2 * (j & 1)) : idesc, sfa + 4 * tile,
                                  sfb + 4 * kSfbSets * tile + sfb_col, (ks | j) != 0 ? 1u : 0u);
                }
                issued_any = true;
                tc_commit_elect(&empty[stage]);
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (failed) break;
            tc_commit_elect(&tmem_full[acc]);
            if (++acc == kAcc) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
        if (failed) {
            if (lane == 0) set_device_error(p.err, NVFP4_ERR_DEVICE_TIMEOUT);
            *abort_flag = 1;
            if (issued_any) {   // wait for the MMAs already issued before TMEM is released
                tc_commit_elect(&drain);
                mbar_wait_bounded(&drain, 0, nullptr, kWaitBudgetCycles);
            }
        }
    } else {
        const int q = warp & 3;                                    // TMEM lane quarter
        float* gcol = s_col[warp - 2][0];
        float* bcol = s_col[warp - 2][1];
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int64_t t = blockIdx.x; t < p.tiles; t += gridDim.x) {
            const int64_t r = t / p.n_tiles * kBM + q * 32 + lane;
            const int n0 = static_cast<int>(t % p.n_tiles) * BN;
            const bool live = r < p.T;
            const float ga = !kMx && live ? __ldg(p.a_g + r) : 1.0f;
            const bool ok = mbar_wait_bounded(&tmem_full[acc], acc_phase, abort_flag, kWaitBudgetCycles);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                if (lane == 0) set_device_error(p.err, NVFP4_ERR_DEVICE_TIMEOUT);
                *abort_flag = 1;
                break;
            }
            tc_fence_after();
            const uint32_t taddr = tmem + acc * kN + (n0 & (kN - BN)) + (static_cast<uint32_t>(q * 32) << 16);
            for (int c = 0; c < BN; c += 32) {
                const int n = n0 + c + lane;
                __syncwarp();
                gcol[lane] = !kMx && n < p.N ? __ldg(p.b_g + n) : 1.0f;
                bcol[lane] = p.bias != nullptr && n < p.N ? __ldg(p.bias + n) : 0.0f;
                __syncwarp();
                uint32_t v[32];
                tmem_ld_32x32b_x32(taddr + c, v);
                tmem_ld_wait();
#pragma unroll
                for (int h = 0; h < 32; h += 16) {
                    float o[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float y = __uint_as_float(v[h + i]);
                        if (!kMx) y = __fmul_rn(__fmul_rn(y, ga), gcol[h + i]);
                        o[i] = __fadd_rn(y, bcol[h + i]);
                    }
                    const int at = n0 + c + h, left = p.N - at;
                    if (!live || left <= 0) continue;
                    const int64_t off = r * p.ldo + at;
                    if (p.out_type == NVFP4_TYPE_F32) store16(static_cast<float*>(p.out) + off, o, left, p.vec);
                    else if (p.out_type == NVFP4_TYPE_BF16) store16(static_cast<__nv_bfloat16*>(p.out) + off, o, left, p.vec);
                    else store16(static_cast<__half*>(p.out) + off, o, left, p.vec);
                }
            }
            tc_fence_before();
            mbar_arrive(&tmem_empty[acc]);
            if (++acc == kAcc) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// 2D byte map over codes [rows][row_bytes] (row_bytes % 16 == 0): boxes of box_rows rows x 128
// bytes, 128B swizzle; what lies outside reads as zero codes.
bool make_map(CUtensorMap* m, const void* base, int64_t rows, int64_t row_bytes, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
    const cuuint32_t box[2] = {kRowBytes, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;
std::mutex g_linear_mutex;

template <bool kMx, int BN>
cudaError_t launch(const LinearArgs& a, cudaStream_t st, bool pdl) {
    static bool ready[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(g_linear_mutex);
        if (!ready[dev]) {
            e = cudaFuncSetAttribute(linear_fp4_kernel<kMx, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kSmemLimit - kFixedBytes);
            if (e != cudaSuccess) return e;
            ready[dev] = true;
        }
    }
    using F = Format<kMx>;
    constexpr int sets = BN > 128 ? 2 : 1;
    Params p{};
    p.T = a.T;
    p.N = a.N;
    p.K = a.K;
    p.a_sf = a.a_sf;
    p.b_sf = a.b_sf;
    p.a_g = a.a_g;
    p.b_g = a.b_g;
    p.bias = a.bias;
    p.out = a.out;
    p.out_type = a.out_type;
    p.ldo = a.ldo;
    const int size = a.out_type == NVFP4_TYPE_F32 ? 4 : 2;
    p.vec = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0 && (a.ldo * size) % 16 == 0;
    p.a_rows = a.T >= kBM ? kBM : static_cast<int>((a.T + 15) / 16 * 16);
    p.stage_bytes = p.a_rows * kRowBytes + mma_n(BN) * kRowBytes + (1 + sets) * F::tiles * kSfAtomBytes;
    p.stage_bytes = (p.stage_bytes + 1023) / 1024 * 1024;
    // An MMA reads 128 rows of A whatever a_rows is (the rows past it give results nobody reads):
    // 16 KB past the last stage's start stay inside the allocation.
    const int room = kSmemLimit - kFixedBytes - 1024 - (kBM - p.a_rows) * kRowBytes;
    p.stages = room / p.stage_bytes;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    const int by_tmem = static_cast<int>(kTmemCols - (BN <= 128 ? 2 : 1) * mma_n(BN)) / (4 * F::tiles * (1 + sets));
    if (p.stages > by_tmem) p.stages = by_tmem;
    const int num_ks = (a.K + kStageK - 1) / kStageK;
    p.n_tiles = (a.N + BN - 1) / BN;
    p.tiles = (a.T + kBM - 1) / kBM * p.n_tiles;
    p.err = a.err;
    const int sms = device_sm_count();
    const unsigned grid = static_cast<unsigned>(p.tiles < sms ? p.tiles : sms);
    if (p.tiles <= sms && p.stages > num_ks) p.stages = num_ks;
    const size_t smem = static_cast<size_t>(p.stages) * p.stage_bytes + (kBM - p.a_rows) * kRowBytes + 1024;
    CUtensorMap ma, mb;
    if (!make_map(&ma, a.a_codes, a.T, a.K / 2, p.a_rows) || !make_map(&mb, a.b_codes, a.N, a.K / 2, BN))
        return cudaErrorInvalidValue;
    return launch_pdl(pdl, linear_fp4_kernel<kMx, BN>, grid, kThreads, smem, st, ma, mb, p);
}

template <bool kMx>
cudaError_t by_tile(const LinearArgs& a, cudaStream_t st, bool pdl) {
    // the widest tile that still gives every SM one
    const int64_t m = (a.T + kBM - 1) / kBM, sms = device_sm_count();
    if (m * ((a.N + 255) / 256) >= sms) return launch<kMx, 256>(a, st, pdl);
    if (m * ((a.N + 127) / 128) >= sms) return launch<kMx, 128>(a, st, pdl);
    if (m * ((a.N + 63) / 64) >= sms) return launch<kMx, 64>(a, st, pdl);
    return launch<kMx, 32>(a, st, pdl);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t st, bool pdl) {
    return a.mx ? by_tile<true>(a, st, pdl) : by_tile<false>(a, st, pdl);
}

}  // namespace nvfp4
