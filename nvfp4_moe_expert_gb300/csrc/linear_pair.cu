// The dense product's kernel for many tokens: a pair of CTAs (two SMs) computes 256 tokens x 256
// outputs with tcgen05.mma.cta_group::2 (M=256, N=256, K=64).  What is computed: linear.cu.
//
// One SM takes in about 56 bytes a cycle by TMA; the 54 KB a stage of a one-CTA 128 x 256 tile needs are
// 980 cycles of that for 512 cycles of MMAs.  In the pair each SM loads its own 128 rows of A and half of
// B's 256 rows, 35 to 38 KB a stage, while its tensor core does the same work.
//
// Per CTA: warp 0 loads A and its scale tiles, warp 2 its half of B and the scale tiles of all of B (each
// SM's tensor core scales with its own TMEM); every copy completes on the leader's barrier.  The leader's
// warp 1 copies the scales of both CTAs to their TMEM and issues the MMAs; its commits free the stage in
// both.  Warps 4-19 of each CTA take the accumulator (128 lanes x 256 columns) to registers, hand TMEM
// back, and put their 32 rows x 64 columns in shared memory for a TMA store while the next tile's MMAs
// run.  (Stores straight from the lanes, 32 rows to an instruction, slowed the loads down: a tile of K = 8192
// took 19700 cycles instead of 17200 without any stores, one of K = 1536 6300 instead of 3900.)
//
// 8192 x 8192 x 8192 MXFP4 149 us, 7.4 PFLOP/s: the tensor pipe is active for 78% of them, at the power limit.  32768 x
// 4096 x 1536 NVFP4 85 us, bound by the operands' way into the SMs beside 268 MB of stores.
#include "linear.cuh"

namespace nvfp4 {
namespace {

constexpr int kPairN = 256;
constexpr int kPairThreads = 640;
constexpr int kPairEpiWarps = 16;
constexpr int kHalfBytes = 128 * kRowBytes;          // 128 rows of a stage: A, or half of B
constexpr uint32_t kAccCols = 256;
constexpr int kPairStatic = 9216;                    // room left for the kernel's static shared memory
constexpr int kOutBytes = 4096;                      // an epilogue warp's outputs on their way: 32 rows of 128 bytes

template <bool kMx>
struct PairStage {
    static constexpr int tiles = Format<kMx>::tiles;
    static constexpr int sfa = 2 * kHalfBytes;                     // then A's scale tiles
    static constexpr int sfb = sfa + tiles * kSfAtomBytes;         // then B's two sets
    static constexpr int bytes = (sfb + 2 * tiles * kSfAtomBytes + 1023) / 1024 * 1024;
    static constexpr uint32_t sf_cols = 12 * tiles;
    static constexpr int by_smem = (kSmemLimit - kPairStatic - 1024 - kPairEpiWarps * kOutBytes) / bytes;
    static constexpr int by_tmem = (kTmemCols - kAccCols) / sf_cols;
    static constexpr int count = by_smem < by_tmem ? by_smem : by_tmem;
    static constexpr int out = count * bytes;                      // the epilogue warps' outputs
    static constexpr int dynamic = out + kPairEpiWarps * kOutBytes + 1024;
    static_assert(count <= 32, "a lane sets up each stage's barriers");
};

struct PairParams {
    int64_t T;
    int N, K;
    const float* a_g;
    const float* b_g;
    const float* bias;
    void* out;
    int out_type;
    int64_t ldo;
    int align;            // of out's rows: out_align()
    int n_tiles;
    int64_t tiles;
    int* err;
};

__device__ __forceinline__ uint32_t cycles32() {
    uint32_t c;
    asm volatile("mov.u32 %0, %%clock;" : "=r"(c));
    return c;
}
__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The leader's copy of a shared-memory variable.
__device__ __forceinline__ uint32_t leader_addr(const void* p) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
    return r;
}

// Bounded wait on a barrier that the peer CTA arrives on.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, const volatile int* abort, long long budget) {
    const long long t0 = clock64();
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if (abort != nullptr && *abort) return false;
        if (clock64() - t0 > budget) return false;
    }
}

#define PAIR_ELECT "{\n\t.reg .pred ep;\n\t.reg .b32 er;\n\telect.sync er|ep, 0xffffffff;\n\t@ep "
// Copies to this CTA's shared memory that complete on the barrier at cluster address `bar`.
__device__ __forceinline__ void tma_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y, uint64_t policy) {
    asm volatile(PAIR_ELECT
                 "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
                 " [%0], [%1, {%3, %4}], [%2], %5;\n\t}" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void tma_3d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z,
                                            uint64_t policy) {
    asm volatile(PAIR_ELECT
                 "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
                 " [%0], [%1, {%3, %4, %5}], [%2], %6;\n\t}" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
                 : "memory");
}
// Arrive on `bar` in both CTAs when the elected lane's tcgen05 operations so far have completed.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
    asm volatile(PAIR_ELECT
                 "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
                     smem_u32(bar)),
                 "h"(static_cast<uint16_t>(3))
                 : "memory");
}
#undef PAIR_ELECT
// Relaxed: what it hands over is TMEM, read to the end before (tcgen05.wait::ld).  A release at cluster
// scope also waits for the outputs the CTA's other warps are storing, 2000 cycles a tile.
__device__ __forceinline__ void arrive_leader(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A warp's 64 columns at n0 of the 32 rows at row0 (this lane's: accumulator values v) through its
// shared-memory buffer: rows of 128 bytes, 128B swizzle, one TMA store for 64 16-bit or 32 FP32 columns.
template <bool kMx, bool kBias, typename T>
__device__ __forceinline__ void outputs_staged(const uint32_t* v, float ga, const float* gcol, const float* bcol, uint8_t* buf,
                                               const CUtensorMap* map, int n0, int row0, int N) {
    constexpr int kCols = 128 / sizeof(T), kChunks = sizeof(T);   // columns of a store; 16-byte chunks of 16 columns
    const int lane = threadIdx.x & 31;
    const uint64_t g2 = pair(ga, ga);
    const uint32_t row = smem_u32(buf) + lane * 128;
#pragma unroll
    for (int c = 0; c < 64; c += kCols) {
        if (n0 + c >= N) break;
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // the buffer's last store has read it
        __syncwarp();
#pragma unroll
        for (int h = 0; h < kCols; h += 16) {
            uint64_t o[8];
            scale16<kMx, kBias>(v + c + h, g2, gcol + c + h, bcol + c + h, o);
            uint32_t w[4 * kChunks];
            pack16<T>(o, w);
#pragma unroll
            for (int i = 0; i < kChunks; ++i)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + (((h / 16 * kChunks + i) ^ (lane & 7)) << 4)),
                             "r"(w[4 * i]), "r"(w[4 * i + 1]), "r"(w[4 * i + 2]), "r"(w[4 * i + 3])
                             : "memory");
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0)
            asm volatile(
                "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];\n\tcp.async.bulk.commit_group;" ::"l"(
                    reinterpret_cast<uint64_t>(map)),
                "r"(smem_u32(buf)), "r"(n0 + c), "r"(row0)
                : "memory");
    }
}
template <bool kMx, typename T>
__device__ __forceinline__ void outputs_staged(const uint32_t* v, float ga, const float* gcol, const float* bcol, uint8_t* buf,
                                               const CUtensorMap* map, int n0, int row0, const PairParams& p) {
    if (p.bias != nullptr) outputs_staged<kMx, true, T>(v, ga, gcol, bcol, buf, map, n0, row0, p.N);
    else outputs_staged<kMx, false, T>(v, ga, gcol, bcol, buf, map, n0, row0, p.N);
}

// kStaged: outputs go through the tensor map tmOut, otherwise row by row (write_by_row).
template <bool kMx, bool kStaged>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmSfa, const __grid_constant__ CUtensorMap tmSfb,
                       const __grid_constant__ CUtensorMap tmOut, const PairParams p) {
    using S = PairStage<kMx>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[S::count], empty[S::count], tmem_full, tmem_empty, drain;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word;
    __shared__ __align__(8) float s_col[kPairEpiWarps][2][64];
    volatile int* abort_flag = &abort_word;
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const uint32_t rank = uniform(cta_rank());

    if (warp == 0) {
        if (lane < S::count) {
            mbar_init(&full[lane], 2);                // the leader's two producers
            mbar_init(&empty[lane], 1);
        }
        if (lane == 0) {
            mbar_init(&tmem_full, 1);
            mbar_init(&tmem_empty, 2 * kPairEpiWarps);
            mbar_init(&drain, 1);
            abort_word = 0;
            prefetch_tensormap(&tmA);
            prefetch_tensormap(&tmSfa);
        }
        fence_barrier_init();
    } else if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else if (warp == 2 && lane == 0) {
        prefetch_tensormap(&tmB);
        prefetch_tensormap(&tmSfb);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                   // both CTAs' barriers and TMEM are there
    tc_fence_after();
    const uint32_t tmem = uniform(tmem_slot);
    const int num_ks = (p.K + kStageK - 1) / kStageK;
    const int64_t first = blockIdx.x >> 1, step = gridDim.x >> 1;
    bool failed = false;

    if (warp == 0 || warp == 2) {
        // ------------------------------------------------------------ producers
        const bool is_a = warp == 0;
        const uint64_t pol = policy_evict_last();
        int stage = 0;
        uint32_t phase = 0, issued = 0, issued_parity = 0;
        if (is_a) pdl_wait();                         // A is what the kernel before writes; B is the call's input
        for (int64_t t = first; t < p.tiles && !failed; t += step) {
            const int mt = static_cast<int>(t / p.n_tiles), nt = static_cast<int>(t % p.n_tiles);
            const int row = is_a ? mt * 256 + 128 * static_cast<int>(rank) : nt * kPairN + 128 * static_cast<int>(rank);
            for (int ks = 0; ks < num_ks; ++ks) {
                const bool ok = mbar_wait_cluster(&empty[stage], phase ^ 1u, abort_flag, kWaitBudgetCycles);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    failed = true;
                    break;
                }
                uint8_t* st = smem + stage * S::bytes;
                const uint32_t bar = leader_addr(&full[stage]);
                if (is_a) {
                    if (rank == 0) mbar_arrive_expect_tx_elect(&full[stage], 2 * (kHalfBytes + S::tiles * kSfAtomBytes));
                    tma_2d_pair(st, &tmA, bar, ks * kRowBytes, row, pol);
                    tma_3d_pair(st + S::sfa, &tmSfa, bar, 0, S::tiles * ks, row / 128, pol);
                } else {
                    if (rank == 0) mbar_arrive_expect_tx_elect(&full[stage], 2 * (kHalfBytes + 2 * S::tiles * kSfAtomBytes));
                    tma_2d_pair(st + kHalfBytes, &tmB, bar, ks * kRowBytes, row, pol);
                    tma_3d_pair(st + S::sfb, &tmSfb, bar, 0, S::tiles * ks, 2 * nt, pol);
                }
                issued |= 1u << stage;
                issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                if (++stage == S::count) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (failed) {
            if (lane == 0) set_device_error(p.err, NVFP4_ERR_DEVICE_TIMEOUT);
            *abort_flag = 1;
            // the leader's barriers count the copies of both CTAs; the peer stays until the leader is done
            if (rank == 0) {
                for (int s = 0; s < S::count; ++s) {
                    if (issued & (1u << s)) mbar_wait_cluster(&full[s], (issued_parity >> s) & 1u, nullptr, kWaitBudgetCycles);
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (the leader's)
        if (rank == 0) {
            const uint32_t idesc = idesc_fp4(kMx, 256, kPairN);
            const uint32_t base = smem_u32(smem);
            int stage = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool issued_any = false;
            for (int64_t t = first; t < p.tiles && !failed; t += step) {
                const bool ok = mbar_wait_cluster(&tmem_empty, acc_phase ^ 1u, abort_flag, kWaitBudgetCycles);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    failed = true;
                    break;
                }
                acc_phase ^= 1u;
                tc_fence_after();
                for (int ks = 0; ks < num_ks; ++ks) {
                    const bool okf = mbar_wait_cluster(&full[stage], phase, abort_flag, kWaitBudgetCycles);
                    if (!__all_sync(0xFFFFFFFFu, okf)) {
                        failed = true;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t st = base + stage * S::bytes;
                    issue_stage<kMx, true>(tmem, sdesc_k_swizzled<kRowBytes>(st), sdesc_k_swizzled<kRowBytes>(st + kHalfBytes),
                                           idesc, sdesc_sf(st + S::sfa), sdesc_sf(st + S::sfb),
                                           sdesc_sf(st + S::sfb + S::tiles * kSfAtomBytes), tmem + kAccCols + stage * S::sf_cols, 0,
                                           min(kStageK / 64, (p.K - kStageK * ks + 63) / 64), ks != 0);
                    issued_any = true;
                    commit_pair(&empty[stage]);
                    if (++stage == S::count) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (failed) break;
                commit_pair(&tmem_full);
            }
            if (failed) {
                if (lane == 0) set_device_error(p.err, NVFP4_ERR_DEVICE_TIMEOUT);
                *abort_flag = 1;
                if (issued_any) {   // the MMAs already issued complete before either CTA's memory goes
                    commit_pair(&drain);
                    mbar_wait_cluster(&drain, 0, nullptr, kWaitBudgetCycles);
                }
            }
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------ epilogue
        pdl_wait();                                   // before a_g is read
        const int q = warp & 3, sub = (warp - 4) >> 2;
        const uint32_t taddr = tmem + 64 * sub + (static_cast<uint32_t>(q * 32) << 16);
        const uint32_t empty_bar = leader_addr(&tmem_empty);
        float* gcol = s_col[warp - 4][0];
        float* bcol = gcol + 64;
        uint8_t* buf = smem + S::out + (warp - 4) * kOutBytes;
        uint32_t acc_phase = 0;
        for (int64_t t = first; t < p.tiles; t += step) {
            const int row0 = static_cast<int>(t / p.n_tiles) * 256 + 128 * static_cast<int>(rank) + q * 32;
            const int n0 = static_cast<int>(t % p.n_tiles) * kPairN + 64 * sub;
            const float ga = !kMx && row0 + lane < p.T ? __ldg(p.a_g + row0 + lane) : 1.0f;
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 64; h += 32) {
                const int n = n0 + h + lane;
                if (!kMx) gcol[h + lane] = n < p.N ? __ldg(p.b_g + n) : 0.0f;
                if (p.bias != nullptr) bcol[h + lane] = n < p.N ? __ldg(p.bias + n) : 0.0f;
            }
            __syncwarp();
            const bool ok = mbar_wait_cluster(&tmem_full, acc_phase, abort_flag, kWaitBudgetCycles);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                if (lane == 0) set_device_error(p.err, NVFP4_ERR_DEVICE_TIMEOUT);
                *abort_flag = 1;
                break;
            }
            acc_phase ^= 1u;
            tc_fence_after();
            uint32_t v[64];
            tmem_ld_32x32b_x32(taddr, *reinterpret_cast<uint32_t(*)[32]>(v));
            tmem_ld_32x32b_x32(taddr + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_leader(empty_bar);
            if (row0 >= p.T || n0 >= p.N) continue;    // the whole warp
            // the column quarters' stores spread over the next tile's main loop (about half of it), if there is one:
            // all at once, in every SM at about the same time, they hold its loads up (8192^3 MXFP4 176.5 -> 171 us of a
            // call on the device, with FP32 outputs 201.5 -> 192.5; 32768 x 4096 x 1536 NVFP4 108.5 -> 106.5 and 142.5 -> 135.5;
            // 16384 x 4096 x 512 30.7 -> 29.9; 4096 x 4096 x 65536 452 and 454; spread over all of the main loop no
            // better).  Outputs that go row by row take long enough by themselves (with the delay 8192 x 1999 x 2048 27.2 ->
            // 28.4 us, 16384 x 4095 x 1024 NVFP4 to FP32 91 -> 103).
            if (kStaged && t + step < p.tiles) {
                const uint32_t start = cycles32();
                while (cycles32() - start < static_cast<uint32_t>(sub * num_ks * 64)) __nanosleep(64);
            }
            if constexpr (kStaged) {
                if (p.out_type == NVFP4_TYPE_BF16) outputs_staged<kMx, __nv_bfloat16>(v, ga, gcol, bcol, buf, &tmOut, n0, row0, p);
                else if (p.out_type == NVFP4_TYPE_F32) outputs_staged<kMx, float>(v, ga, gcol, bcol, buf, &tmOut, n0, row0, p);
                else outputs_staged<kMx, __half>(v, ga, gcol, bcol, buf, &tmOut, n0, row0, p);
            } else {
                const int rows = static_cast<int>(min(p.T - row0, static_cast<int64_t>(32)));
                if (p.out_type == NVFP4_TYPE_BF16)
                    write_by_row<kMx, __nv_bfloat16, 64, 64>(v, ga, gcol, bcol, buf, row0, n0, rows, p);
                else if (p.out_type == NVFP4_TYPE_F32)
                    write_by_row<kMx, float, 64, 32>(v, ga, gcol, bcol, buf, row0, n0, rows, p);
                else
                    write_by_row<kMx, __half, 64, 64>(v, ga, gcol, bcol, buf, row0, n0, rows, p);
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();                                   // no signal or MMA of one CTA reaches the other after this
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// Map over out [T][N] for stores of 32 rows x 128 bytes (rows on 16-byte boundaries).
bool make_out_map(CUtensorMap* m, const LinearArgs& a) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const int size = a.out_type == NVFP4_TYPE_F32 ? 4 : 2;
    const CUtensorMapDataType type = a.out_type == NVFP4_TYPE_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : a.out_type == NVFP4_TYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                                     : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.N), static_cast<cuuint64_t>(a.T)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.ldo * size)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / size), 32};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, type, 2, a.out, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kMx, bool kStaged>
cudaError_t launch_pair(const LinearArgs& a, cudaStream_t st, bool pdl) {
    using S = PairStage<kMx>;
    static bool ready[kMaxDevices];
    cudaError_t e = prepare(linear_pair_kernel<kMx, kStaged>, S::dynamic, ready);
    if (e != cudaSuccess) return e;
    PairParams p{};
    p.T = a.T;
    p.N = a.N;
    p.K = a.K;
    p.a_g = a.a_g;
    p.b_g = a.b_g;
    p.bias = a.bias;
    p.out = a.out;
    p.out_type = a.out_type;
    p.ldo = a.ldo;
    p.align = out_align(a);
    p.err = a.err;
    p.n_tiles = (a.N + kPairN - 1) / kPairN;
    p.tiles = (a.T + 255) / 256 * p.n_tiles;
    const int64_t sf_tiles = (a.K + Format<kMx>::tile_k - 1) / Format<kMx>::tile_k;
    CUtensorMap ma, mb, msa, msb, mo = {};
    if (kStaged && !make_out_map(&mo, a)) return cudaErrorInvalidValue;
    if (!make_map(&ma, a.a_codes, a.T, a.K / 2, 128) || !make_map(&mb, a.b_codes, a.N, a.K / 2, 128) ||
        !make_sf_map(&msa, a.a_sf, (a.T + 127) / 128, sf_tiles, S::tiles, 1) ||
        !make_sf_map(&msb, a.b_sf, (a.N + 127) / 128, sf_tiles, S::tiles, 2))
        return cudaErrorInvalidValue;
    const int64_t pairs = linear_pair_count();
    const unsigned grid = static_cast<unsigned>(2 * (p.tiles < pairs ? p.tiles : pairs));
    return launch_pdl(pdl, linear_pair_kernel<kMx, kStaged>, grid, kPairThreads, S::dynamic, st, ma, mb, msa, msb, mo, p);
}

}  // namespace

// Pairs of CTAs that the device runs at once (asked once per device).
int linear_pair_count() {
    static int count[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 1;
    static bool ready[kMaxDevices];
    if (prepare(linear_pair_kernel<false, true>, PairStage<false>::dynamic, ready) != cudaSuccess) return 1;
    std::lock_guard<std::mutex> lock(g_linear_mutex);
    if (!count[dev]) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = 2 * device_sm_count();
        cfg.blockDim = kPairThreads;
        cfg.dynamicSmemBytes = PairStage<false>::dynamic;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, linear_pair_kernel<false, true>, &cfg) != cudaSuccess || n < 1) n = device_sm_count() / 2;
        count[dev] = n < 1 ? 1 : n;
    }
    return count[dev];
}

cudaError_t launch_linear_pair(const LinearArgs& a, cudaStream_t st, bool pdl) {
    // A TMA store writes whole 16-byte units: of a row that ends inside one it would also write what lies behind.
    const bool staged = out_align(a) > 0 && static_cast<int64_t>(a.N) * (a.out_type == NVFP4_TYPE_F32 ? 4 : 2) % 16 == 0;
    if (staged) return a.mx ? launch_pair<true, true>(a, st, pdl) : launch_pair<false, true>(a, st, pdl);
    return a.mx ? launch_pair<true, false>(a, st, pdl) : launch_pair<false, false>(a, st, pdl);
}

}  // namespace nvfp4
