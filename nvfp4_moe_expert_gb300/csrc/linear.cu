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
#include "linear.cuh"
#include "mxfp4_quant.cuh"
#include "nvfp4_quant.cuh"

namespace nvfp4 {
namespace {

constexpr int kMaxStages = 12;
constexpr int kEpiWarps = 4;
constexpr int kThreads = 32 * (2 + kEpiWarps);

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
    int align;            // of out's rows: out_align()
    int a_rows;           // rows of A loaded per tile (a multiple of 8, at most 128)
    int stages, stage_bytes;
    int n_tiles;
    int64_t tiles;
    int* err;
};

// BN outputs of row r from the accumulator's columns at taddr (this warp's lanes): outer scales
// (ga: the row's), bias, one rounding.  gcol, bcol: the warp's 32 column values in shared memory.
template <bool kMx, int BN, typename P>
__device__ __forceinline__ void epilogue_row(uint32_t taddr, bool live, int64_t r, int n0, float ga, const P& p, float* gcol,
                                             float* bcol) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int c = 0; c < BN; c += 32) {
        const int n = n0 + c + lane;
        uint32_t v[32];
        tmem_ld_32x32b_x32(taddr + c, v);
        __syncwarp();
        gcol[lane] = !kMx && n < p.N ? __ldg(p.b_g + n) : 1.0f;
        bcol[lane] = p.bias != nullptr && n < p.N ? __ldg(p.bias + n) : 0.0f;
        __syncwarp();
        tmem_ld_wait();
        if (live && n0 + c < p.N) write_outputs<kMx, 32>(v, ga, gcol, bcol, r, n0 + c, p);
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
    __shared__ __align__(8) float s_col[kEpiWarps][2][32];
    volatile int* abort_flag = &abort_word;
    const int warp = warp_index(), lane = threadIdx.x & 31;
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
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(tmem_slot);
    const int num_ks = (p.K + kStageK - 1) / kStageK;
    const int sf_tiles = (p.K + F::tile_k - 1) / F::tile_k;        // scale tiles of a 128-row set, all of K
    bool failed = false;

    if (warp == 0) {
        const uint64_t pol_a = policy_evict_last(), pol_b = policy_evict_normal();
        int stage = 0;
        uint32_t phase = 0, issued = 0, issued_parity = 0;
        auto load_b = [&](int n0, int ks) {
            uint8_t* b = smem + stage * p.stage_bytes + a_bytes;
            const uint32_t sf_bytes = static_cast<uint32_t>(min(F::tiles, sf_tiles - F::tiles * ks)) * kSfAtomBytes;
            // the second set of a BN = 256 tile is past the end of B when N has none
            const int sets = kSfbSets == 2 && n0 + 128 < p.N ? 2 : 1;
            mbar_arrive_expect_tx_elect(&full[stage], a_bytes + BN * kRowBytes + (1 + sets) * sf_bytes);
            tma_load_2d_elect(b + (n0 & (kN - BN)) * kRowBytes, &tmB, &full[stage], ks * kRowBytes, n0, pol_b);
            for (int i = 0; i < sets; ++i)
                bulk_load_elect(b + kBBytes + (1 + i) * kSfSet,
                                p.b_sf + (static_cast<int64_t>(n0 / 128 + i) * sf_tiles + F::tiles * ks) * kSfAtomBytes,
                                sf_bytes, &full[stage], pol_b);
            issued |= 1u << stage;
            issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
        };
        auto load_a = [&](int64_t mt, int ks) {
            uint8_t* a = smem + stage * p.stage_bytes;
            const uint32_t sf_bytes = static_cast<uint32_t>(min(F::tiles, sf_tiles - F::tiles * ks)) * kSfAtomBytes;
            tma_load_2d_elect(a, &tmA, &full[stage], ks * kRowBytes, static_cast<int>(mt * kBM), pol_a);
            bulk_load_elect(a + a_bytes + kBBytes, p.a_sf + (mt * sf_tiles + F::tiles * ks) * kSfAtomBytes, sf_bytes,
                            &full[stage], pol_a);
        };
        // the weights are the call's input: their first stages load while x is still being quantised
        const int early = min(p.stages, num_ks);
        for (int ks = 0; ks < early; ++ks) {
            load_b(static_cast<int>(blockIdx.x % p.n_tiles) * BN, ks);
            ++stage;
        }
        stage = 0;
        pdl_wait();
        for (int64_t t = blockIdx.x; t < p.tiles && !failed; t += gridDim.x) {
            const int64_t mt = t / p.n_tiles;
            const int n0 = static_cast<int>(t % p.n_tiles) * BN;
            for (int ks = 0; ks < num_ks; ++ks) {
                if (t != blockIdx.x || ks >= early) {
                    const bool ok = mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, kWaitBudgetCycles);
                    if (!__all_sync(0xFFFFFFFFu, ok)) {
                        failed = true;
                        break;
                    }
                    load_b(n0, ks);
                }
                load_a(mt, ks);
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
                const uint32_t sf = st + a_bytes + kBBytes;
                const int nk = min(kStageK / 64, (p.K - kStageK * ks + 63) / 64);
                issue_stage<kMx, kSfbSets, 1>(tmem + acc * kN, sdesc_k_swizzled<kRowBytes>(st),
                                           sdesc_k_swizzled<kRowBytes>(st + a_bytes), idesc, sdesc_sf(sf),
                                           sdesc_sf(sf + kSfSet), sdesc_sf(sf + kSfbSets * kSfSet), sf0 + stage * kSfCols,
                                           sfb_col, nk, ks != 0);
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
        pdl_wait();                                                // before a_g is read
        const int q = warp & 3;                                    // TMEM lane quarter
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
            epilogue_row<kMx, BN>(taddr, live, r, n0, ga, p, s_col[warp - 2][0], s_col[warp - 2][1]);
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

// ---------------------------------------------------------------- at most 16 tokens: one kernel
// The work is the weights' bytes, so a kernel of its own for quantising x would cost more than it
// does: every CTA quantises the few rows of x itself into shared memory, in the layout a TMA load of
// quantised rows would give (bit-equal to the row quantisers), while its weights stream in, and
// keeps them there for all its output tiles.  The MMAs are those of the general kernel (M=128, of
// which T rows are real), K in the same order.
// Warps: 0 loads weights, 1 issues the MMAs, 2-17 quantise x, then warp 4 (TMEM lanes 0-31) writes
// the outputs.
namespace decode {
constexpr int kMaxT = 16;
constexpr int kQuantWarps = 16;
constexpr int kQuantThreads = 32 * kQuantWarps;
constexpr int kThreadsD = 32 * (2 + kQuantWarps);
constexpr int kEpiWarp = 4;
constexpr int kMaxK = 8192;
constexpr int kChunkBytes = kMaxT * kRowBytes;       // one 256-element chunk of the 16 rows
constexpr int kPer = 4;                              // chunks of the weights per stage: 1024 K-elements
// A quantiser warp takes pieces of one row: 1024 columns (MXFP4, one block of 32 to a lane) or 512 (NVFP4,
// one of 16), several loaded before the first is used.  The pieces are ordered by columns, then rows, and a
// batch (all warps' pieces of one turn) becomes ready as a whole.
template <bool kMx>
__host__ __device__ constexpr int piece_cols() { return kMx ? 1024 : 512; }
template <bool kMx>
__host__ __device__ constexpr int pieces_held() { return kMx ? 1 : 4; }
template <bool kMx>
__host__ __device__ constexpr int batch_size() { return pieces_held<kMx>() * kQuantWarps; }
constexpr int kMaxBatches = 8;                       // 16 rows of 8192
static_assert(kMaxT * (kMaxK / piece_cols<true>()) <= kMaxBatches * batch_size<true>(), "batches");
static_assert(kMaxT * (kMaxK / piece_cols<false>()) <= kMaxBatches * batch_size<false>(), "batches");
constexpr int kMaxStagesD = 8;

struct DecodeParams {
    const void* x;
    int x_type;
    int64_t ldx;
    int x_align;          // of x's rows: mx_align()
    int T, N, K;
    uint32_t t_magic;     // ceil(2^16 / T): q / T = q * t_magic >> 16 for q < 4096
    const uint8_t* b_sf;
    const float* b_g;
    const float* bias;
    void* out;
    int out_type;
    int64_t ldo;
    int align;
    int stages, n_tiles;
    int* err;
};
static_assert(kMaxT * (kMaxK / piece_cols<false>()) + batch_size<false>() <= 4096, "t_magic's range (a turn may pass the last piece)");

// Piece q: its row and its place among the row's pieces.
__device__ __forceinline__ void piece(const DecodeParams& p, int q, int& r, int& i) {
    i = static_cast<int>(static_cast<uint32_t>(q) * p.t_magic >> 16);
    r = q - i * p.T;
}

// Shared-memory byte of 4-byte word w (of 32) of row r in its chunk: 128B swizzle.
__device__ __forceinline__ int swizzled(int r, int w) { return r * kRowBytes + ((((w >> 2) ^ (r & 7)) << 4) | ((w & 3) << 2)); }

__device__ __forceinline__ void sync_quantisers() { asm volatile("barrier.sync 1, %0;" ::"r"(kQuantThreads) : "memory"); }
// The CTA's start: warp 0, which has set the barriers up, does not wait for the others.
__device__ __forceinline__ void start_arrive() { asm volatile("barrier.arrive 2, %0;" ::"r"(kThreadsD) : "memory"); }
__device__ __forceinline__ void start_wait() { asm volatile("barrier.sync 2, %0;" ::"r"(kThreadsD) : "memory"); }

template <typename X, int kAlign>
__device__ __forceinline__ void quantise_mx(const DecodeParams& p, int warp, int lane, uint8_t* codes, uint8_t* sf,
                                            uint64_t* a_full) {
    constexpr int kCols = piece_cols<true>();
    const X* x = static_cast<const X*>(p.x);
    const int pieces = p.T * ((p.K + kCols - 1) / kCols);
    const int sf_cols = (p.K + kMxTileCols - 1) / kMxTileCols * kMxTileCols;   // the blocks past K get zero scales
    MxBlock<X, kAlign> held, next;
    auto load = [&](MxBlock<X, kAlign>& h, int q) {
        int r, at;
        piece(p, q, r, at);
        const int c = at * kCols + kMxBlock * lane;
        h.load(x + r * p.ldx + c, q < pieces && c < p.K);
    };
    load(held, warp);
    start_wait();                                     // the first loads are on their way before the CTA is set up
    for (int first = 0, batch = 0; first < pieces; first += kQuantWarps, ++batch) {
        const int q = first + warp;
        load(next, q + kQuantWarps);
        if (q < pieces) {
            int r, at;
            piece(p, q, r, at);
            const int c = at * kCols + kMxBlock * lane;
            uint4 word;
            uint32_t scale;
            held.quantise(word, scale, p.err);
            if (c < p.K) *reinterpret_cast<uint4*>(codes + c / kStageK * kChunkBytes + swizzled(r, 4 * (lane & 7))) = word;
            if (c < sf_cols) sf[c / kMxTileCols * kSfAtomBytes + r * 16 + (lane & 3)] = static_cast<uint8_t>(scale);
        }
        fence_proxy_async_shared();
        mbar_arrive(&a_full[batch]);
        held = next;
    }
}

// The block of 16 this lane has of piece q, or zeros.
__device__ __forceinline__ bool nv_block(const DecodeParams& p, int q, int pieces, int lane, uint4& v0, uint4& v1) {
    int r, at;
    piece(p, q, r, at);
    const int c = at * piece_cols<false>() + 16 * lane;
    const bool live = q < pieces && c < p.K;
    v0 = v1 = make_uint4(0u, 0u, 0u, 0u);
    if (live) {
        const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) + r * p.ldx + c);
        v0 = __ldg(s);
        v1 = __ldg(s + 1);
    }
    return live;
}

__device__ __forceinline__ void quantise_nv(const DecodeParams& p, int warp, int lane, uint8_t* codes, uint8_t* sf,
                                            uint32_t* row_max, float* row_g, uint64_t* a_full) {
    constexpr int kCols = piece_cols<false>(), kHeld = pieces_held<false>(), kBatch = batch_size<false>();
    const int pieces = p.T * ((p.K + kCols - 1) / kCols);
    uint4 v[kHeld][2];
    // the rows' maxima, then their outer scales; the last batch comes first, so that the first, which
    // the second pass starts with, is still held then
    const int last = (pieces - 1) / kBatch * kBatch;
    for (int first = last; first >= 0; first -= kBatch) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) nv_block(p, first + i * kQuantWarps + warp, pieces, lane, v[i][0], v[i][1]);
        if (first == last) start_wait();
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int q = first + i * kQuantWarps + warp;
            if (q >= pieces) break;                   // the whole warp
            const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, block_absmax_bits(v[i][0], v[i][1]));
            int r, at;
            piece(p, q, r, at);
            if (lane == 0) atomicMax(&row_max[r], top);
        }
    }
    sync_quantisers();
    if (warp == 0 && lane < p.T) {
        const uint32_t top = row_max[lane];
        const bool finite = top < 0x7F800000u;
        if (!finite) set_device_error(p.err, NVFP4_ERR_NONFINITE);
        row_g[lane] = finite ? __fdiv_rn(__uint_as_float(top), kOuterDivisor) : 0.0f;
    }
    sync_quantisers();
    for (int first = 0, batch = 0; first < pieces; first += kBatch, ++batch) {
        if (first > 0) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) nv_block(p, first + i * kQuantWarps + warp, pieces, lane, v[i][0], v[i][1]);
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int q = first + i * kQuantWarps + warp;
            int r, at;
            piece(p, q, r, at);
            const int c = at * kCols + 16 * lane;
            if (q >= pieces || c >= p.K) continue;
            uint32_t w0, w1, scale;
            nv_quantize16(v[i][0], v[i][1], row_g[r], w0, w1, scale);
            uint8_t* d = codes + c / kStageK * kChunkBytes + swizzled(r, (c & (kStageK - 1)) >> 3);
            *reinterpret_cast<uint2*>(d) = make_uint2(w0, w1);
            sf[c / 64 * kSfAtomBytes + r * 16 + ((c & 63) >> 4)] = static_cast<uint8_t>(scale);
        }
        fence_proxy_async_shared();
        mbar_arrive(&a_full[batch]);
    }
}

template <typename X>
__device__ __forceinline__ void quantise_mx_rows(const DecodeParams& p, int warp, int lane, uint8_t* codes, uint8_t* sf,
                                                 uint64_t* a_full) {
    if (p.x_align == 2) quantise_mx<X, 2>(p, warp, lane, codes, sf, a_full);
    else if (p.x_align == 1) quantise_mx<X, 1>(p, warp, lane, codes, sf, a_full);
    else quantise_mx<X, 0>(p, warp, lane, codes, sf, a_full);
}

// Quantise the T rows of x; warp 0..kQuantWarps-1 of the quantisers.
template <bool kMx>
__device__ __forceinline__ void quantise_x(const DecodeParams& p, int warp, int lane, uint8_t* codes, uint8_t* sf,
                                           uint32_t* row_max, float* row_g, uint64_t* a_full) {
    if (!kMx) {
        quantise_nv(p, warp, lane, codes, sf, row_max, row_g, a_full);
    } else if (p.x_type == NVFP4_TYPE_BF16) {
        quantise_mx_rows<__nv_bfloat16>(p, warp, lane, codes, sf, a_full);
    } else if (p.x_type == NVFP4_TYPE_F16) {
        quantise_mx_rows<__half>(p, warp, lane, codes, sf, a_full);
    } else {
        quantise_mx_rows<float>(p, warp, lane, codes, sf, a_full);
    }
}

template <bool kMx, int BN>
__global__ void __launch_bounds__(kThreadsD, 1)
    linear_decode_kernel(const __grid_constant__ CUtensorMap tmB, const DecodeParams p) {
    using F = Format<kMx>;
    constexpr int kN = mma_n(BN);
    constexpr int kBBytes = kN * kRowBytes;                        // codes of one chunk
    constexpr int kSfBytes = F::tiles * kSfAtomBytes;              // its scale tiles
    constexpr int kStageBytes = kPer * (kBBytes + kSfBytes);       // codes chunk by chunk, then scales
    constexpr uint32_t kSfCols = 8 * F::tiles;                     // TMEM columns of a chunk's scales
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[kMaxStagesD], empty[kMaxStagesD], a_full[kMaxBatches], tmem_full[2], tmem_empty[2], drain;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word;
    __shared__ uint32_t row_max[kMaxT];
    __shared__ float row_g[kMaxT];
    __shared__ __align__(8) float s_col[2][32];
    volatile int* abort_flag = &abort_word;
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int num_ks = (p.K + kStageK - 1) / kStageK;              // chunks of 256
    const int num_st = (num_ks + kPer - 1) / kPer;                 // stages of the weights
    const int sf_tiles = (p.K + F::tile_k - 1) / F::tile_k;
    // x: chunks of codes, then its scale tiles; the weights' stages follow, so the 128 rows an MMA
    // reads from a chunk of 16 stay inside the allocation
    uint8_t* a_codes = smem;
    uint8_t* a_sf = a_codes + num_ks * kChunkBytes;
    uint8_t* stages = a_sf + (sf_tiles * kSfAtomBytes + 1023) / 1024 * 1024;
    bool failed = false;

    if (warp == 0) {
        // one barrier of each kind to a lane: one after the other they took 1000 cycles
        static_assert(kMaxStagesD <= 32 && kMaxBatches <= 32 && kMaxT <= 32, "a lane each");
        if (lane < kMaxStagesD) {
            mbar_init(&full[lane], 1);
            mbar_init(&empty[lane], 1);
        }
        if (lane < kMaxBatches) mbar_init(&a_full[lane], kQuantThreads);
        if (lane < 2) {
            mbar_init(&tmem_full[lane], 1);
            mbar_init(&tmem_empty[lane], 32);
        }
        if (lane < kMaxT) row_max[lane] = 0u;
        if (lane == 0) {
            mbar_init(&drain, 1);
            abort_word = 0;
        }
        fence_barrier_init();
        __syncwarp();
        start_arrive();
        const uint64_t pol = policy_evict_normal();
        int stage = 0;
        uint32_t phase = 0, issued = 0, issued_parity = 0;
        for (int t = blockIdx.x; t < p.n_tiles && !failed; t += gridDim.x) {
            const int n0 = t * BN;
            const uint8_t* bsf = p.b_sf + static_cast<int64_t>(n0 / 128) * sf_tiles * kSfAtomBytes;
            for (int st = 0; st < num_st; ++st) {
                const bool ok = mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, kWaitBudgetCycles);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    failed = true;
                    break;
                }
                uint8_t* b = stages + stage * kStageBytes;
                uint8_t* box = b + (n0 & (kN - BN)) * kRowBytes;
                const int chunks = min(kPer, num_ks - kPer * st);
                const uint32_t sf_bytes = static_cast<uint32_t>(min(kPer * F::tiles, sf_tiles - kPer * F::tiles * st)) * kSfAtomBytes;
                load_operand_elect(&full[stage], chunks * BN * kRowBytes + sf_bytes, box, &tmB, kPer * st * kRowBytes, n0,
                                   b + kPer * kBBytes, bsf + kPer * F::tiles * st * kSfAtomBytes, sf_bytes, pol);
                for (int i = 1; i < chunks; ++i)
                    tma_load_2d_elect(box + i * kBBytes, &tmB, &full[stage], (kPer * st + i) * kRowBytes, n0, pol);
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
        tmem_alloc(&tmem_slot, kTmemCols);
        tmem_relinquish();
        tc_fence_before();
        start_wait();
        tc_fence_after();
        const uint32_t tmem = uniform(tmem_slot);
        const uint32_t idesc = idesc_fp4(kMx, kBM, kN);
        const uint32_t sf0 = tmem + 2 * kN;
        const uint32_t a_base = smem_u32(a_codes), a_sf_base = smem_u32(a_sf), b_base = smem_u32(stages);
        int stage = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool issued_any = false;
        int batch = 0;                                   // batches of x known to be ready
        const bool reused = p.stages < num_st || p.n_tiles > static_cast<int>(gridDim.x);   // stages are filled again
        for (int t = blockIdx.x; t < p.n_tiles && !failed; t += gridDim.x) {
            const uint32_t sfb_col = kN == 64 ? static_cast<uint32_t>((t * BN) & 64) / 32 : 0u;
            const bool ok = mbar_wait_bounded(&tmem_empty[acc], acc_phase ^ 1u, abort_flag, kWaitBudgetCycles);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                failed = true;
                break;
            }
            for (int st = 0; st < num_st; ++st) {
                const int chunks = min(kPer, num_ks - kPer * st);
                bool okf = true;
                if (t == static_cast<int>(blockIdx.x)) {   // the batches that complete x's columns of this stage
                    const int whole = (kPer * st + chunks + piece_cols<kMx>() / kStageK - 1) / (piece_cols<kMx>() / kStageK);
                    const int need = (whole * p.T - 1) / batch_size<kMx>() + 1;
                    while (okf && batch < need)
                        okf = mbar_wait_bounded(&a_full[batch++], 0, abort_flag, kWaitBudgetCycles);
                }
                okf = okf && mbar_wait_bounded(&full[stage], phase, abort_flag, kWaitBudgetCycles);
                if (!__all_sync(0xFFFFFFFFu, okf)) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                const uint32_t b = b_base + stage * kStageBytes;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    if (i >= chunks) break;
                    const int ks = kPer * st + i;
                    issue_stage<kMx, 1, 1>(tmem + acc * kN, sdesc_k_swizzled<kRowBytes>(a_base + ks * kChunkBytes),
                                        sdesc_k_swizzled<kRowBytes>(b + i * kBBytes), idesc,
                                        sdesc_sf(a_sf_base + ks * kSfBytes), sdesc_sf(b + kPer * kBBytes + i * kSfBytes), 0,
                                        sf0 + (kPer * stage + i) * kSfCols, sfb_col, min(kStageK / 64, (p.K - kStageK * ks + 63) / 64),
                                        ks != 0);
                }
                issued_any = true;
                if (reused) tc_commit_elect(&empty[stage]);
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (failed) break;
            tc_commit_elect(&tmem_full[acc]);
            if (++acc == 2) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
        if (failed) {
            if (lane == 0) set_device_error(p.err, NVFP4_ERR_DEVICE_TIMEOUT);
            *abort_flag = 1;
            if (issued_any) {
                tc_commit_elect(&drain);
                mbar_wait_bounded(&drain, 0, nullptr, kWaitBudgetCycles);
            }
        }
    } else {
        quantise_x<kMx>(p, warp - 2, lane, a_codes, a_sf, row_max, row_g, a_full);
        if (warp == kEpiWarp) {
            tc_fence_after();
            const uint32_t tmem = uniform(tmem_slot);                   // written before the CTA's start
            const float ga = !kMx && lane < p.T ? row_g[lane] : 1.0f;   // before the quantisers' barrier
            int acc = 0;
            uint32_t acc_phase = 0;
            for (int t = blockIdx.x; t < p.n_tiles; t += gridDim.x) {
                const int n0 = t * BN;
                const bool ok = mbar_wait_bounded(&tmem_full[acc], acc_phase, abort_flag, kWaitBudgetCycles);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    if (lane == 0) set_device_error(p.err, NVFP4_ERR_DEVICE_TIMEOUT);
                    *abort_flag = 1;
                    break;
                }
                tc_fence_after();
                epilogue_row<kMx, BN>(tmem + acc * kN + (n0 & (kN - BN)), lane < p.T, lane, n0, ga, p, s_col[0], s_col[1]);
                tc_fence_before();
                mbar_arrive(&tmem_empty[acc]);
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(uniform(tmem_slot), kTmemCols);
    }
}
}  // namespace decode

template <bool kMx, int BN>
cudaError_t launch_decode(const LinearInput& x, const LinearArgs& a, cudaStream_t st) {
    using namespace decode;
    using F = Format<kMx>;
    static bool ready[kMaxDevices];
    cudaError_t e = prepare(linear_decode_kernel<kMx, BN>, kSmemLimit - kFixedBytes, ready);
    if (e != cudaSuccess) return e;
    DecodeParams p{};
    p.x = x.x;
    p.x_type = x.type;
    p.ldx = x.ld;
    p.x_align = mx_align(x.x, x.ld, x.type == NVFP4_TYPE_F32 ? 4 : 2);
    p.T = static_cast<int>(a.T);
    p.t_magic = (65536u + p.T - 1) / p.T;
    p.N = a.N;
    p.K = a.K;
    p.b_sf = a.b_sf;
    p.b_g = a.b_g;
    p.bias = a.bias;
    p.out = a.out;
    p.out_type = a.out_type;
    p.ldo = a.ldo;
    p.align = out_align(a);
    p.err = a.err;
    const int num_ks = (a.K + kStageK - 1) / kStageK, num_st = (num_ks + kPer - 1) / kPer;
    const int sf_bytes = (a.K + F::tile_k - 1) / F::tile_k * kSfAtomBytes;
    const int x_bytes = num_ks * kChunkBytes + (sf_bytes + 1023) / 1024 * 1024;
    const int stage_bytes = kPer * (mma_n(BN) * kRowBytes + F::tiles * kSfAtomBytes);
    // an MMA reads 128 rows from x's last chunk: a stage lies behind it
    static_assert(kPer * mma_n(BN) * kRowBytes >= kBM * kRowBytes, "rows an MMA reads past x");
    p.n_tiles = (a.N + BN - 1) / BN;
    const int sms = device_sm_count();
    const int grid = p.n_tiles < sms ? p.n_tiles : sms;
    p.stages = (kSmemLimit - kFixedBytes - 1024 - x_bytes) / stage_bytes;
    const int by_tmem = static_cast<int>(kTmemCols - 2 * mma_n(BN)) / (8 * kPer * F::tiles);
    if (p.stages > kMaxStagesD) p.stages = kMaxStagesD;
    if (p.stages > by_tmem) p.stages = by_tmem;
    if (p.n_tiles <= sms && p.stages > num_st) p.stages = num_st;
    const size_t smem = static_cast<size_t>(x_bytes) + static_cast<size_t>(p.stages) * stage_bytes + 1024;
    CUtensorMap mb;
    if (!make_map(&mb, a.b_codes, a.N, a.K / 2, BN)) return cudaErrorInvalidValue;
    return launch_pdl(false, linear_decode_kernel<kMx, BN>, grid, kThreadsD, smem, st, mb, p);
}

template <bool kMx, int BN>
cudaError_t launch(const LinearArgs& a, cudaStream_t st, bool pdl) {
    static bool ready[kMaxDevices];
    cudaError_t e = prepare(linear_fp4_kernel<kMx, BN>, kSmemLimit - kFixedBytes, ready);
    if (e != cudaSuccess) return e;
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
    p.align = out_align(a);
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

bool linear_quantises_x(const LinearArgs& a) { return a.T <= decode::kMaxT && a.K <= decode::kMaxK; }

cudaError_t launch_linear_x(const LinearInput& x, const LinearArgs& a, cudaStream_t st) {
    // a tile takes the time of its MMAs' issue, about the same for 32 and 64 outputs and a fifth more
    // for 128: the narrowest tile that needs the fewest rounds over the SMs
    const int sms = device_sm_count();
    if (a.N <= 32 * sms) return a.mx ? launch_decode<true, 32>(x, a, st) : launch_decode<false, 32>(x, a, st);
    if (a.N <= 64 * sms) return a.mx ? launch_decode<true, 64>(x, a, st) : launch_decode<false, 64>(x, a, st);
    return a.mx ? launch_decode<true, 128>(x, a, st) : launch_decode<false, 128>(x, a, st);
}

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t st, bool pdl) {
    if ((a.T + 255) / 256 * ((a.N + 255) / 256) >= linear_pair_count()) return launch_linear_pair(a, st, pdl);
    return a.mx ? by_tile<true>(a, st, pdl) : by_tile<false>(a, st, pdl);
}

}  // namespace nvfp4
