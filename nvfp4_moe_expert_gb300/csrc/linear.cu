// Dense 4-bit product out[t, n] = sum_k a[t, k] b[n, k] (+ bias[n]) of quantised rows on tcgen05.
//
//   NVFP4: acc = sum_k (qa*sa)[t,k] (qb*sb)[n,k] (E4M3 scales per 16), out = (acc*ga[t])*gb[n] + bias
//   MXFP4: acc = the same with E8M0 scales per 32 and no outer scales
//
// Three kernels: for few elements of x one that quantises them itself, below (linear_quantises_x); for many tiles
// a pair of CTAs to each (linear_pair.cu); between them the general one here (launch_linear chooses by time).
//
// General kernel (sm_103a): one CTA per SM walks the (128 tokens x BN outputs) tiles.  Warps 0 and 6 load the stages'
// 512 K-elements of A and B through TMA (128B swizzle) with their 512-byte scale tiles; warp 1 copies the scales to
// TMEM and issues the K=64 MMAs (M=128, N=BN) into one of two FP32 TMEM accumulators; warps 2-5 apply the outer scales
// and the bias and write their rows.  All waits are bounded (NVFP4_ERR_DEVICE_TIMEOUT, then a clean exit).
//
// What bounds it: the way of the operands into the SM.  64 x 8192 x 8192 MXFP4 take 11.9 us on the device, 2.0 of them the
// quantisation of x, for 37 MB of weights (5.5 us at the copy rate): 128 SMs have a tile each and take in a row of x for
// every row of the weights.  512 x 4096 x 8192: 14.2 us, 2.9 of them x, 2.4 PFLOP/s.
//
// K is walked 0..K-1 in 64-wide steps into one accumulator whatever the kernel and the tile, so a token's output
// does not depend on how many tokens there are.
#include "linear.cuh"
#include "mxfp4_quant.cuh"
#include "nvfp4_quant.cuh"

namespace nvfp4 {
namespace {

constexpr int kMaxStages = 8;
constexpr int kPer = 2;                              // chunks of 256 K-elements per stage
constexpr int kEpiWarps = 4;
constexpr int kOutBuf = 2048;                        // an epilogue warp's 32 rows of 16 outputs
constexpr int kWarpB = 2 + kEpiWarps;                // the producer of B
constexpr int kThreads = 32 * (kWarpB + 1);

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
    int a_rows;           // rows of A loaded per tile (a multiple of 16, at most 128)
    int stages, stage_bytes;
    int n_tiles;
    int64_t tiles;
    int* err;
};

// BN outputs of `rows` rows from row0 on, a lane each, from the accumulator's columns at taddr: outer scales (ga: this
// lane's row's), bias, one rounding.  gcol, bcol: the warp's 32 column values, in shared memory.  buf: 2 KB of it for
// outputs row by row where rows lie on no 16-byte boundary; nullptr: each lane its own row all the same, which is
// faster for the few rows of linear_decode_kernel (16 x 8191 x 2048 6.4 and 7.5 us).
template <bool kMx, int BN, typename P>
__device__ __forceinline__ void epilogue_rows(uint32_t taddr, int64_t row0, int rows, int n0, float ga, const P& p,
                                              float* gcol, float* bcol, uint8_t* buf) {
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
        if (n0 + c >= p.N || rows <= 0) continue;     // the whole warp
        if (p.align > 0 || buf == nullptr) {
            if (lane < rows) write_outputs<kMx, 32>(v, ga, gcol, bcol, row0 + lane, n0 + c, p);
        } else if (p.out_type == NVFP4_TYPE_BF16) {
            write_by_row<kMx, __nv_bfloat16, 32, 16>(v, ga, gcol, bcol, buf, row0, n0 + c, rows, p);
        } else if (p.out_type == NVFP4_TYPE_F32) {
            write_by_row<kMx, float, 32, 16>(v, ga, gcol, bcol, buf, row0, n0 + c, rows, p);
        } else {
            write_by_row<kMx, __half, 32, 16>(v, ga, gcol, bcol, buf, row0, n0 + c, rows, p);
        }
    }
}

template <bool kMx, int BN>
__global__ void __launch_bounds__(kThreads, 1)
    linear_fp4_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const Params p) {
    using F = Format<kMx>;
    constexpr int kSfBytes = F::tiles * kSfAtomBytes;              // scale tiles of a chunk
    constexpr uint32_t kSfCols = 8 * F::tiles;                     // TMEM columns of a chunk's scales
    constexpr int kN = mma_n(BN);
    constexpr int kBBytes = kN * kRowBytes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], tmem_full[2], tmem_empty[2], drain;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word;
    __shared__ __align__(8) float s_col[kEpiWarps][2][32];
    __shared__ __align__(16) uint8_t s_out[kEpiWarps][kOutBuf];
    volatile int* abort_flag = &abort_word;
    const int warp = warp_index(), lane = threadIdx.x & 31;
    // a stage: A's chunks, B's chunks, then their scale tiles
    const int a_bytes = p.a_rows * kRowBytes;
    const int b_off = kPer * a_bytes, sfa_off = b_off + kPer * kBBytes, sfb_off = sfa_off + kPer * kSfBytes;

    if (warp == 0) {
        if (lane < kMaxStages) {
            mbar_init(&full[lane], 2);                             // both producers
            mbar_init(&empty[lane], 1);
        }
        if (lane < 2) {
            mbar_init(&tmem_full[lane], 1);
            mbar_init(&tmem_empty[lane], 32 * kEpiWarps);
        }
        if (lane == 0) {
            mbar_init(&drain, 1);
            abort_word = 0;
            prefetch_tensormap(&tmA);
            prefetch_tensormap(&tmB);
        }
        fence_barrier_init();
    } else if (warp == 1) {
        tmem_alloc(&tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(tmem_slot);
    const int num_ks = (p.K + kStageK - 1) / kStageK, num_st = (num_ks + kPer - 1) / kPer;
    const int sf_tiles = (p.K + F::tile_k - 1) / F::tile_k;        // scale tiles of a 128-row set, all of K
    bool failed = false;

    if (warp == 0 || warp == kWarpB) {
        const bool is_a = warp == 0;
        const uint64_t pol = is_a ? policy_evict_last() : policy_evict_normal();
        const CUtensorMap* map = is_a ? &tmA : &tmB;
        const uint8_t* sf = is_a ? p.a_sf : p.b_sf;
        const int box = is_a ? a_bytes : BN * kRowBytes, pitch = is_a ? a_bytes : kBBytes;
        const int off = is_a ? 0 : b_off, sf_at = is_a ? sfa_off : sfb_off;
        int stage = 0;
        uint32_t phase = 0, issued = 0, issued_parity = 0;
        if (is_a) pdl_wait();                         // A is what the kernel before writes; B is the call's input
        for (int64_t t = blockIdx.x; t < p.tiles && !failed; t += gridDim.x) {
            const int nt = static_cast<int>(t % p.n_tiles);
            const int row = is_a ? static_cast<int>(t / p.n_tiles * kBM) : nt * BN;
            const uint8_t* tile_sf = sf + static_cast<int64_t>(row / 128) * sf_tiles * kSfAtomBytes;
            const int skip = is_a ? 0 : (row & (kN - BN)) * kRowBytes;
            for (int st = 0; st < num_st; ++st) {
                const bool ok = mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, kWaitBudgetCycles);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    failed = true;
                    break;
                }
                uint8_t* base = smem + stage * p.stage_bytes;
                const int chunks = min(kPer, num_ks - kPer * st);
                const uint32_t sf_bytes =
                    static_cast<uint32_t>(min(kPer * F::tiles, sf_tiles - kPer * F::tiles * st)) * kSfAtomBytes;
                load_operand_elect(&full[stage], chunks * box + sf_bytes, base + off + skip, map, kPer * st * kRowBytes, row,
                                   base + sf_at, tile_sf + kPer * F::tiles * st * kSfAtomBytes, sf_bytes, pol);
                if (chunks == 2)
                    tma_load_2d_elect(base + off + skip + pitch, map, &full[stage], (kPer * st + 1) * kRowBytes, row, pol);
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
            // let the copies in flight land before the CTA's shared memory goes away (a stage that the other
            // producer never filled runs out its bounded wait)
            for (int s = 0; s < p.stages; ++s) {
                if (issued & (1u << s)) mbar_wait_bounded(&full[s], (issued_parity >> s) & 1u, nullptr, kWaitBudgetCycles);
            }
        }
    } else if (warp == 1) {
        const uint32_t idesc = idesc_fp4(kMx, kBM, kN);
        const uint32_t sf0 = tmem + 2 * kN, base = smem_u32(smem);
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
            for (int st = 0; st < num_st; ++st) {
                const bool okf = mbar_wait_bounded(&full[stage], phase, abort_flag, kWaitBudgetCycles);
                if (!__all_sync(0xFFFFFFFFu, okf)) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                const uint32_t at = base + stage * p.stage_bytes;
                const int chunks = min(kPer, num_ks - kPer * st);
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    if (i >= chunks) break;
                    const int ks = kPer * st + i;
                    issue_stage<kMx, false>(tmem + acc * kN, sdesc_k_swizzled<kRowBytes>(at + i * a_bytes),
                                           sdesc_k_swizzled<kRowBytes>(at + b_off + i * kBBytes), idesc,
                                           sdesc_sf(at + sfa_off + i * kSfBytes), sdesc_sf(at + sfb_off + i * kSfBytes), 0,
                                           sf0 + (kPer * stage + i) * kSfCols, sfb_col,
                                           min(kStageK / 64, (p.K - kStageK * ks + 63) / 64), ks != 0);
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
            if (++acc == 2) {
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
            const int64_t row0 = t / p.n_tiles * kBM + q * 32;
            const int n0 = static_cast<int>(t % p.n_tiles) * BN;
            const int rows = static_cast<int>(min(p.T - row0, static_cast<int64_t>(32)));
            const float ga = !kMx && lane < rows ? __ldg(p.a_g + row0 + lane) : 1.0f;
            const bool ok = mbar_wait_bounded(&tmem_full[acc], acc_phase, abort_flag, kWaitBudgetCycles);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                if (lane == 0) set_device_error(p.err, NVFP4_ERR_DEVICE_TIMEOUT);
                *abort_flag = 1;
                break;
            }
            tc_fence_after();
            const uint32_t taddr = tmem + acc * kN + (n0 & (kN - BN)) + (static_cast<uint32_t>(q * 32) << 16);
            epilogue_rows<kMx, BN>(taddr, row0, rows, n0, ga, p, s_col[warp - 2][0], s_col[warp - 2][1], s_out[warp - 2]);
            tc_fence_before();
            mbar_arrive(&tmem_empty[acc]);
            if (++acc == 2) {
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

// ---------------------------------------------------------------- few tokens: one kernel
// The work is the weights' bytes, so a kernel of its own for quantising x would cost more than it
// does: every CTA quantises the few rows of x itself into shared memory, in the layout a TMA load of
// quantised rows would give (bit-equal to the row quantisers), while its weights stream in, and
// keeps them there for all its output tiles.  The MMAs are those of the general kernel (M=128, of
// which T rows are real), K in the same order.
// Warps: 0 loads weights, 1 issues the MMAs, 2-17 quantise x, then warp 4 (TMEM lanes 0-31) writes
// the outputs.
//
// Bound by latency, one thing after the other: the CTA's start, the first loads, the quantisation, the MMAs, the
// outputs.  One token through 4096 x 4096 MXFP4 (8.9 MB) 5.3 us, 16 through 1536 x 2048 NVFP4 6.6 us.
namespace decode {
constexpr int kMaxT = 16;
constexpr int kQuantWarps = 16;
constexpr int kQuantThreads = 32 * kQuantWarps;
constexpr int kThreadsD = 32 * (2 + kQuantWarps);
constexpr int kEpiWarp = 4;
constexpr int kMaxK = 8192;
constexpr int kChunkBytes = kMaxT * kRowBytes;       // one 256-element chunk of the 16 rows
constexpr int kPerD = 4;                              // chunks of the weights per stage: 1024 K-elements
// A quantiser warp takes pieces of one row: 1024 columns (MXFP4, one block of 32 to a lane) or 512 (NVFP4,
// one of 16), all of them loaded before the first is used: 32768 elements of x at most (few_tokens).
template <bool kMx>
__host__ __device__ constexpr int piece_cols() { return kMx ? 1024 : 512; }
template <bool kMx>
__host__ __device__ constexpr int pieces_held() { return kMx ? 2 : 4; }
template <bool kMx>
__host__ __device__ constexpr int max_pieces() { return pieces_held<kMx>() * kQuantWarps; }

constexpr int kMaxStagesD = 8;

struct DecodeParams {
    const void* x;
    int x_type;
    int64_t ldx;
    int x_align;          // of x's rows: mx_align()
    int T, N, K;
    uint32_t t_magic;     // ceil(2^16 / T): q / T = q * t_magic >> 16 for q < 4096 (at most 64 pieces)
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
    MxBlock<X, kAlign> held[pieces_held<true>()];
#pragma unroll
    for (int i = 0; i < pieces_held<true>(); ++i) {
        const int q = i * kQuantWarps + warp;
        int r, at;
        piece(p, q, r, at);
        const int c = at * kCols + kMxBlock * lane;
        held[i].load(x + r * p.ldx + c, q < pieces && c < p.K);
    }
    start_wait();                                     // the loads are on their way before the CTA is set up
#pragma unroll
    for (int i = 0; i < pieces_held<true>(); ++i) {
        const int q = i * kQuantWarps + warp;
        if (q >= pieces) break;                       // the whole warp
        int r, at;
        piece(p, q, r, at);
        const int c = at * kCols + kMxBlock * lane;
        uint4 word;
        uint32_t scale;
        held[i].quantise(word, scale, p.err);
        if (c < p.K) *reinterpret_cast<uint4*>(codes + c / kStageK * kChunkBytes + swizzled(r, 4 * (lane & 7))) = word;
        if (c < sf_cols) sf[c / kMxTileCols * kSfAtomBytes + r * 16 + (lane & 3)] = static_cast<uint8_t>(scale);
    }
    fence_proxy_async_shared();
    mbar_arrive(a_full);
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
    constexpr int kCols = piece_cols<false>(), kHeld = pieces_held<false>();
    const int pieces = p.T * ((p.K + kCols - 1) / kCols);
    uint4 v[kHeld][2];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) nv_block(p, i * kQuantWarps + warp, pieces, lane, v[i][0], v[i][1]);
    start_wait();
    // the rows' maxima, then their outer scales
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int q = i * kQuantWarps + warp;
        if (q >= pieces) break;                       // the whole warp
        const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, block_absmax_bits(v[i][0], v[i][1]));
        int r, at;
        piece(p, q, r, at);
        if (lane == 0) atomicMax(&row_max[r], top);
    }
    sync_quantisers();
    if (warp == 0 && lane < p.T) row_g[lane] = nv_outer_scale(row_max[lane], p.err);
    sync_quantisers();
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int q = i * kQuantWarps + warp;
        int r, at;
        piece(p, q, r, at);
        const int c = at * kCols + 16 * lane;
        if (q >= pieces || c >= p.K) continue;
        uint32_t w0, w1, scale;
        nv_quantize16(v[i][0], v[i][1], __uint_as_float(block_absmax_bits(v[i][0], v[i][1])), nv_row(row_g[r]), w0, w1, scale);
        uint8_t* d = codes + c / kStageK * kChunkBytes + swizzled(r, (c & (kStageK - 1)) >> 3);
        *reinterpret_cast<uint2*>(d) = make_uint2(w0, w1);
        sf[c / 64 * kSfAtomBytes + r * 16 + ((c & 63) >> 4)] = static_cast<uint8_t>(scale);
    }
    fence_proxy_async_shared();
    mbar_arrive(a_full);
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
    constexpr int kStageBytes = kPerD * (kBBytes + kSfBytes);       // codes chunk by chunk, then scales
    constexpr uint32_t kSfCols = 8 * F::tiles;                     // TMEM columns of a chunk's scales
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[kMaxStagesD], empty[kMaxStagesD], a_full, tmem_full[2], tmem_empty[2], drain;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word;
    __shared__ uint32_t row_max[kMaxT];
    __shared__ float row_g[kMaxT];
    __shared__ __align__(8) float s_col[2][32];
    volatile int* abort_flag = &abort_word;
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int num_ks = (p.K + kStageK - 1) / kStageK;              // chunks of 256
    const int num_st = (num_ks + kPerD - 1) / kPerD;                 // stages of the weights
    const int sf_tiles = (p.K + F::tile_k - 1) / F::tile_k;
    // x: chunks of codes, then its scale tiles; the weights' stages follow, so the 128 rows an MMA
    // reads from a chunk of 16 stay inside the allocation
    uint8_t* a_codes = smem;
    uint8_t* a_sf = a_codes + num_ks * kChunkBytes;
    uint8_t* stages = a_sf + (sf_tiles * kSfAtomBytes + 1023) / 1024 * 1024;
    bool failed = false;

    if (warp == 0) {
        // one barrier of each kind to a lane: one after the other they took 1000 cycles
        static_assert(kMaxStagesD <= 32 && kMaxT <= 32, "a lane each");
        if (lane < kMaxStagesD) {
            mbar_init(&full[lane], 1);
            mbar_init(&empty[lane], 1);
        }
        if (lane < 2) {
            mbar_init(&tmem_full[lane], 1);
            mbar_init(&tmem_empty[lane], 32);
        }
        if (lane < kMaxT) row_max[lane] = 0u;
        if (lane == 0) {
            mbar_init(&a_full, kQuantThreads);
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
                const int chunks = min(kPerD, num_ks - kPerD * st);
                const uint32_t sf_bytes =
                    static_cast<uint32_t>(min(kPerD * F::tiles, sf_tiles - kPerD * F::tiles * st)) * kSfAtomBytes;
                load_operand_elect(&full[stage], chunks * BN * kRowBytes + sf_bytes, box, &tmB, kPerD * st * kRowBytes, n0,
                                   b + kPerD * kBBytes, bsf + kPerD * F::tiles * st * kSfAtomBytes, sf_bytes, pol);
                for (int i = 1; i < chunks; ++i)
                    tma_load_2d_elect(box + i * kBBytes, &tmB, &full[stage], (kPerD * st + i) * kRowBytes, n0, pol);
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
        const bool reused = p.stages < num_st || p.n_tiles > static_cast<int>(gridDim.x);   // stages are filled again
        for (int t = blockIdx.x; t < p.n_tiles && !failed; t += gridDim.x) {
            const uint32_t sfb_col = kN == 64 ? static_cast<uint32_t>((t * BN) & 64) / 32 : 0u;
            const bool ok = mbar_wait_bounded(&tmem_empty[acc], acc_phase ^ 1u, abort_flag, kWaitBudgetCycles);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                failed = true;
                break;
            }
            for (int st = 0; st < num_st; ++st) {
                const int chunks = min(kPerD, num_ks - kPerD * st);
                bool okf = true;
                if (st == 0 && t == static_cast<int>(blockIdx.x))   // x
                    okf = mbar_wait_bounded(&a_full, 0, abort_flag, kWaitBudgetCycles);
                okf = okf && mbar_wait_bounded(&full[stage], phase, abort_flag, kWaitBudgetCycles);
                if (!__all_sync(0xFFFFFFFFu, okf)) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                const uint32_t b = b_base + stage * kStageBytes;
#pragma unroll
                for (int i = 0; i < kPerD; ++i) {
                    if (i >= chunks) break;
                    const int ks = kPerD * st + i;
                    issue_stage<kMx, false>(tmem + acc * kN, sdesc_k_swizzled<kRowBytes>(a_base + ks * kChunkBytes),
                                        sdesc_k_swizzled<kRowBytes>(b + i * kBBytes), idesc,
                                        sdesc_sf(a_sf_base + ks * kSfBytes), sdesc_sf(b + kPerD * kBBytes + i * kSfBytes), 0,
                                        sf0 + (kPerD * stage + i) * kSfCols, sfb_col,
                                        min(kStageK / 64, (p.K - kStageK * ks + 63) / 64), ks != 0);
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
        quantise_x<kMx>(p, warp - 2, lane, a_codes, a_sf, row_max, row_g, &a_full);
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
                epilogue_rows<kMx, BN>(tmem + acc * kN + (n0 & (kN - BN)), 0, p.T, n0, ga, p, s_col[0], s_col[1], nullptr);
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

// Shared memory of x and of a stage of the weights, and the stages that fit.
template <bool kMx>
int decode_x_bytes(int K) {
    using F = Format<kMx>;
    const int sf_bytes = (K + F::tile_k - 1) / F::tile_k * kSfAtomBytes;
    return (K + kStageK - 1) / kStageK * decode::kChunkBytes + (sf_bytes + 1023) / 1024 * 1024;
}
template <bool kMx, int BN>
constexpr int decode_stage_bytes() {
    return decode::kPerD * (mma_n(BN) * kRowBytes + Format<kMx>::tiles * kSfAtomBytes);
}
template <bool kMx, int BN>
int decode_stages(int K) {
    constexpr int by_tmem = static_cast<int>(kTmemCols - 2 * mma_n(BN)) / (8 * decode::kPerD * Format<kMx>::tiles);
    constexpr int most = by_tmem < decode::kMaxStagesD ? by_tmem : decode::kMaxStagesD;
    const int fit = (kSmemLimit - kFixedBytes - 1024 - decode_x_bytes<kMx>(K)) / decode_stage_bytes<kMx, BN>();
    return fit < most ? fit : most;
}

template <bool kMx, int BN>
cudaError_t launch_decode(const LinearInput& x, const LinearArgs& a, cudaStream_t st) {
    using namespace decode;
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
    const int num_st = (a.K + kPerD * kStageK - 1) / (kPerD * kStageK);
    const int x_bytes = decode_x_bytes<kMx>(a.K), stage_bytes = decode_stage_bytes<kMx, BN>();
    // an MMA reads 128 rows from x's last chunk: a stage lies behind it
    static_assert(kPerD * mma_n(BN) * kRowBytes >= kBM * kRowBytes, "rows an MMA reads past x");
    p.n_tiles = (a.N + BN - 1) / BN;
    const int sms = device_sm_count();
    const int grid = p.n_tiles < sms ? p.n_tiles : sms;
    p.stages = decode_stages<kMx, BN>(a.K);
    if (p.n_tiles <= sms && p.stages > num_st) p.stages = num_st;
    const size_t smem = static_cast<size_t>(x_bytes) + static_cast<size_t>(p.stages) * stage_bytes + 1024;
    CUtensorMap mb;
    if (!make_map(&mb, a.b_codes, a.N, a.K / 2, BN)) return cudaErrorInvalidValue;
    return launch_pdl(false, linear_decode_kernel<kMx, BN>, grid, kThreadsD, smem, st, mb, p);
}

// Rows of A in a tile.
int rows_of_a(int64_t T) { return T >= kBM ? kBM : static_cast<int>((T + 15) / 16 * 16); }

template <bool kMx, int BN>
cudaError_t launch(const LinearArgs& a, cudaStream_t st, bool pdl) {
    using F = Format<kMx>;
    static bool ready[kMaxDevices];
    cudaError_t e = prepare(linear_fp4_kernel<kMx, BN>, kSmemLimit - kFixedBytes, ready);
    if (e != cudaSuccess) return e;
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
    p.a_rows = rows_of_a(a.T);
    p.stage_bytes = kPer * ((p.a_rows + mma_n(BN)) * kRowBytes + 2 * F::tiles * kSfAtomBytes);
    // An MMA reads 128 rows of A whatever a_rows is (the rows past it give results nobody reads): 16 KB past
    // the start of the last stage's last chunk of A stay inside the allocation.
    const int past = (kBM - p.a_rows) * kRowBytes;
    p.stages = (kSmemLimit - kFixedBytes - 1024 - past) / p.stage_bytes;
    const int by_tmem = static_cast<int>(kTmemCols - 2 * mma_n(BN)) / (8 * kPer * F::tiles);
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    if (p.stages > by_tmem) p.stages = by_tmem;
    const int num_st = (a.K + kPer * kStageK - 1) / (kPer * kStageK);
    p.n_tiles = (a.N + BN - 1) / BN;
    p.tiles = (a.T + kBM - 1) / kBM * p.n_tiles;
    p.err = a.err;
    const int sms = device_sm_count();
    const unsigned grid = static_cast<unsigned>(p.tiles < sms ? p.tiles : sms);
    if (p.tiles <= sms && p.stages > num_st) p.stages = num_st;
    const size_t smem = static_cast<size_t>(p.stages) * p.stage_bytes + past + 1024;
    CUtensorMap ma, mb;
    if (!make_map(&ma, a.a_codes, a.T, a.K / 2, p.a_rows) || !make_map(&mb, a.b_codes, a.N, a.K / 2, BN))
        return cudaErrorInvalidValue;
    return launch_pdl(pdl, linear_fp4_kernel<kMx, BN>, grid, kThreads, smem, st, ma, mb, p);
}

}  // namespace

// Whether one kernel quantises x and multiplies: as many elements as its quantisers hold.  At that limit it takes as
// long on the device as two kernels (16 x 1536 x 2048: MXFP4 4.9 and 5.6 us, NVFP4 7.8 and 6.7) and saves the caller
// a launch and a workspace; twice as many elements take it longer (16 x 4096 x 4096 NVFP4 11.7 and 8.6 us).
bool linear_quantises_x(bool mx, int64_t T, int64_t K) {
    using namespace decode;
    return T <= kMaxT && K <= kMaxK &&
           (mx ? T * ((K + piece_cols<true>() - 1) / piece_cols<true>()) <= max_pieces<true>()
               : T * ((K + piece_cols<false>() - 1) / piece_cols<false>()) <= max_pieces<false>());
}

cudaError_t launch_linear_x(const LinearInput& x, const LinearArgs& a, cudaStream_t st) {
    // A tile takes the time of its MMAs' issue, about the same for 32 and 64 outputs and a fifth more for 128: the
    // narrowest tile that needs one round over the SMs, or the widest.  One token MXFP4, tiles 32, 64 and 128 wide:
    // 4096 x 4096 5.3, 5.5 and 6.5 us, 8192 x 4096 8.4, 5.9 and 6.6, 20000 x 2048 9.7, 7.1 and 6.7.
    // The widest only where two stages of its weights fit beside x: with one (MXFP4 above K = 6656, NVFP4 above 4608)
    // each load waits for the last one's MMAs.  One token, 64 and 128 wide, MXFP4 and NVFP4: 28672 x 8192 24.7 and 41.5 us,
    // 30.6 and 46.0; 12000 x 8192 16.7 and 20.8, 21.0 and 24.3; with two stages 28672 x 4096 14.3 and 15.8, 16.8 and 18.6.
    const int sms = device_sm_count();
    if (a.N <= 32 * sms) return a.mx ? launch_decode<true, 32>(x, a, st) : launch_decode<false, 32>(x, a, st);
    if (a.N <= 64 * sms || (a.mx ? decode_stages<true, 128>(a.K) : decode_stages<false, 128>(a.K)) < 2)
        return a.mx ? launch_decode<true, 64>(x, a, st) : launch_decode<false, 64>(x, a, st);
    return a.mx ? launch_decode<true, 128>(x, a, st) : launch_decode<false, 128>(x, a, st);
}

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t st, bool pdl) {
    // The kernel and tile with the least time, in cycles: over the SMs (or pairs of them) a round of tiles takes the
    // longer of its main loop and its outputs, and one of each is left at the ends.  A 256-element chunk of K takes the
    // larger of its MMAs (240 for N = 64, 310 for 128) and its operands' way into the SM (about 2.4 a row of 128
    // bytes), in a pair 560; a tile's outputs 700 and 22 a column, 93 row by row, a pair's 4500 or 9600.  Both sides,
    // us of MXFP4 with the quantisation of x (* the rule's):
    //                         32      64      128     pair
    //   300 x 1536 x 2048     6.1 *   6.1     6.8     8.6
    //   256 x 4096 x 4096    10.7     7.7 *   8.8    10.7
    //   512 x 4096 x 4096    17.3    10.9     9.2 *  10.9
    //   700 x 4096 x 4096    23.6    14.3    13.0    11.2 *
    //   4096 x 4096 x 4096   94.1    51.8    36.4    29.9 *
    //   5000 x 2048 x 512    14.7    11.9    11.2     9.4 *
    //   300 x 1533 x 2048     7.0 *   8.3    11.1    10.8     rows on no 16-byte boundary
    //   8192 x 1999 x 2048   58.2    54.9    51.9    28.1 *   the same
    const int64_t sms = device_sm_count(), m = (a.T + kBM - 1) / kBM, num_ks = (a.K + kStageK - 1) / kStageK;
    const int rows = rows_of_a(a.T);
    const bool wide = out_align(a) > 0;
    auto cost = [](int64_t tiles, int64_t at_once, int64_t main, int64_t out) {
        return (tiles + at_once - 1) / at_once * (main > out ? main : out) + (main > out ? out : main);
    };
    auto one = [&](int bn, int mma) {
        const int load = 12 * (rows + bn) / 5;
        return cost(m * ((a.N + bn - 1) / bn), sms, num_ks * (load > mma ? load : mma), 700 + bn * (wide ? 22 : 93));
    };
    const int64_t c32 = one(32, 240), c64 = one(64, 240), c128 = one(128, 310);
    const int64_t pair_tiles = (a.T + 255) / 256 * ((a.N + 255) / 256);
    const int64_t cpair = cost(pair_tiles, linear_pair_count(), num_ks * 560 + 800, wide ? 4500 : 9600);
    if (cpair <= c32 && cpair <= c64 && cpair <= c128) return launch_linear_pair(a, st, pdl);
    if (c128 <= c64 && c128 <= c32) return a.mx ? launch<true, 128>(a, st, pdl) : launch<false, 128>(a, st, pdl);
    if (c64 <= c32) return a.mx ? launch<true, 64>(a, st, pdl) : launch<false, 64>(a, st, pdl);
    return a.mx ? launch<true, 32>(a, st, pdl) : launch<false, 32>(a, st, pdl);
}

}  // namespace nvfp4
