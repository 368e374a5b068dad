// Low-rank adapters of many requests beside a shared projection: what its kernels share.
//
//   forward    h_t = A_a x_t,           y_t += s_a B_a h_t        a = adapter of token t, A [R][K], B [N][R]
//   backward   dh_t = s_a B_a^T dy_t,   dx_t += A_a^T dh_t,   dA_a = sum_t dh_t x_t^T,  dB_a = sum_t s_a dy_t h_t^T
//
// Forward and dx have one shape: a row of C columns shrinks to R and expands to D columns.  Tokens of an adapter are put
// together in tiles of 16 or 128 rows; a cluster of CTAs takes a tile, each CTA its share of C, then its share of D.
//
// The order of the sum over C goes by C alone, so a token's row does not depend on the batch: C is cut into 8 groups of 8
// sub-slices of 16 ceil(C / 1024) columns, from 32768 columns on of twice, three times, ... as many of no more than 512; a
// sub-slice is one chain of m16n8k16 products from zero, the sub-slices of a group
// are added in order, the groups as a binary tree (which clusters of 2, 4 and 8 CTAs can share).  The tensor cores cut an
// accumulator's low bits off at each step: h of values of one sign is 8e-7 low after chains of 32 steps (32768 columns), and was
// 8e-5 low with chains of 1024 (2^20 columns).  mma.sync serves this
// better than tcgen05: a tile has as few as one real row and 8 to 128 columns of accumulator, the two products together
// have 2 R operations to a byte that is moved, and accumulators in registers need no pass through TMEM between the two
// products (its rate, 600 TFLOP/s measured, is enough for R <= 64 at the memory's rate).
//
// Between the products h is FP32; the second product takes it as a sum of 16-bit terms (two for 16-bit outputs, which leaves
// 2^-17 of h beside the output's own 2^-9; three for FP32 outputs), so h is not rounded to 16 bits.
#pragma once

#include "cluster.cuh"
#include "common.cuh"
#include "ops.cuh"
#include "scores.cuh"

namespace nvfp4 {
namespace lora {

constexpr int kThreads = 256, kWarps = 8;
constexpr int kGroups = 8;                // of C; CTAs of a cluster at most
constexpr int kFewRows = 16, kManyRows = 128, kStageRows = 32;
constexpr int kMaxCtas = 320;             // of the adapters' gradients
constexpr unsigned kAll = 0xFFFFFFFFu;

// The tiles that the sort kernel lists, in the workspace.
struct Tiles {
    const int32_t* perm;        // [T] rows, adapter by adapter, those without one last
    const int32_t* adapter;     // [count] -1: rows without an adapter
    const int32_t* start;       // [count] first row of the tile in perm
    const int32_t* offsets;     // [L + 2] first row of each adapter in perm
    const int32_t* count;
    const int32_t* prefix;      // [L + 1] stages of 32 rows of the adapters in front (one of an adapter without rows)
    int32_t* pieces;            // [kMaxCtas] zeros: counters for the adapters' gradients
};

struct Params {
    const void* x;              // [T][ldx], C columns; rows on 16-byte boundaries
    int64_t ldx;
    const void* down;           // what x is multiplied with: [L][R][C], or [L][C][R] (transposed)
    const void* up;             // and h: [L][D][R], or [L][R][D] (transposed)
    const float* scale;         // [L] or nullptr
    const int32_t* ids;         // [T]
    const void* y;              // [T][ldy] of y_type, or nullptr (zeros)
    void* out;                  // [T][ldo]
    float* h;                   // [T][R] or nullptr
    int64_t ldy, ldo;
    int y_type, y_wide, out_wide;   // y's, and out's rows start on 16-byte boundaries
    int h_scaled;               // h holds s_a h
    int skip_none;              // rows without an adapter need no work
    int T, L, R, C, D;
    Tiles tiles;
    int* err;
};

// ------------------------------------------------------------------ pieces of the kernels
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {   // the rest of the 16 are zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }

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
// The 8 warps that multiply; each arrives as one.
__device__ __forceinline__ void consumer_barrier() {
    __syncwarp();
    asm volatile("bar.sync 1, 256;" ::: "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma(__nv_bfloat16, float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(__half, float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Tiles of 64 16-bit columns: rows of 128 bytes, their 16-byte chunks exchanged by the row, so that the eight rows of a
// matrix lie in different banks.
__device__ __forceinline__ uint32_t swizzled(int row, int chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }
// The same for rows of 32 or 64 bytes, as TMA's 32B and 64B swizzles lay them out.
template <int kBytes>
__device__ __forceinline__ uint32_t swizzled_rows(int row, int chunk) {
    return row * kBytes + ((chunk ^ (row * kBytes >> 7 & (kBytes / 16 - 1))) << 4);
}
// Bytes of a row of ranks in shared memory: 16, 32 or 64 of them (two blocks of 64 above that).
__host__ __device__ constexpr int rank_bytes(int R) { return R <= 16 ? 32 : R <= 32 ? 64 : 128; }
// Tiles of R columns: rows padded by 16 bytes (the eight rows of a matrix in different banks where R is a multiple of 16).
__host__ __device__ constexpr int padded_pitch(int R) { return 2 * R + 16; }
__host__ __device__ constexpr int rank_up(int R) { return (R + 15) / 16 * 16; }   // the second product's steps are 16 wide

// Sub-slices of the first product: 64 to a round, of as many steps of 16 columns, at most kChainSteps.
constexpr int kChainSteps = 32;
__host__ __device__ inline int sub_rounds(int C) { return (C + 1024 * kChainSteps - 1) / (1024 * kChainSteps); }
__host__ __device__ inline int sub_steps(int C) { return (C + 1024 * sub_rounds(C) - 1) / (1024 * sub_rounds(C)); }

// 16 bytes of a row from 16-bit unit c on (zeros from `units` on) into shared memory.  Rows that do not start on a 16-byte
// boundary are read in the aligned 16-byte words that hold a unit of theirs, two of them shifted together, in place of eight
// loads of single elements.
struct Straddle {
    uint4 lo, hi;
    int left, off;                        // units that are there, bytes in front of them
    __device__ __forceinline__ void load(const uint16_t* row, int c, int units) { load(row + c, units - c); }
    __device__ __forceinline__ void load(const uint16_t* from, int units) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(from);
        left = min(max(units, 0), 8);
        off = static_cast<int>(at & 15);
        const uint4* p = reinterpret_cast<const uint4*>(at & ~uintptr_t(15));
        lo = hi = make_uint4(0, 0, 0, 0);
        if (left > 0) lo = __ldg(p);
        if (2 * left > 16 - off) hi = __ldg(p + 1);
    }
    __device__ __forceinline__ uint4 value() const {
        uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        if (off & 4) {
#pragma unroll
            for (int i = 0; i < 7; ++i) w[i] = w[i + 1];
        }
        if (off & 8) {
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 2];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = __funnelshift_r(w[i], w[i + 1], (off & 2) * 8);
            if (2 * i + 1 >= left) w[i] = 2 * i < left ? w[i] & 0xFFFFu : 0;
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void store(uint32_t dst) const {
        const uint4 v = value();
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
    }
};
// The same of rows that do start on one.
__device__ __forceinline__ void copy_chunk(uint32_t dst, const uint16_t* row, int c, int units) {
    const int left = min(max(units - c, 0), 8);
    cp_async16(dst, left ? row + c : row, 2 * left);
}
// Operand of the first product: `cols` (a multiple of 16, at most 64) columns from c on of the adapter's matrix.
template <bool kTrans>
__device__ __forceinline__ void load_down(uint32_t dst, const uint16_t* down, int R, int C, int c, int cols, int thread, int threads) {
    if (!kTrans) {                        // [R][C]: R rows of 64 columns, swizzled
        const int q = thread & 7;
        if (8 * q < cols) {
            for (int r = thread >> 3; r < R; r += threads >> 3)
                copy_chunk(dst + swizzled(r, q), down + static_cast<int64_t>(r) * C, c + 8 * q, C);
        }
    } else {                              // [C][R]: rows of R columns, padded
        const int per = R / 8, at_once = threads / per, n0 = thread / per, q = thread - n0 * per;
        if (n0 < at_once) {
            const uint16_t* src = down + static_cast<int64_t>(c + n0) * R + 8 * q;
            dst += n0 * padded_pitch(R) + 16 * q;
            for (int n = n0; n < cols; n += at_once, src += at_once * R, dst += at_once * padded_pitch(R)) {
                if (c + n < C) cp_async16(dst, src);
                else cp_async16(dst, down, 0);
            }
        }
    }
}
template <bool kTrans>
__host__ __device__ constexpr int down_bytes(int R, int cols) { return kTrans ? cols * padded_pitch(R) : rank_up(R) * 128; }

// A lane's address in a swizzled tile for ldmatrix, of step 0; step kk is at ^ (kk << 5) of it, 8 more rows 1024 further.
__device__ __forceinline__ uint32_t lane_rows(int lane) {   // matrices: 8 rows, the next 8, then the next 8 columns of both
    return swizzled((lane & 7) + ((lane >> 3) & 1) * 8, lane >> 4);
}
template <bool kTrans>
__device__ __forceinline__ uint32_t lane_down(int lane, int R) {
    return kTrans ? (((lane >> 3) & 1) * 8 + (lane & 7)) * padded_pitch(R) + 16 * (lane >> 4)
                  : swizzled(8 * (lane >> 4) + (lane & 7), (lane >> 3) & 1);
}
// Products of 16 rows x 16 columns of x (a) with step kk of the operand above (`down`: its address + lane_down): acc[j]
// gets ranks 8 j to 8 j + 7.
template <typename T, bool kTrans, int kTiles>
__device__ __forceinline__ void multiply_down(float (&acc)[kTiles][4], const uint32_t (&a)[4], uint32_t down, int kk, int R) {
    const uint32_t at = kTrans ? down + 16 * kk * padded_pitch(R) : down ^ (kk << 5);
#pragma unroll
    for (int j = 0; j < kTiles; j += 2) {
        if (8 * j >= R) break;
        uint32_t b[4];
        if (!kTrans) ldsm4(at + 1024 * j, b);
        else ldsm4_trans(at + 16 * j, b);
        mma(T(), acc[j], a, b[0], b[1]);
        if (8 * (j + 1) < R) mma(T(), acc[j + 1], a, b[2], b[3]);
    }
}

// Operand of the second product: `cols` (32 or 64) outputs from n on of the adapter's matrix; ranks from R to rank_up(R) are zeros.
// Not transposed, output 8 q + 2 i + l of a group of 32 lies in row 8 i + 2 q + l: the accumulators of a lane are then 8
// consecutive outputs of a row.
template <bool kTrans>
__device__ __forceinline__ void load_up(uint32_t dst, const uint16_t* up, int R, int D, int n, int cols, int thread, int threads) {
    const int Rp = rank_up(R);
    if (!kTrans) {                        // [D][R]
        const int per = Rp / 8, at_once = threads / per, j0 = thread / per, q = thread - j0 * per;
        if (j0 < at_once) {
            const uint16_t* src = up + static_cast<int64_t>(n + j0) * R + 8 * q;
            dst += 16 * q;
            for (int j = j0; j < cols; j += at_once, src += at_once * R) {
                const int at = (j & ~31) + 8 * ((j & 7) >> 1) + 2 * ((j & 31) >> 3) + (j & 1);
                if (n + j < D && 8 * q < R) cp_async16(dst + at * padded_pitch(Rp), src);
                else cp_async16(dst + at * padded_pitch(Rp), up, 0);
            }
        }
    } else {                              // [R][D]: rows of 64 columns, swizzled
        const int q = thread & 7;
        if (8 * q < cols) {
            for (int r = thread >> 3; r < Rp; r += threads >> 3) {
                if (r < R) copy_chunk(dst + swizzled(r, q), up + static_cast<int64_t>(r) * D, n + 8 * q, D);
                else cp_async16(dst + swizzled(r, q), up, 0);
            }
        }
    }
}
template <bool kTrans>
__host__ __device__ constexpr int up_bytes(int R, int cols) { return kTrans ? rank_up(R) * 128 : cols * padded_pitch(rank_up(R)); }

// h (16 rows from `h`, `terms` arrays of 16-bit terms that add up to it) times the operand above, group g32 of 32 outputs:
// o[i] gets the 8 consecutive outputs 8 (lane % 4) of row lane / 4 + 8 i.
template <typename T, bool kTrans>
__device__ __forceinline__ void multiply_up(float (&o)[2][8], uint32_t h, int term_bytes, int terms, uint32_t up, int g32, int R, int lane) {
    const int Rp = rank_up(R);
    float acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
    }
    const uint32_t ha = h + ((lane & 7) + ((lane >> 3) & 1) * 8) * padded_pitch(Rp) + 16 * (lane >> 4);
    for (int kk = 0; kk < Rp / 16; ++kk) {
        uint32_t b[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {     // two tiles of 8 outputs at once
            if (!kTrans) ldsm4(up + (32 * g32 + 8 * (2 * i + (lane >> 4)) + (lane & 7)) * padded_pitch(Rp) + 16 * (2 * kk + ((lane >> 3) & 1)), b[i]);
            else ldsm4_trans(up + swizzled(16 * kk + ((lane >> 3) & 1) * 8 + (lane & 7), 4 * g32 + 2 * i + (lane >> 4)), b[i]);
        }
        for (int t = 0; t < terms; ++t) {
            uint32_t a[4];
            ldsm4(ha + t * term_bytes + 32 * kk, a);
#pragma unroll
            for (int i = 0; i < 4; ++i) mma(T(), acc[i], a, b[i >> 1][2 * (i & 1)], b[i >> 1][2 * (i & 1) + 1]);
        }
    }
    if (!kTrans) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[0][2 * i] = acc[i][0], o[0][2 * i + 1] = acc[i][1];
            o[1][2 * i] = acc[i][2], o[1][2 * i + 1] = acc[i][3];
        }
    } else {
        // lane q of a quad has outputs 2 q, 2 q + 1 of four tiles and gets all 8 of tile q: a transposition in two steps,
        // with the lane two away, then with the one beside
        const int q = lane & 3;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float v[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i][0] = acc[i][2 * r], v[i][1] = acc[i][2 * r + 1];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int l = 0; l < 2; ++l) {
                    const float got = __shfl_xor_sync(kAll, q & 2 ? v[i][l] : v[i + 2][l], 2);
                    if (q & 2) v[i][l] = got;
                    else v[i + 2][l] = got;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
#pragma unroll
                for (int l = 0; l < 2; ++l) {
                    const float got = __shfl_xor_sync(kAll, q & 1 ? v[i][l] : v[i + 1][l], 1);
                    if (q & 1) v[i][l] = got;
                    else v[i + 1][l] = got;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) o[r][2 * i] = v[i][0], o[r][2 * i + 1] = v[i][1];
        }
    }
}

// 8 consecutive elements of a row of y or out, raw (kept so while they are on their way).
struct Eight {
    uint4 a, b;                           // b: FP32 only
};
__device__ __forceinline__ uint32_t element(const void* row, int64_t i, int type) {
    return type == NVFP4_TYPE_F32 ? static_cast<const uint32_t*>(row)[i] : static_cast<const uint16_t*>(row)[i];
}
__device__ __forceinline__ Eight load_eight(const void* base, int type, int64_t row, int64_t ld, int n, int D, bool wide) {
    Eight e = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (n >= D) return e;
    const int size = type == NVFP4_TYPE_F32 ? 4 : 2;
    const uint8_t* p = static_cast<const uint8_t*>(base) + (row * ld + n) * size;
    if (wide && n + 8 <= D) {
        e.a = *reinterpret_cast<const uint4*>(p);
        if (size == 4) e.b = *reinterpret_cast<const uint4*>(p + 16);
        return e;
    }
    uint32_t w[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (n + i >= D) continue;
        if (size == 4) w[i] = element(p, i, type);
        else w[i / 2] |= element(p, i, type) << (16 * (i & 1));
    }
    e.a = make_uint4(w[0], w[1], w[2], w[3]);
    e.b = make_uint4(w[4], w[5], w[6], w[7]);
    return e;
}
__device__ __forceinline__ float2 unpack2(uint32_t w, int type) {
    if (type == NVFP4_TYPE_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, int type) {
    if (type == NVFP4_TYPE_BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t add2(uint32_t y, float lo, float hi, int type) {
    const float2 f = unpack2(y, type);
    return pack2(f.x + lo, f.y + hi, type);
}
// y += o, in FP32 with one rounding.
__device__ __forceinline__ void add_eight(Eight& y, const float (&o)[8], int type) {
    if (type == NVFP4_TYPE_BF16) {        // one branch for all
        y.a = make_uint4(add2(y.a.x, o[0], o[1], NVFP4_TYPE_BF16), add2(y.a.y, o[2], o[3], NVFP4_TYPE_BF16),
                         add2(y.a.z, o[4], o[5], NVFP4_TYPE_BF16), add2(y.a.w, o[6], o[7], NVFP4_TYPE_BF16));
    } else if (type == NVFP4_TYPE_F16) {
        y.a = make_uint4(add2(y.a.x, o[0], o[1], NVFP4_TYPE_F16), add2(y.a.y, o[2], o[3], NVFP4_TYPE_F16),
                         add2(y.a.z, o[4], o[5], NVFP4_TYPE_F16), add2(y.a.w, o[6], o[7], NVFP4_TYPE_F16));
    } else {
        const auto add = [](uint32_t w, float v) { return __float_as_uint(__uint_as_float(w) + v); };
        y.a = make_uint4(add(y.a.x, o[0]), add(y.a.y, o[1]), add(y.a.z, o[2]), add(y.a.w, o[3]));
        y.b = make_uint4(add(y.b.x, o[4]), add(y.b.y, o[5]), add(y.b.z, o[6]), add(y.b.w, o[7]));
    }
}
// Columns [n, D) of 8 consecutive elements at p.
__device__ __forceinline__ void store_eight(uint8_t* p, int type, int n, int D, bool wide, const Eight& v) {
    if (n >= D) return;
    if (wide && n + 8 <= D) {
        *reinterpret_cast<uint4*>(p) = v.a;
        if (type == NVFP4_TYPE_F32) *reinterpret_cast<uint4*>(p + 16) = v.b;
        return;
    }
    const uint32_t w[8] = {v.a.x, v.a.y, v.a.z, v.a.w, v.b.x, v.b.y, v.b.z, v.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (n + i >= D) continue;
        if (type == NVFP4_TYPE_F32) reinterpret_cast<uint32_t*>(p)[i] = w[i];
        else reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
    }
}

// The 16-bit terms of v: v = t0 + t1 (+ t2) but for the last one's rounding.  Where a term is infinite the rest is 0.
template <typename T>
__device__ __forceinline__ uint16_t next_term(float& v) {
    const T t = from_f32<T>(v);
    const float f = to_f32(t), left = v - f;
    v = fabsf(f) == INFINITY ? 0.0f : left;
    return *reinterpret_cast<const uint16_t*>(&t);
}
// FP16 has no room for h of any size: its rows are scaled by a power of two that puts their largest value near 2^14
// (exact, and undone in FP32 behind the product).  The exponent that is taken out of a row whose largest |h| is m.
__device__ __forceinline__ int row_exponent(float m) {
    if (!(m > 0.0f) || m == INFINITY) return 0;
    return max(static_cast<int>(__float_as_uint(m) >> 23) - 127, -100) - 14;
}

// A row of h: lane l of kLanes sums the 2, 4 or 8 CTAs' parts of columns 2 l, 2 l + 1, 2 l + 2 kLanes, ... as a tree, and hands
// over the row's terms, two columns (32 bits) at a time.
template <typename T, int kRank, int kLanes, typename Store>
__device__ __forceinline__ void finish_row(const float* part, int parts, int row, int pitch, int R, float scale, int terms, int term_bytes,
                                           float* h_out, bool h_scaled, int l, Store&& store, float& undo) {
    constexpr int kStep = 2 * kLanes, kMine = (kRank + kStep - 1) / kStep;
    float v[kMine][2], m = 0.0f;
    uint32_t from[kGroups];
#pragma unroll
    for (int c = 0; c < kGroups; ++c) from[c] = cluster_addr(part, c < parts ? c : 0) + 4 * row * pitch;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int r = 2 * l + kStep * i;
        v[i][0] = v[i][1] = 0.0f;
        if (r < R) {
            float got[kGroups][2];
#pragma unroll
            for (int c = 0; c < kGroups; ++c) {
                if (c < parts)
                    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(got[c][0]), "=f"(got[c][1]) : "r"(from[c] + 4 * r));
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int n = kGroups / 2; n >= 1; n /= 2) {
                    if (2 * n > parts) continue;
#pragma unroll
                    for (int c = 0; c < n; ++c) got[c][k] = got[2 * c][k] + got[2 * c + 1][k];
                }
                v[i][k] = got[0][k];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int r = 2 * l + kStep * i;
        const float sum[2] = {v[i][0], v[i][1]};
        v[i][0] *= scale;
        v[i][1] *= scale;
        if (h_out != nullptr && r < R) *reinterpret_cast<float2*>(h_out + r) = h_scaled ? make_float2(v[i][0], v[i][1]) : make_float2(sum[0], sum[1]);
        m = fmaxf(m, fmaxf(fabsf(v[i][0]), fabsf(v[i][1])));
    }
    undo = 1.0f;
    if (std::is_same<T, __half>::value) {
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        const int e = row_exponent(m);
        undo = ldexpf(1.0f, e);
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            v[i][0] = ldexpf(v[i][0], -e);
            v[i][1] = ldexpf(v[i][1], -e);
        }
    }
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int r = 2 * l + kStep * i;
        if (r >= rank_up(R)) continue;
        for (int t = 0; t < terms; ++t) {
            const uint32_t lo = next_term<T>(v[i][0]), hi = next_term<T>(v[i][1]);
            store(t * term_bytes + 2 * r, lo | hi << 16);
        }
    }
}

}  // namespace lora
}  // namespace nvfp4
