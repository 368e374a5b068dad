// What the dense product's kernels (linear.cu, linear_pair.cu) share: the formats, instruction
// descriptors, uniform values, output stores and host-side tensor maps.
#pragma once

#include <mutex>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ops.cuh"
#include "ptx.cuh"

namespace nvfp4 {
namespace {

constexpr int kBM = 128;
constexpr int kRowBytes = 128;                       // bytes of K per row and stage: 256 elements
constexpr int kStageK = 256;
constexpr uint32_t kTmemCols = 512;
constexpr int kSmemLimit = 227 * 1024;
constexpr int kFixedBytes = 10240;                   // room left for static shared memory

// A value all lanes hold, taken from lane 0: the compiler then knows that it is the same in all of them.
// Roles chosen by such a warp index, and descriptors made of such values, stay on the uniform
// datapath that the tcgen05 and TMA instructions take their operands from; from threadIdx.x >> 5 every
// operand is moved over first.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }
__device__ __forceinline__ int warp_index() { return static_cast<int>(uniform(threadIdx.x >> 5)); }

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

// One stage of the main loop, in one block of PTX with one elect.sync: the scale tiles go to TMEM (from column sf on,
// A's first, then B's, one set of 128 rows or, by a pair of CTAs, two), then nk <= 4 K=64 MMAs accumulate into d.
// sa, sb, sb2: descriptors of the scale tiles of A and of B's first and second 128 rows (the next tile 512 bytes, 32
// units, further); a K step is 32 bytes (2 units) of the operands' rows.  (As twelve separately elected instructions
// a stage took 730-800 cycles to issue, so 260.)
#define LINEAR_CP(G, P, dst, src) "@" P " tcgen05.cp.cta_group::" G ".32x128b.warpx4 [" dst "], " src ";\n\t"
#define LINEAR_MMA_NV(G, P, acc, sfb)                                                                        \
    "@" P " tcgen05.mma.cta_group::" G ".kind::mxf4nvf4.block_scale.scale_vec::4X [%0], a, b, %3, [ca], [" sfb "], " acc ";\n\t"
#define LINEAR_MMA_MX(G, P, acc, idesc, sfb)                                                                 \
    "@" P " tcgen05.mma.cta_group::" G ".kind::mxf4.block_scale.scale_vec::2X [%0], a, b, " idesc ", [ca], [" sfb "], " acc ";\n\t"
#define LINEAR_STEP "add.s64 a, a, 2;\n\tadd.s64 b, b, 2;\n\t"
#define LINEAR_BEGIN                                                                                         \
    "{\n\t.reg .pred ep, e1, e2, e3, p0, p1;\n\t.reg .b32 er, ca, cb, cc, i2;\n\t.reg .b64 a, b, s0, s1, s2;\n\t"     \
    "elect.sync er|ep, 0xffffffff;\n\tsetp.ne.b32 p0, %9, 0;\n\tsetp.eq.b32 p1, %9, %9;\n\t"                    \
    "setp.gt.and.s32 e1, %10, 1, ep;\n\tsetp.gt.and.s32 e2, %10, 2, ep;\n\tsetp.gt.and.s32 e3, %10, 3, ep;\n\t"      \
    "mov.b64 a, %1;\n\tmov.b64 b, %2;\n\tmov.b64 s0, %4;\n\tmov.b64 s1, %5;\n\tmov.b64 s2, %6;\n\tmov.b32 ca, %7;\n\t" \
    "add.u32 cb, %7, %11;\n\t"
#define LINEAR_NEXT(cols) \
    "add.s64 s0, s0, 32;\n\tadd.s64 s1, s1, 32;\n\tadd.s64 s2, s2, 32;\n\tadd.u32 ca, ca, 4;\n\tadd.u32 cb, cb, " cols ";\n\t"
#define LINEAR_OPERANDS \
    ::"r"(d), "l"(a), "l"(b), "r"(idesc), "l"(sa), "l"(sb), "l"(sb2), "r"(sf), "r"(sfb_col),       \
        "r"(accumulate ? 1u : 0u), "r"(nk), "n"(4 * Format<kMx>::tiles) : "memory"
// one 128-row set of B: its MMA's scales may start at the tile's third column
#define LINEAR_NV1(P, acc) LINEAR_CP("1", P, "ca", "s0") LINEAR_CP("1", P, "cb", "s1") "add.u32 cc, cb, %8;\n\t" LINEAR_MMA_NV("1", P, acc, "cc")
// a pair of CTAs, two sets
#define LINEAR_NV2(P, acc)                                                                                   \
    LINEAR_CP("2", P, "ca", "s0") LINEAR_CP("2", P, "cb", "s1") "add.u32 cc, cb, 4;\n\t" LINEAR_CP("2", P, "cc", "s2") \
        LINEAR_MMA_NV("2", P, acc, "cb")
#define LINEAR_MX1(P, Q, acc)                                                                                \
    LINEAR_CP("1", P, "ca", "s0") LINEAR_CP("1", P, "cb", "s1") "add.u32 cc, cb, %8;\n\t"                       \
        LINEAR_MMA_MX("1", P, acc, "%3", "cc") LINEAR_STEP LINEAR_MMA_MX("1", Q, "p1", "i2", "cc")
#define LINEAR_MX2(P, Q, acc)                                                                                \
    LINEAR_CP("2", P, "ca", "s0") LINEAR_CP("2", P, "cb", "s1") "add.u32 cc, cb, 4;\n\t" LINEAR_CP("2", P, "cc", "s2") \
        LINEAR_MMA_MX("2", P, acc, "%3", "cb") LINEAR_STEP LINEAR_MMA_MX("2", Q, "p1", "i2", "cb")
#define LINEAR_ID2 "or.b32 i2, %3, 0x40000020;\n\t"

template <bool kMx, bool kPair>
__device__ __forceinline__ void issue_stage(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint64_t sa, uint64_t sb,
                                            uint64_t sb2, uint32_t sf, uint32_t sfb_col, int nk, bool accumulate) {
    static_assert(idesc_sf_id(2) == 0x40000020u, "scale-factor id of the second half of a word");
    if constexpr (!kMx && !kPair)
        asm volatile(LINEAR_BEGIN LINEAR_NV1("ep", "p0") LINEAR_STEP LINEAR_NEXT("4") LINEAR_NV1("e1", "p1") LINEAR_STEP
                         LINEAR_NEXT("4") LINEAR_NV1("e2", "p1") LINEAR_STEP LINEAR_NEXT("4") LINEAR_NV1("e3", "p1") "}"
                     LINEAR_OPERANDS);
    else if constexpr (!kPair)
        asm volatile(LINEAR_BEGIN LINEAR_ID2 LINEAR_MX1("ep", "e1", "p0") LINEAR_STEP LINEAR_NEXT("4")
                         LINEAR_MX1("e2", "e3", "p1") "}" LINEAR_OPERANDS);
    else if constexpr (!kMx)
        asm volatile(LINEAR_BEGIN LINEAR_NV2("ep", "p0") LINEAR_STEP LINEAR_NEXT("8") LINEAR_NV2("e1", "p1") LINEAR_STEP
                         LINEAR_NEXT("8") LINEAR_NV2("e2", "p1") LINEAR_STEP LINEAR_NEXT("8") LINEAR_NV2("e3", "p1") "}"
                     LINEAR_OPERANDS);
    else
        asm volatile(LINEAR_BEGIN LINEAR_ID2 LINEAR_MX2("ep", "e1", "p0") LINEAR_STEP LINEAR_NEXT("8")
                         LINEAR_MX2("e2", "e3", "p1") "}" LINEAR_OPERANDS);
}
#undef LINEAR_CP
#undef LINEAR_MMA_NV
#undef LINEAR_MMA_MX
#undef LINEAR_STEP
#undef LINEAR_BEGIN
#undef LINEAR_NEXT
#undef LINEAR_OPERANDS
#undef LINEAR_NV1
#undef LINEAR_NV2
#undef LINEAR_MX1
#undef LINEAR_MX2
#undef LINEAR_ID2

// ---- outputs

// Pairs of FP32 values in one 64-bit register (the first low); products and sums round each.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ uint64_t pair_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t pair_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

// The 32-bit words of 16 outputs of type T.
template <typename T>
__device__ __forceinline__ void pack16(const uint64_t (&v)[8], uint32_t (&w)[4 * sizeof(T)]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float lo, hi;
        unpair(v[i], lo, hi);
        if constexpr (sizeof(T) == 4) {
            w[2 * i] = __float_as_uint(lo);
            w[2 * i + 1] = __float_as_uint(hi);
        } else if constexpr (std::is_same<T, __half>::value) {
            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(hi), "f"(lo));
        } else {
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(hi), "f"(lo));
        }
    }
}

// 16 consecutive outputs of a row, of which the first `n` exist.  align: 2 where rows lie on 32-byte
// boundaries (whole sectors in one store), 1 on 16-byte ones, less otherwise.
template <typename T>
__device__ __forceinline__ void store16(T* p, const uint64_t (&v)[8], int n, int align) {
    constexpr int kWords = 4 * sizeof(T);
    uint32_t w[kWords];
    pack16<T>(v, w);
    if (n >= 16 && align > 1) {
#pragma unroll
        for (int i = 0; i < kWords; i += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(reinterpret_cast<uint32_t*>(p) + i),
                         "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]),
                         "r"(w[i + 7])
                         : "memory");
    } else if (n >= 16 && align > 0) {
#pragma unroll
        for (int i = 0; i < kWords; i += 4)
            *reinterpret_cast<uint4*>(reinterpret_cast<uint32_t*>(p) + i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (i >= n) break;
            if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t*>(p)[i] = w[i];
            else reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
        }
    }
}

// Byte of 16-byte chunk c of row r among rows of kRow bytes in shared memory: eight rows' same chunk lie in eight
// different banks' groups.
template <int kRow>
__device__ __forceinline__ int row_chunk(int r, int c) { return (c ^ (r / (128 / kRow) & (kRow / 16 - 1))) << 4; }

// 16 outputs from a lane's accumulator values: NVFP4 outer scales (g2: the row's twice, gcol: the
// columns'), the bias (bcol) if there is one.  gcol, bcol: 8-byte aligned shared memory.
template <bool kMx, bool kBias>
__device__ __forceinline__ void scale16(const uint32_t* v, uint64_t g2, const float* gcol, const float* bcol, uint64_t (&o)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        o[i] = pair(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
        if (!kMx) o[i] = pair_mul(pair_mul(o[i], g2), *reinterpret_cast<const uint64_t*>(gcol + 2 * i));
        if (kBias) o[i] = pair_add(o[i], *reinterpret_cast<const uint64_t*>(bcol + 2 * i));
    }
}

// kCols outputs of a row, of which the first `left` exist, straight to memory.
template <bool kMx, bool kBias, typename T, int kCols>
__device__ __forceinline__ void outputs(const uint32_t* v, float ga, const float* gcol, const float* bcol, T* row, int left,
                                        int align) {
    const uint64_t g2 = pair(ga, ga);
#pragma unroll
    for (int h = 0; h < kCols; h += 16) {
        if (left <= h) break;
        uint64_t o[8];
        scale16<kMx, kBias>(v + h, g2, gcol + h, bcol + h, o);
        store16<T>(row + h, o, left - h, align);
    }
}
// The same for a warp's `rows` rows (this lane's: v) where rows lie on no 16-byte boundary: kPass columns at a time
// through the warp's shared memory (buf, 32 rows of kPass outputs in swizzled 16-byte chunks) and from there row by
// row, in 4-byte words where rows lie on such boundaries.  (With each lane storing its own row, 32 sectors to an
// instruction, the MXFP4 product of 8192 x 1999 x 2048 took 173 us instead of 28.)  left: columns that exist.
template <typename U, typename T, int kPass>
__device__ __forceinline__ void copy_rows(const uint8_t* buf, T* out, int64_t ldo, int rows, int left) {
    constexpr int kRow = kPass * sizeof(T), kUnits = kRow / sizeof(U), kEach = sizeof(U) / sizeof(T);
    const int lane = threadIdx.x & 31;
#pragma unroll 4
    for (int i = lane; i < rows * kUnits; i += 32) {
        const int r = i / kUnits, u = i % kUnits, at = u * sizeof(U), col = u * kEach;
        const U v = *reinterpret_cast<const U*>(buf + r * kRow + row_chunk<kRow>(r, at / 16) + at % 16);
        T* dst = out + r * ldo + col;
        if (col + kEach <= left) *reinterpret_cast<U*>(dst) = v;
        else if (kEach > 1 && col < left) *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(v);
    }
}
template <bool kMx, bool kBias, typename T, int kCols, int kPass>
__device__ __forceinline__ void outputs_by_row(const uint32_t* v, float ga, const float* gcol, const float* bcol, uint8_t* buf,
                                               T* out, int64_t ldo, int rows, int left, bool words) {
    constexpr int kRow = kPass * sizeof(T), kChunks = sizeof(T);   // 16-byte chunks of 16 columns
    const int lane = threadIdx.x & 31;
    const uint64_t g2 = pair(ga, ga);
#pragma unroll
    for (int c = 0; c < kCols; c += kPass) {
        if (left <= c) break;
        __syncwarp();                                 // the last columns have been read
#pragma unroll
        for (int h = 0; h < kPass; h += 16) {
            uint64_t o[8];
            scale16<kMx, kBias>(v + c + h, g2, gcol + c + h, bcol + c + h, o);
            uint32_t w[4 * kChunks];
            pack16<T>(o, w);
#pragma unroll
            for (int i = 0; i < kChunks; ++i)
                *reinterpret_cast<uint4*>(buf + lane * kRow + row_chunk<kRow>(lane, h / 16 * kChunks + i)) =
                    make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
        __syncwarp();
        if (sizeof(T) == 4 || words) copy_rows<uint32_t, T, kPass>(buf, out + c, ldo, rows, left - c);
        else copy_rows<uint16_t, T, kPass>(buf, out + c, ldo, rows, left - c);
    }
}
template <bool kMx, typename T, int kCols, int kPass, typename P>
__device__ __forceinline__ void write_by_row(const uint32_t* v, float ga, const float* gcol, const float* bcol, uint8_t* buf,
                                             int64_t row0, int n0, int rows, const P& p) {
    T* out = static_cast<T*>(p.out) + row0 * p.ldo + n0;
    if (p.bias)
        outputs_by_row<kMx, true, T, kCols, kPass>(v, ga, gcol, bcol, buf, out, p.ldo, rows, p.N - n0, p.align >= 0);
    else
        outputs_by_row<kMx, false, T, kCols, kPass>(v, ga, gcol, bcol, buf, out, p.ldo, rows, p.N - n0, p.align >= 0);
}

template <bool kMx, int kCols, typename P>
__device__ __forceinline__ void write_outputs(const uint32_t* v, float ga, const float* gcol, const float* bcol, int64_t r,
                                              int n0, const P& p) {
    const int64_t off = r * p.ldo + n0;
    const int left = p.N - n0;
    if (p.out_type == NVFP4_TYPE_BF16) {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + off;
        if (p.bias) outputs<kMx, true, __nv_bfloat16, kCols>(v, ga, gcol, bcol, o, left, p.align);
        else outputs<kMx, false, __nv_bfloat16, kCols>(v, ga, gcol, bcol, o, left, p.align);
    } else if (p.out_type == NVFP4_TYPE_F32) {
        float* o = static_cast<float*>(p.out) + off;
        if (p.bias) outputs<kMx, true, float, kCols>(v, ga, gcol, bcol, o, left, p.align);
        else outputs<kMx, false, float, kCols>(v, ga, gcol, bcol, o, left, p.align);
    } else {
        __half* o = static_cast<__half*>(p.out) + off;
        if (p.bias) outputs<kMx, true, __half, kCols>(v, ga, gcol, bcol, o, left, p.align);
        else outputs<kMx, false, __half, kCols>(v, ga, gcol, bcol, o, left, p.align);
    }
}

// A stage's loads of one operand in one block: expect `bytes` on bar, then the codes' box at (x, y)
// of the tensor map and `sf_bytes` of scale tiles from sf.
__device__ __forceinline__ void load_operand_elect(uint64_t* bar, uint32_t bytes, void* codes, const CUtensorMap* map, int x,
                                                   int y, void* sf_dst, const void* sf, uint32_t sf_bytes, uint64_t policy) {
    asm volatile(
        "{\n\t.reg .pred ep;\n\t.reg .b32 er;\n\telect.sync er|ep, 0xffffffff;\n\t"
        "@ep mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t"
        "@ep cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%2], [%3, {%4, %5}], [%0], %9;\n\t"
        "@ep cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%6], [%7], %8, [%0], %9;\n\t}" ::"r"(
            smem_u32(bar)),
        "r"(bytes), "r"(smem_u32(codes)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(sf_dst)),
        "l"(sf), "r"(sf_bytes), "l"(policy)
        : "memory");
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

// 3D map over scale tiles [row tiles][sf_tiles][512 bytes]: boxes of `tiles` tiles of `sets` row tiles; what
// lies outside reads as zero.
bool make_sf_map(CUtensorMap* m, const void* base, int64_t row_tiles, int64_t sf_tiles, int tiles, int sets) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {kSfAtomBytes / 4, static_cast<cuuint64_t>(sf_tiles), static_cast<cuuint64_t>(row_tiles)};
    const cuuint64_t strides[2] = {kSfAtomBytes, static_cast<cuuint64_t>(sf_tiles * kSfAtomBytes)};
    const cuuint32_t box[3] = {kSfAtomBytes / 4, static_cast<cuuint32_t>(tiles), static_cast<cuuint32_t>(sets)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;
std::mutex g_linear_mutex;

// Shared-memory attribute of a kernel (the dynamic bytes it may ask for), once per device.
template <typename... A>
cudaError_t prepare(void (*kernel)(A...), int bytes, bool (&ready)[kMaxDevices]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(g_linear_mutex);
    if (!ready[dev]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        ready[dev] = true;
    }
    return cudaSuccess;
}

// Rows of out lie on 32-byte (2), 16-byte (1), 4-byte (0) or 2-byte (-1) boundaries.
int out_align(const LinearArgs& a) {
    const int64_t bits = static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.out)) | (a.ldo * (a.out_type == NVFP4_TYPE_F32 ? 4 : 2));
    return bits % 32 == 0 ? 2 : bits % 16 == 0 ? 1 : bits % 4 == 0 ? 0 : -1;
}

}  // namespace
}  // namespace nvfp4
