// What the dense product's kernels (linear.cu, linear_pair.cu) share: the formats, instruction
// descriptors, uniform values, output stores and host-side tensor maps.
#pragma once

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
constexpr uint32_t kTmemCols = 512;
constexpr int kSmemLimit = 227 * 1024;
constexpr int kFixedBytes = 4096;                    // column data, barriers, alignment slack

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

// One stage of the main loop, in one block of PTX with one elect.sync: the scale tiles go to TMEM
// (columns sf .. , A's first, then B's kSets per tile), then nk <= 4 K=64 MMAs accumulate into d.
// sa, sb, sb2: descriptors of the scale tiles of A and of B's first and second 128 rows (the next tile
// 512 bytes, 32 units, further); a K step is 32 bytes (2 units) of the operands' rows.  kGroup: the
// CTAs of the MMA.  (As twelve separately elected instructions a stage took 730-800 cycles to issue.)
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
#define LINEAR_NV2(G, P, acc)                                                                                \
    LINEAR_CP(G, P, "ca", "s0") LINEAR_CP(G, P, "cb", "s1") "add.u32 cc, cb, 4;\n\t" LINEAR_CP(G, P, "cc", "s2") LINEAR_MMA_NV(G, P, acc, "cb")
#define LINEAR_MX1(P, Q, acc)                                                                                \
    LINEAR_CP("1", P, "ca", "s0") LINEAR_CP("1", P, "cb", "s1") "add.u32 cc, cb, %8;\n\t"                       \
        LINEAR_MMA_MX("1", P, acc, "%3", "cc") LINEAR_STEP LINEAR_MMA_MX("1", Q, "p1", "i2", "cc")
#define LINEAR_MX2(G, P, Q, acc)                                                                             \
    LINEAR_CP(G, P, "ca", "s0") LINEAR_CP(G, P, "cb", "s1") "add.u32 cc, cb, 4;\n\t" LINEAR_CP(G, P, "cc", "s2")  \
        LINEAR_MMA_MX(G, P, acc, "%3", "cb") LINEAR_STEP LINEAR_MMA_MX(G, Q, "p1", "i2", "cb")
#define LINEAR_NV2_STAGE(G)                                                                                  \
    LINEAR_BEGIN LINEAR_NV2(G, "ep", "p0") LINEAR_STEP LINEAR_NEXT("8") LINEAR_NV2(G, "e1", "p1") LINEAR_STEP    \
        LINEAR_NEXT("8") LINEAR_NV2(G, "e2", "p1") LINEAR_STEP LINEAR_NEXT("8") LINEAR_NV2(G, "e3", "p1") "}"
#define LINEAR_MX2_STAGE(G)                                                                                  \
    LINEAR_BEGIN "or.b32 i2, %3, 0x40000020;\n\t" LINEAR_MX2(G, "ep", "e1", "p0") LINEAR_STEP LINEAR_NEXT("8")   \
        LINEAR_MX2(G, "e2", "e3", "p1") "}"

template <bool kMx, int kSets, int kGroup>
__device__ __forceinline__ void issue_stage(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint64_t sa, uint64_t sb,
                                            uint64_t sb2, uint32_t sf, uint32_t sfb_col, int nk, bool accumulate) {
    static_assert(idesc_sf_id(2) == 0x40000020u, "scale-factor id of the second half of a word");
    static_assert(kGroup == 1 || kSets == 2, "variants");
    if constexpr (!kMx && kSets == 1)
        asm volatile(LINEAR_BEGIN LINEAR_NV1("ep", "p0") LINEAR_STEP LINEAR_NEXT("4") LINEAR_NV1("e1", "p1") LINEAR_STEP
                         LINEAR_NEXT("4") LINEAR_NV1("e2", "p1") LINEAR_STEP LINEAR_NEXT("4") LINEAR_NV1("e3", "p1") "}"
                     LINEAR_OPERANDS);
    else if constexpr (kSets == 1)
        asm volatile(LINEAR_BEGIN "or.b32 i2, %3, 0x40000020;\n\t" LINEAR_MX1("ep", "e1", "p0") LINEAR_STEP LINEAR_NEXT("4")
                         LINEAR_MX1("e2", "e3", "p1") "}" LINEAR_OPERANDS);
    else if constexpr (!kMx && kGroup == 1)
        asm volatile(LINEAR_NV2_STAGE("1") LINEAR_OPERANDS);
    else if constexpr (!kMx)
        asm volatile(LINEAR_NV2_STAGE("2") LINEAR_OPERANDS);
    else if constexpr (kGroup == 1)
        asm volatile(LINEAR_MX2_STAGE("1") LINEAR_OPERANDS);
    else
        asm volatile(LINEAR_MX2_STAGE("2") LINEAR_OPERANDS);
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
#undef LINEAR_NV2_STAGE
#undef LINEAR_MX2_STAGE

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

// Rows of out start and end on 16-byte boundaries.
int out_vec(const LinearArgs& a) {
    const int size = a.out_type == NVFP4_TYPE_F32 ? 4 : 2;
    return (reinterpret_cast<uintptr_t>(a.out) & 15) == 0 && (a.ldo * size) % 16 == 0;
}

}  // namespace
}  // namespace nvfp4
