// C ABI of the NVFP4 MoE expert forward: argument validation, workspace
// layout, per-device state (error word, SM count) and the launch sequences.
// The operations themselves are documented in include/nvfp4_moe.h.
#include <cstring>
#include <mutex>

#include "backward.cuh"
#include "common.cuh"
#include "ops.cuh"

namespace nvfp4 {

// First device-side error since the last nvfp4_get_device_error (0 = none).
__device__ int g_device_error;

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_dev_mutex;
int* g_err_ptr[kMaxDevices];
void* g_err_ctx[kMaxDevices];
int g_sm_count[kMaxDevices];

using CtxGetCurrentFn = CUresult (*)(CUcontext*);

CtxGetCurrentFn ctx_get_current_fn() {
    static CtxGetCurrentFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess) {
            fn = reinterpret_cast<CtxGetCurrentFn>(p);
        }
    });
    return fn;
}

int current_device() {
    int d = -1;
    if (cudaGetDevice(&d) != cudaSuccess) return -1;
    return (d >= 0 && d < kMaxDevices) ? d : -1;
}

// Device address of this device's error word (looked up once per device and context).
int* device_error_ptr() {
    const int d = current_device();
    if (d < 0) return nullptr;
    void* ctx = current_context();
    std::lock_guard<std::mutex> lock(g_dev_mutex);
    if (!g_err_ptr[d] || g_err_ctx[d] != ctx) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_device_error) != cudaSuccess) return nullptr;
        g_err_ptr[d] = static_cast<int*>(p);
        g_err_ctx[d] = ctx;
    }
    return g_err_ptr[d];
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool moe_shape_ok(int64_t T, int H, int I, int E, int k) {
    if (T < 0 || E < 1 || E > 1024 || k < 1 || k > 32 || k > E) return false;
    if (H < 256 || H > 8192 || H % 256) return false;
    if (I < 128 || I > 8192 || I % 128) return false;
    if (T * static_cast<int64_t>(k) >= (int64_t(1) << 30)) return false;
    return true;
}

// capacity > 0: the fixed-capacity layout, E*capacity routed rows (expert e at e*capacity).
void compute_layout(int64_t T, int H, int I, int E, int k, moe_workspace_layout* L, int capacity = 0) {
    std::memset(L, 0, sizeof(*L));
    L->T = T;
    L->H = H;
    L->I = I;
    L->E = E;
    L->k = k;
    const int64_t R = T * k;
    const int64_t live_experts = R < E ? R : E;
    L->rows_cap = capacity > 0 ? static_cast<int64_t>(E) * capacity
                               : (R + live_experts * (kTileM - 1) + kTileM - 1) / kTileM * kTileM;
    L->n_chunks = (T + 255) / 256;
    const int64_t rc = L->rows_cap;
    size_t o = 0;
    auto take = [&o](size_t bytes) {
        const size_t at = o;
        o = align_up(o + bytes, 256);
        return at;
    };
    L->a_codes = take(rc * H / 2);
    L->a_sf = take(rc * H / 16);
    L->a_g = take(rc * 4);
    L->row_pair = take(rc * 4);
    L->row_prob = take(rc * 4);
    L->amax2 = take(rc * 4);
    L->pair_row = take(R * 4);
    L->a_sf_rows = take(rc * H / 16);
    L->chunk_count = take(static_cast<size_t>(E) * L->n_chunks * 4);
    L->chunk_base = take(static_cast<size_t>(E) * L->n_chunks * 4);
    L->pair_rank = take(R * 4);
    L->expert_count = take(static_cast<size_t>(E) * 4);
    L->route_end = o;
    L->h = take(rc * I * 2);
    L->a2_codes = take(rc * I / 2);
    L->a2_sf = take(rc * I / 16);
    L->a2_g = take(rc * 4);
    L->y = take(rc * H * 2);
    L->total = o;
}

// Scratch of the straight-through backward (sizes from the forward's contiguous layout).
void compute_backward_layout(int64_t T, int H, int I, int E, int k, moe_backward_layout* B) {
    moe_workspace_layout L;
    compute_layout(T, H, I, E, k, &L);
    std::memset(B, 0, sizeof(*B));
    B->T = T;
    B->H = H;
    B->I = I;
    B->E = E;
    B->k = k;
    const int64_t rc = L.rows_cap;
    B->rows_cap = rc;
    size_t o = 0;
    auto take = [&o](size_t bytes) {
        const size_t at = o;
        o = align_up(o + bytes, 256);
        return at;
    };
    B->dy_rows = take(rc * H * 2);
    B->dh = take(rc * I * 2);
    B->dgu = take(rc * 2 * I * 2);
    B->dx_pairs = take(T * k * H * 2);
    B->x_rows = take(rc * H * 2);
    B->real_end = take(static_cast<size_t>(E) * 4);
    B->total = o;
}

// The CUDA error behind the calling thread's last NVFP4_ERR_CUDA (cudaSuccess if none yet).
thread_local cudaError_t t_last_cuda_error = cudaSuccess;

nvfp4_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return NVFP4_OK;
    t_last_cuda_error = e;
    return NVFP4_ERR_CUDA;
}

template <typename T>
T* at(void* ws, size_t off) {
    return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

// Shared validation of the calls that run on a filled workspace.
bool capacity_ok(int E, int capacity) {
    return capacity >= kTileM && capacity % kTileM == 0 && static_cast<int64_t>(E) * capacity < (int64_t(1) << 30);
}

nvfp4_status check_forward_args(const moe_nvfp4_weights* w, int64_t T, int k, const void* ws, size_t ws_bytes,
                                moe_workspace_layout* L, int capacity = 0) {
    if (!w || !ws) return NVFP4_ERR_INVALID_ARG;
    if (!w->w1_codes || !w->w1_sf || !w->w1_g || !w->w2_codes || !w->w2_sf || !w->w2_g) return NVFP4_ERR_INVALID_ARG;
    if (!aligned(w->w1_codes, 16) || !aligned(w->w1_sf, 16) || !aligned(w->w2_codes, 16) || !aligned(w->w2_sf, 16) ||
        !aligned(ws, 256))
        return NVFP4_ERR_INVALID_ARG;
    if (!moe_shape_ok(T, w->H, w->I, w->E, k)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (capacity != 0 && !capacity_ok(w->E, capacity)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    compute_layout(T, w->H, w->I, w->E, k, L, capacity);
    if (ws_bytes < L->total) return NVFP4_ERR_WORKSPACE_TOO_SMALL;
    return NVFP4_OK;
}

GemmArgs fc1_args(const moe_nvfp4_weights* w, const int32_t* offsets, void* ws, const moe_workspace_layout& L,
                  float* debug, int* err) {
    GemmArgs a{};
    a.a_codes = at<uint8_t>(ws, L.a_codes);
    a.a_sf = at<uint8_t>(ws, L.a_sf);
    a.a_g = at<float>(ws, L.a_g);
    a.b_codes = static_cast<const uint8_t*>(w->w1_codes);
    a.b_sf = static_cast<const uint8_t*>(w->w1_sf);
    a.b_g = w->w1_g;
    a.rows_cap = L.rows_cap;
    a.K = w->H;
    a.Nw = 2 * w->I;
    a.E = w->E;
    a.offsets = offsets;
    a.row_pair = at<int32_t>(ws, L.row_pair);
    a.row_prob = at<float>(ws, L.row_prob);
    a.I = w->I;
    a.h = at<uint16_t>(ws, L.h);
    a.amax2 = at<uint32_t>(ws, L.amax2);
    a.H = w->H;
    a.y = nullptr;
    a.debug = debug;
    a.err = err;
    return a;
}

GemmArgs fc2_args(const moe_nvfp4_weights* w, const int32_t* offsets, void* ws, const moe_workspace_layout& L,
                  float* debug, int* err) {
    GemmArgs a{};
    a.a_codes = at<uint8_t>(ws, L.a2_codes);
    a.a_sf = at<uint8_t>(ws, L.a2_sf);
    a.a_g = at<float>(ws, L.a2_g);
    a.b_codes = static_cast<const uint8_t*>(w->w2_codes);
    a.b_sf = static_cast<const uint8_t*>(w->w2_sf);
    a.b_g = w->w2_g;
    a.rows_cap = L.rows_cap;
    a.K = w->I;
    a.Nw = w->H;
    a.E = w->E;
    a.offsets = offsets;
    a.row_pair = at<int32_t>(ws, L.row_pair);
    a.row_prob = at<float>(ws, L.row_prob);
    a.I = w->I;
    a.h = nullptr;
    a.amax2 = nullptr;
    a.H = w->H;
    a.y = at<uint16_t>(ws, L.y);
    a.debug = debug;
    a.err = err;
    return a;
}

}  // namespace

int* device_error_word() { return device_error_ptr(); }

void* current_context() {
    CtxGetCurrentFn fn = ctx_get_current_fn();
    CUcontext c = nullptr;
    if (!fn || fn(&c) != CUDA_SUCCESS) return nullptr;
    return c;
}

int device_sm_count() {
    const int d = current_device();
    if (d < 0) return 1;
    std::lock_guard<std::mutex> lock(g_dev_mutex);
    if (!g_sm_count[d]) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d) != cudaSuccess || n < 1) n = 1;
        g_sm_count[d] = n;
    }
    return g_sm_count[d];
}

}  // namespace nvfp4

using namespace nvfp4;

namespace nvfp4 {
// defined in quant.cu: the route sort with an optional fixed capacity per expert
cudaError_t launch_route_sort_quant_cap(const uint16_t* x, int64_t T, int H, int E, int k, const int32_t* ids,
                                        const float* probs, int32_t* offsets, const RouteBufs& b, int capacity,
                                        int* err, cudaStream_t st);
// defined in router.cu
cudaError_t launch_router_topk(const uint16_t* x, int64_t T, int H, const uint16_t* w, int E, int k, int32_t* ids,
                               float* probs, float* logits, int* err, cudaStream_t st);
}  // namespace nvfp4

extern "C" {

const char* nvfp4_status_string(int status) {
    switch (status) {
        case NVFP4_OK: return "NVFP4_OK";
        case NVFP4_ERR_INVALID_ARG: return "NVFP4_ERR_INVALID_ARG";
        case NVFP4_ERR_UNSUPPORTED_SHAPE: return "NVFP4_ERR_UNSUPPORTED_SHAPE";
        case NVFP4_ERR_WORKSPACE_TOO_SMALL: return "NVFP4_ERR_WORKSPACE_TOO_SMALL";
        case NVFP4_ERR_CUDA: return "NVFP4_ERR_CUDA";
        case NVFP4_ERR_BAD_EXPERT_ID: return "NVFP4_ERR_BAD_EXPERT_ID";
        case NVFP4_ERR_NONFINITE: return "NVFP4_ERR_NONFINITE";
        case NVFP4_ERR_DEVICE_TIMEOUT: return "NVFP4_ERR_DEVICE_TIMEOUT";
        case NVFP4_ERR_CAPACITY: return "NVFP4_ERR_CAPACITY";
        default: return "NVFP4_UNKNOWN_STATUS";
    }
}

int64_t nvfp4_rows_padded(int64_t rows) {
    if (rows < 0) return 0;
    return (rows + kTileM - 1) / kTileM * kTileM;
}

size_t nvfp4_sf_bytes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols <= 0 || cols % 64) return 0;
    return static_cast<size_t>(nvfp4_rows_padded(rows)) * static_cast<size_t>(cols / 16);
}

nvfp4_status nvfp4_quantize_rows(const void* x_dev, int64_t rows, int64_t cols, int64_t ld, void* codes_dev,
                                 void* sf_dev, float* g_dev, void* stream) {
    if (rows < 0 || cols < 64 || cols > 8192 || cols % 64 || ld < cols || ld % 8) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return NVFP4_OK;
    if (!x_dev || !codes_dev || !sf_dev || !g_dev) return NVFP4_ERR_INVALID_ARG;
    if (!aligned(x_dev, 16) || !aligned(codes_dev, 32) || !aligned(sf_dev, 16) || !aligned(g_dev, 4))
        return NVFP4_ERR_INVALID_ARG;
    int* err = device_error_ptr();
    if (!err) return NVFP4_ERR_CUDA;
    return from_cuda(launch_quantize_rows(static_cast<const uint16_t*>(x_dev), rows, cols, ld,
                                          static_cast<uint8_t*>(codes_dev), static_cast<uint8_t*>(sf_dev), g_dev, err,
                                          static_cast<cudaStream_t>(stream)));
}

nvfp4_status moe_workspace_layout_query(int64_t T, int H, int I, int E, int k, moe_workspace_layout* out) {
    if (!out) return NVFP4_ERR_INVALID_ARG;
    if (!moe_shape_ok(T, H, I, E, k)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    compute_layout(T, H, I, E, k, out);
    return NVFP4_OK;
}

size_t moe_workspace_bytes(int64_t T, int H, int I, int E, int k) {
    if (!moe_shape_ok(T, H, I, E, k)) return 0;
    moe_workspace_layout L;
    compute_layout(T, H, I, E, k, &L);
    return L.total;
}

static nvfp4_status route_impl(const void* x_dev, int64_t T, int H, int E, int k, const int32_t* topk_ids_dev,
                               const float* topk_w_dev, int32_t* expert_offsets_dev, void* ws_dev, size_t ws_bytes,
                               int capacity, void* stream) {
    if (!moe_shape_ok(T, H, 128, E, k)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (capacity != 0 && !capacity_ok(E, capacity)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (!expert_offsets_dev || !ws_dev) return NVFP4_ERR_INVALID_ARG;
    if (T > 0 && (!x_dev || !topk_ids_dev || !topk_w_dev)) return NVFP4_ERR_INVALID_ARG;
    if (!aligned(x_dev, 16) || !aligned(ws_dev, 256) || !aligned(topk_ids_dev, 4) || !aligned(topk_w_dev, 4) ||
        !aligned(expert_offsets_dev, 4))
        return NVFP4_ERR_INVALID_ARG;
    moe_workspace_layout L;
    compute_layout(T, H, 128, E, k, &L, capacity);
    if (ws_bytes < L.route_end) return NVFP4_ERR_WORKSPACE_TOO_SMALL;
    int* err = device_error_ptr();
    if (!err) return NVFP4_ERR_CUDA;
    RouteBufs b;
    b.a_codes = at<uint8_t>(ws_dev, L.a_codes);
    b.a_sf = at<uint8_t>(ws_dev, L.a_sf);
    b.a_g = at<float>(ws_dev, L.a_g);
    b.row_pair = at<int32_t>(ws_dev, L.row_pair);
    b.row_prob = at<float>(ws_dev, L.row_prob);
    b.amax2 = at<uint32_t>(ws_dev, L.amax2);
    b.pair_row = at<int32_t>(ws_dev, L.pair_row);
    b.a_sf_rows = at<uint8_t>(ws_dev, L.a_sf_rows);
    b.rows_cap = L.rows_cap;
    b.chunk_count = at<int32_t>(ws_dev, L.chunk_count);
    b.chunk_base = at<int32_t>(ws_dev, L.chunk_base);
    b.pair_rank = at<int32_t>(ws_dev, L.pair_rank);
    b.expert_count = at<int32_t>(ws_dev, L.expert_count);
    b.n_chunks = L.n_chunks;
    return from_cuda(launch_route_sort_quant_cap(static_cast<const uint16_t*>(x_dev), T, H, E, k, topk_ids_dev,
                                                 topk_w_dev, expert_offsets_dev, b, capacity, err,
                                                 static_cast<cudaStream_t>(stream)));
}

nvfp4_status moe_route_sort_amax(const void* x_dev, int64_t T, int H, int E, int k, const int32_t* topk_ids_dev,
                                 const float* topk_w_dev, int32_t* expert_offsets_dev, void* ws_dev, size_t ws_bytes,
                                 void* stream) {
    return route_impl(x_dev, T, H, E, k, topk_ids_dev, topk_w_dev, expert_offsets_dev, ws_dev, ws_bytes, 0, stream);
}

nvfp4_status moe_route_sort_amax_masked(const void* x_dev, int64_t T, int H, int E, int k,
                                        const int32_t* topk_ids_dev, const float* topk_w_dev, int capacity,
                                        int32_t* expert_offsets_dev, void* ws_dev, size_t ws_bytes, void* stream) {
    if (capacity == 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    return route_impl(x_dev, T, H, E, k, topk_ids_dev, topk_w_dev, expert_offsets_dev, ws_dev, ws_bytes, capacity,
                      stream);
}

nvfp4_status moe_workspace_layout_query_masked(int64_t T, int H, int I, int E, int k, int capacity,
                                               moe_workspace_layout* out) {
    if (!out) return NVFP4_ERR_INVALID_ARG;
    if (!moe_shape_ok(T, H, I, E, k) || !capacity_ok(E, capacity)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    compute_layout(T, H, I, E, k, out, capacity);
    return NVFP4_OK;
}

size_t moe_workspace_bytes_masked(int64_t T, int H, int I, int E, int k, int capacity) {
    if (!moe_shape_ok(T, H, I, E, k) || !capacity_ok(E, capacity)) return 0;
    moe_workspace_layout L;
    compute_layout(T, H, I, E, k, &L, capacity);
    return L.total;
}

static nvfp4_status moe_fc1_swiglu_nvfp4_impl(const moe_nvfp4_weights* w, int64_t T, int k, const int32_t* expert_offsets_dev,
                                  void* ws_dev, size_t ws_bytes, float* fc1_debug_dev, void* stream, bool pdl, int capacity = 0,
                                  uint16_t* gu_save = nullptr) {
    moe_workspace_layout L;
    const nvfp4_status s = check_forward_args(w, T, k, ws_dev, ws_bytes, &L, capacity);
    if (s != NVFP4_OK) return s;
    if (!expert_offsets_dev) return NVFP4_ERR_INVALID_ARG;
    if (T == 0) return NVFP4_OK;
    int* err = device_error_ptr();
    if (!err) return NVFP4_ERR_CUDA;
    GemmArgs a = fc1_args(w, expert_offsets_dev, ws_dev, L, fc1_debug_dev, err);
    a.gu_save = gu_save;
    return from_cuda(launch_fc1(a, static_cast<cudaStream_t>(stream), pdl));
}

static nvfp4_status moe_requant_nvfp4_impl(const moe_nvfp4_weights* w, int64_t T, int k, const int32_t* expert_offsets_dev,
                               void* ws_dev, size_t ws_bytes, void* stream, bool pdl, int capacity = 0) {
    moe_workspace_layout L;
    const nvfp4_status s = check_forward_args(w, T, k, ws_dev, ws_bytes, &L, capacity);
    if (s != NVFP4_OK) return s;
    if (!expert_offsets_dev) return NVFP4_ERR_INVALID_ARG;
    if (T == 0) return NVFP4_OK;
    int* err = device_error_ptr();
    if (!err) return NVFP4_ERR_CUDA;
    return from_cuda(launch_requant(at<uint16_t>(ws_dev, L.h), at<uint32_t>(ws_dev, L.amax2),
                                    at<int32_t>(ws_dev, L.row_pair), expert_offsets_dev, w->E, L.rows_cap, w->I,
                                    at<uint8_t>(ws_dev, L.a2_codes), at<uint8_t>(ws_dev, L.a2_sf),
                                    at<float>(ws_dev, L.a2_g), err, static_cast<cudaStream_t>(stream), pdl));
}

static nvfp4_status moe_fc2_nvfp4_impl(const moe_nvfp4_weights* w, int64_t T, int k, const int32_t* expert_offsets_dev,
                           void* ws_dev, size_t ws_bytes, float* fc2_debug_dev, void* stream, bool pdl, int capacity = 0) {
    moe_workspace_layout L;
    const nvfp4_status s = check_forward_args(w, T, k, ws_dev, ws_bytes, &L, capacity);
    if (s != NVFP4_OK) return s;
    if (!expert_offsets_dev) return NVFP4_ERR_INVALID_ARG;
    if (T == 0) return NVFP4_OK;
    int* err = device_error_ptr();
    if (!err) return NVFP4_ERR_CUDA;
    return from_cuda(launch_fc2(fc2_args(w, expert_offsets_dev, ws_dev, L, fc2_debug_dev, err),
                                static_cast<cudaStream_t>(stream), pdl));
}

static nvfp4_status moe_fc2_requant_nvfp4_impl(const moe_nvfp4_weights* w, int64_t T, int k,
                                               const int32_t* expert_offsets_dev, void* ws_dev, size_t ws_bytes,
                                               float* fc2_debug_dev, void* stream, bool pdl, int capacity = 0) {
    moe_workspace_layout L;
    const nvfp4_status s = check_forward_args(w, T, k, ws_dev, ws_bytes, &L, capacity);
    if (s != NVFP4_OK) return s;
    if (w->I > fc2_requant_max_i() || w->E > fc2_requant_max_e()) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (!expert_offsets_dev) return NVFP4_ERR_INVALID_ARG;
    if (T == 0) return NVFP4_OK;
    int* err = device_error_ptr();
    if (!err) return NVFP4_ERR_CUDA;
    GemmArgs a = fc2_args(w, expert_offsets_dev, ws_dev, L, fc2_debug_dev, err);
    a.h = at<uint16_t>(ws_dev, L.h);             // the FC2 input before requantisation, and its maxima
    a.amax2 = at<uint32_t>(ws_dev, L.amax2);
    return from_cuda(launch_fc2_requant(a, static_cast<cudaStream_t>(stream), pdl));
}

static nvfp4_status moe_combine_bf16_impl(const moe_nvfp4_weights* w, int64_t T, int k, void* out_dev, void* ws_dev,
                              size_t ws_bytes, void* stream, bool pdl, int capacity = 0) {
    moe_workspace_layout L;
    const nvfp4_status s = check_forward_args(w, T, k, ws_dev, ws_bytes, &L, capacity);
    if (s != NVFP4_OK) return s;
    if (T == 0) return NVFP4_OK;
    if (!out_dev || !aligned(out_dev, 16)) return NVFP4_ERR_INVALID_ARG;
    return from_cuda(launch_combine(at<uint16_t>(ws_dev, L.y), at<int32_t>(ws_dev, L.pair_row), T, k, w->H,
                                    static_cast<uint16_t*>(out_dev),
                                    static_cast<cudaStream_t>(stream), pdl));
}

// FC1, the FC2 input's requantisation, FC2, the combine; every kernel after FC1 starts early
// (programmatic dependent launch) and waits on its predecessor in the device.  The forward runs
// requant and FC2 as two kernels: on GB300 at the measured sizes that is faster than the fused
// moe_fc2_requant_nvfp4 (same bits), whose in-kernel quantisation is issue-bound on the few
// warps the FC2 kernel's registers and shared memory leave for it.
static nvfp4_status forward_stages(const moe_nvfp4_weights* w, int64_t T, int k, const int32_t* offs, void* out_dev,
                                   void* ws_dev, size_t ws_bytes, void* stream, int capacity, bool pdl_fc1 = false) {
    nvfp4_status s = moe_fc1_swiglu_nvfp4_impl(w, T, k, offs, ws_dev, ws_bytes, nullptr, stream, pdl_fc1, capacity);
    if (s != NVFP4_OK) return s;
    s = moe_requant_nvfp4_impl(w, T, k, offs, ws_dev, ws_bytes, stream, true, capacity);
    if (s != NVFP4_OK) return s;
    s = moe_fc2_nvfp4_impl(w, T, k, offs, ws_dev, ws_bytes, nullptr, stream, true, capacity);
    if (s != NVFP4_OK) return s;
    return moe_combine_bf16_impl(w, T, k, out_dev, ws_dev, ws_bytes, stream, true, capacity);
}

// The stage entry points: each one's kernel is ordered after all earlier work on the stream.
nvfp4_status moe_fc1_swiglu_nvfp4(const moe_nvfp4_weights* w, int64_t T, int k, const int32_t* expert_offsets_dev,
                                  void* ws_dev, size_t ws_bytes, float* fc1_debug_dev, void* stream) {
    return moe_fc1_swiglu_nvfp4_impl(w, T, k, expert_offsets_dev, ws_dev, ws_bytes, fc1_debug_dev, stream, false);
}

nvfp4_status moe_fc1_swiglu_save_nvfp4(const moe_nvfp4_weights* w, int64_t T, int k, const int32_t* expert_offsets_dev,
                                       void* ws_dev, size_t ws_bytes, void* gu_save_dev, void* stream) {
    if (!gu_save_dev || !aligned(gu_save_dev, 4)) return NVFP4_ERR_INVALID_ARG;
    return moe_fc1_swiglu_nvfp4_impl(w, T, k, expert_offsets_dev, ws_dev, ws_bytes, nullptr, stream, false, 0,
                                     static_cast<uint16_t*>(gu_save_dev));
}

nvfp4_status moe_requant_nvfp4(const moe_nvfp4_weights* w, int64_t T, int k, const int32_t* expert_offsets_dev,
                               void* ws_dev, size_t ws_bytes, void* stream) {
    return moe_requant_nvfp4_impl(w, T, k, expert_offsets_dev, ws_dev, ws_bytes, stream, false);
}

nvfp4_status moe_fc2_nvfp4(const moe_nvfp4_weights* w, int64_t T, int k, const int32_t* expert_offsets_dev,
                           void* ws_dev, size_t ws_bytes, float* fc2_debug_dev, void* stream) {
    return moe_fc2_nvfp4_impl(w, T, k, expert_offsets_dev, ws_dev, ws_bytes, fc2_debug_dev, stream, false);
}

nvfp4_status moe_combine_bf16(const moe_nvfp4_weights* w, int64_t T, int k, void* out_dev, void* ws_dev,
                              size_t ws_bytes, void* stream) {
    return moe_combine_bf16_impl(w, T, k, out_dev, ws_dev, ws_bytes, stream, false);
}

nvfp4_status moe_fc2_requant_nvfp4(const moe_nvfp4_weights* w, int64_t T, int k, const int32_t* expert_offsets_dev,
                                   void* ws_dev, size_t ws_bytes, float* fc2_debug_dev, void* stream) {
    return moe_fc2_requant_nvfp4_impl(w, T, k, expert_offsets_dev, ws_dev, ws_bytes, fc2_debug_dev, stream, false);
}

int moe_fc2_requant_max_intermediate(void) { return fc2_requant_max_i(); }

nvfp4_status moe_expert_forward_nvfp4(const moe_nvfp4_weights* w, int64_t T, int k, const int32_t* expert_offsets_dev,
                                      void* out_dev, void* ws_dev, size_t ws_bytes, void* stream) {
    moe_workspace_layout L;
    nvfp4_status s = check_forward_args(w, T, k, ws_dev, ws_bytes, &L);
    if (s != NVFP4_OK) return s;
    if (T == 0) return NVFP4_OK;
    if (!expert_offsets_dev || !out_dev || !aligned(out_dev, 16)) return NVFP4_ERR_INVALID_ARG;
    return forward_stages(w, T, k, expert_offsets_dev, out_dev, ws_dev, ws_bytes, stream, 0);
}

// Route sort + quantise and the expert forward in one call: every argument of both is checked
// before anything is launched, and FC1 is launched as a programmatic dependent of the route's
// last kernel (its set-up overlaps that kernel's tail; its reads of the routed rows wait for
// the route to complete), which the two separate calls cannot do.
nvfp4_status moe_layer_forward_nvfp4(const moe_nvfp4_weights* w, const void* x_dev, int64_t T, int k,
                                     const int32_t* topk_ids_dev, const float* topk_w_dev,
                                     int32_t* expert_offsets_dev, void* out_dev, void* ws_dev, size_t ws_bytes,
                                     void* stream) {
    moe_workspace_layout L;
    nvfp4_status s = check_forward_args(w, T, k, ws_dev, ws_bytes, &L);
    if (s != NVFP4_OK) return s;
    if (T > 0 && (!out_dev || !aligned(out_dev, 16))) return NVFP4_ERR_INVALID_ARG;
    s = route_impl(x_dev, T, w->H, w->E, k, topk_ids_dev, topk_w_dev, expert_offsets_dev, ws_dev, ws_bytes, 0,
                   stream);
    if (s != NVFP4_OK || T == 0) return s;
    return forward_stages(w, T, k, expert_offsets_dev, out_dev, ws_dev, ws_bytes, stream, 0, true);
}

nvfp4_status moe_router_topk(const void* x_dev, int64_t T, int H, const void* w_router_dev, int E, int k,
                             int32_t* topk_ids_dev, float* topk_w_dev, float* logits_dev, void* stream) {
    if (T < 0 || H <= 0 || H % 64 != 0 || H > (1 << 20) || E < 16 || E > 256 || E % 16 != 0 || k < 1 || k > E ||
        k > 32)
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return NVFP4_OK;
    if (!x_dev || !w_router_dev || !topk_ids_dev || !topk_w_dev) return NVFP4_ERR_INVALID_ARG;
    if (!aligned(x_dev, 16) || !aligned(w_router_dev, 16) || !aligned(topk_ids_dev, 4) || !aligned(topk_w_dev, 4) ||
        (logits_dev && !aligned(logits_dev, 32)))
        return NVFP4_ERR_INVALID_ARG;
    int* err = device_error_ptr();
    if (!err) return NVFP4_ERR_CUDA;
    return from_cuda(launch_router_topk(static_cast<const uint16_t*>(x_dev), T, H,
                                        static_cast<const uint16_t*>(w_router_dev), E, k, topk_ids_dev, topk_w_dev,
                                        logits_dev, err, static_cast<cudaStream_t>(stream)));
}

nvfp4_status moe_expert_forward_nvfp4_masked(const moe_nvfp4_weights* w, int64_t T, int k, int capacity,
                                             const int32_t* expert_offsets_dev, void* out_dev, void* ws_dev,
                                             size_t ws_bytes, void* stream) {
    if (capacity == 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    moe_workspace_layout L;
    nvfp4_status s = check_forward_args(w, T, k, ws_dev, ws_bytes, &L, capacity);
    if (s != NVFP4_OK) return s;
    if (T == 0) return NVFP4_OK;
    if (!expert_offsets_dev || !out_dev || !aligned(out_dev, 16)) return NVFP4_ERR_INVALID_ARG;
    return forward_stages(w, T, k, expert_offsets_dev, out_dev, ws_dev, ws_bytes, stream, capacity);
}

nvfp4_status moe_layer_forward_nvfp4_masked(const moe_nvfp4_weights* w, const void* x_dev, int64_t T, int k,
                                            const int32_t* topk_ids_dev, const float* topk_w_dev, int capacity,
                                            int32_t* expert_offsets_dev, void* out_dev, void* ws_dev,
                                            size_t ws_bytes, void* stream) {
    if (capacity == 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    moe_workspace_layout L;
    nvfp4_status s = check_forward_args(w, T, k, ws_dev, ws_bytes, &L, capacity);
    if (s != NVFP4_OK) return s;
    if (T > 0 && (!out_dev || !aligned(out_dev, 16))) return NVFP4_ERR_INVALID_ARG;
    s = route_impl(x_dev, T, w->H, w->E, k, topk_ids_dev, topk_w_dev, expert_offsets_dev, ws_dev, ws_bytes,
                   capacity, stream);
    if (s != NVFP4_OK || T == 0) return s;
    return forward_stages(w, T, k, expert_offsets_dev, out_dev, ws_dev, ws_bytes, stream, capacity, true);
}

nvfp4_status moe_backward_layout_query(int64_t T, int H, int I, int E, int k, moe_backward_layout* out) {
    if (!out) return NVFP4_ERR_INVALID_ARG;
    if (!moe_shape_ok(T, H, I, E, k)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    compute_backward_layout(T, H, I, E, k, out);
    return NVFP4_OK;
}

size_t moe_backward_workspace_bytes(int64_t T, int H, int I, int E, int k) {
    if (!moe_shape_ok(T, H, I, E, k)) return 0;
    moe_backward_layout B;
    compute_backward_layout(T, H, I, E, k, &B);
    return B.total;
}

nvfp4_status moe_expert_backward_ste(const moe_bf16_weights_t* w, int64_t T, int k, const void* x_dev,
                                     const void* dout_dev, const int32_t* expert_offsets_dev, const void* fwd_ws_dev,
                                     size_t fwd_ws_bytes, const void* gu_dev, void* dx_dev, float* dw1_dev,
                                     float* dw2_dev, float* dprob_dev, void* bwd_ws_dev, size_t bwd_ws_bytes,
                                     void* stream) {
    if (!w) return NVFP4_ERR_INVALID_ARG;
    if (!moe_shape_ok(T, w->H, w->I, w->E, k)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (!w->w1 || !w->w2 || !dw1_dev || !dw2_dev) return NVFP4_ERR_INVALID_ARG;
    if (!aligned(w->w1, 16) || !aligned(w->w2, 16) || !aligned(dw1_dev, 32) || !aligned(dw2_dev, 32))
        return NVFP4_ERR_INVALID_ARG;
    const int H = w->H, I = w->I, E = w->E;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        cudaError_t e = cudaMemsetAsync(dw1_dev, 0, static_cast<size_t>(E) * 2 * I * H * 4, st);
        if (e == cudaSuccess) e = cudaMemsetAsync(dw2_dev, 0, static_cast<size_t>(E) * H * I * 4, st);
        return from_cuda(e);
    }
    if (!x_dev || !dout_dev || !expert_offsets_dev || !fwd_ws_dev || !gu_dev || !dx_dev || !dprob_dev ||
        !bwd_ws_dev)
        return NVFP4_ERR_INVALID_ARG;
    if (!aligned(x_dev, 16) || !aligned(dout_dev, 16) || !aligned(expert_offsets_dev, 4) || !aligned(fwd_ws_dev, 256) ||
        !aligned(gu_dev, 16) || !aligned(dx_dev, 16) || !aligned(dprob_dev, 4) || !aligned(bwd_ws_dev, 256))
        return NVFP4_ERR_INVALID_ARG;
    moe_workspace_layout L;
    compute_layout(T, H, I, E, k, &L);
    // the backward's GEMMs address routed rows as int32 tensor-map coordinates
    if (L.rows_cap >= (int64_t(1) << 30)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    moe_backward_layout B;
    compute_backward_layout(T, H, I, E, k, &B);
    if (fwd_ws_bytes < L.total || bwd_ws_bytes < B.total) return NVFP4_ERR_WORKSPACE_TOO_SMALL;
    int* err = device_error_ptr();
    if (!err) return NVFP4_ERR_CUDA;
    void* fws = const_cast<void*>(fwd_ws_dev);
    BackwardArgs a{};
    a.T = T;
    a.H = H;
    a.I = I;
    a.E = E;
    a.k = k;
    a.rows_cap = L.rows_cap;
    a.w1 = static_cast<const uint16_t*>(w->w1);
    a.w2 = static_cast<const uint16_t*>(w->w2);
    a.x = static_cast<const uint16_t*>(x_dev);
    a.dout = static_cast<const uint16_t*>(dout_dev);
    a.offsets = expert_offsets_dev;
    a.row_pair = at<int32_t>(fws, L.row_pair);
    a.row_prob = at<float>(fws, L.row_prob);
    a.h = at<uint16_t>(fws, L.h);
    a.gu = static_cast<const uint16_t*>(gu_dev);
    a.dx = static_cast<uint16_t*>(dx_dev);
    a.dw1 = dw1_dev;
    a.dw2 = dw2_dev;
    a.dprob = dprob_dev;
    a.dy_rows = at<uint16_t>(bwd_ws_dev, B.dy_rows);
    a.dh = at<uint16_t>(bwd_ws_dev, B.dh);
    a.dgu = at<uint16_t>(bwd_ws_dev, B.dgu);
    a.dx_pairs = at<uint16_t>(bwd_ws_dev, B.dx_pairs);
    a.x_rows = at<uint16_t>(bwd_ws_dev, B.x_rows);
    a.real_end = at<int32_t>(bwd_ws_dev, B.real_end);
    a.err = err;
    return from_cuda(launch_moe_backward_ste(a, st));
}

// ---- routing of given logits, and the dense 4-bit products

namespace {

int type_size(int type) { return type == NVFP4_TYPE_F32 ? 4 : 2; }
bool type_ok(int type) { return type == NVFP4_TYPE_F32 || type == NVFP4_TYPE_BF16 || type == NVFP4_TYPE_F16; }

// Every row start rows are read or written at stays inside 63-bit byte offsets.
bool rows_ok(int64_t rows, int64_t ld) { return ld <= 0 || rows <= (int64_t(1) << 60) / ld; }

// Whether two sets of `rows` rows share a byte: of bytes_a and bytes_b bytes each, pitch_a and pitch_b (at least as many)
// apart.  Rows side by side in one buffer do not.
bool rows_overlap(const void* a, int64_t pitch_a, int64_t bytes_a, const void* b, int64_t pitch_b, int64_t bytes_b,
                  int64_t rows) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    const uintptr_t pa = pitch_a, pb = pitch_b, na = bytes_a, nb = bytes_b, last = rows - 1;
    if (a0 + last * pa + na <= b0 || b0 + last * pb + nb <= a0) return false;
    if (pa == pb) {                                   // b's rows start d bytes behind a's
        const uintptr_t d = b0 >= a0 ? (b0 - a0) % pa : (pa - (a0 - b0) % pa) % pa;
        return rows == 1 || d < na || d + nb > pa;
    }
    for (uintptr_t i = 0, j = 0; i <= last && j <= last;) {
        if (a0 + i * pa + na <= b0 + j * pb) ++i;
        else if (b0 + j * pb + nb <= a0 + i * pa) ++j;
        else return true;
    }
    return false;
}

// The parameters both routing calls use.
bool route_params_ok(const moe_route_params& p, int E) {
    return (p.score == MOE_SCORE_SOFTMAX || p.score == MOE_SCORE_SIGMOID) && (p.renormalize == 0 || p.renormalize == 1) &&
           p.k >= 1 && p.k <= 32 && p.k <= E && p.scale - p.scale == 0.0f;
}

RouteParams route_params(const moe_route_params& p) {
    return {p.score, p.k, p.n_group, p.topk_group, p.group_score, p.renormalize, p.scale, 0, 0, 0};
}

constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 256;
constexpr int64_t kMaxMxCols = int64_t(1) << 20;

bool mx_shape_ok(int64_t rows, int64_t cols) {
    return rows >= 0 && rows < kMaxTokens && cols >= kMxBlock && cols <= kMaxMxCols && cols % kMxBlock == 0 &&
           (rows + kTileM) * 4 * mx_sf_tiles(cols) < (int64_t(1) << 31);   // blocks of 32 elements
}
bool nv_shape_ok(int64_t rows, int64_t cols) {
    return rows >= 0 && rows < kMaxTokens && cols >= 64 && cols <= 8192 && cols % 64 == 0;
}

// Workspace of a dense product: the quantised rows of x.
struct LinearLayout {
    size_t codes, sf, g, total;
};
LinearLayout linear_layout(bool mx, int64_t T, int64_t K) {
    const size_t rows = static_cast<size_t>(nvfp4_rows_padded(T));
    LinearLayout L = {};
    if (linear_quantises_x(mx, T, K)) return L;   // x is quantised in shared memory
    L.codes = 0;
    L.sf = align_up(rows * (K / 2), 256);
    L.g = align_up(L.sf + (mx ? mxfp4_sf_bytes(T, K) : nvfp4_sf_bytes(T, K)), 256);
    L.total = mx ? L.g : align_up(L.g + rows * 4, 256);
    return L;
}

nvfp4_status linear_impl(bool mx, const fp4_linear_weights* w, const void* x, int x_type, int64_t T, int64_t ldx,
                         const float* bias, void* out, int out_type, int64_t ldo, void* ws, size_t ws_bytes,
                         cudaStream_t st) {
    if (!w) return NVFP4_ERR_INVALID_ARG;
    if (!(mx ? mx_shape_ok(T, w->K) : nv_shape_ok(T, w->K)) || w->N < 1 || w->N >= kMaxTokens || ldx < w->K ||
        ldo < w->N || !type_ok(x_type) || !type_ok(out_type) || (!mx && ldx % 8) || !rows_ok(T, ldx) || !rows_ok(T, ldo))
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (!w->codes || !w->sf || (!mx && !w->g) || !aligned(w->codes, 16) || !aligned(w->sf, 16) || !aligned(w->g, 4))
        return NVFP4_ERR_INVALID_ARG;
    if (T == 0) return NVFP4_OK;
    const LinearLayout L = linear_layout(mx, T, w->K);
    if (!x || !out || (!ws && L.total) || !aligned(x, mx ? type_size(x_type) : 16) || !aligned(out, type_size(out_type)) ||
        !aligned(bias, 4) || !aligned(ws, 256))
        return NVFP4_ERR_INVALID_ARG;
    if (ws_bytes < L.total) return NVFP4_ERR_WORKSPACE_TOO_SMALL;
    // one kernel reads x and stores outputs: a thread block's outputs must not be what another still reads
    const int64_t x_size = type_size(x_type), out_size = type_size(out_type);
    if (L.total == 0 && rows_overlap(x, ldx * x_size, w->K * x_size, out, ldo * out_size, w->N * out_size, T))
        return NVFP4_ERR_INVALID_ARG;
    int* err = device_error_ptr();
    if (!err) return NVFP4_ERR_CUDA;
    LinearArgs a{};
    a.mx = mx;
    a.T = T;
    a.N = static_cast<int>(w->N);
    a.K = static_cast<int>(w->K);
    a.a_codes = at<uint8_t>(ws, L.codes);
    a.a_sf = at<uint8_t>(ws, L.sf);
    a.a_g = mx ? nullptr : at<float>(ws, L.g);
    a.b_codes = static_cast<const uint8_t*>(w->codes);
    a.b_sf = static_cast<const uint8_t*>(w->sf);
    a.b_g = w->g;
    a.bias = bias;
    a.out = out;
    a.out_type = out_type;
    a.ldo = ldo;
    a.err = err;
    if (L.total == 0) return from_cuda(launch_linear_x({x, x_type, ldx}, a, st));
    const cudaError_t e =
        mx ? launch_mxfp4_quantize_rows(x, x_type, T, w->K, ldx, at<uint8_t>(ws, L.codes), at<uint8_t>(ws, L.sf), err, st)
           : launch_nvfp4_quantize_x(static_cast<const uint16_t*>(x), T, a.K, ldx, at<uint8_t>(ws, L.codes),
                                     at<uint8_t>(ws, L.sf), at<float>(ws, L.g), err, st);
    if (e != cudaSuccess) return from_cuda(e);
    return from_cuda(launch_linear(a, st, true));
}

}  // namespace

nvfp4_status moe_route_topk(const void* logits_dev, int type, int64_t T, int E, int64_t ld,
                            const moe_route_params* params, const float* bias_dev, int32_t* topk_ids_dev,
                            float* topk_w_dev, void* stream) {
    if (!params) return NVFP4_ERR_INVALID_ARG;
    const moe_route_params& p = *params;
    if (T < 0 || T >= kMaxTokens || E < 1 || E > 1024 || ld < E || !rows_ok(T, ld) || !type_ok(type) ||
        !route_params_ok(p, E) || p.n_group < 1 || p.n_group > 32 || E % p.n_group || p.topk_group < 1 ||
        p.topk_group > p.n_group || p.k > p.topk_group * (E / p.n_group) ||
        (p.group_score != MOE_GROUP_MAX && p.group_score != MOE_GROUP_TOP2))
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return NVFP4_OK;
    if (!logits_dev || !topk_ids_dev || !topk_w_dev || !aligned(logits_dev, type_size(type)) || !aligned(bias_dev, 4) ||
        !aligned(topk_ids_dev, 4) || !aligned(topk_w_dev, 4))
        return NVFP4_ERR_INVALID_ARG;
    int* err = device_error_ptr();
    if (!err) return NVFP4_ERR_CUDA;
    return from_cuda(launch_route_topk(logits_dev, type, T, E, ld, route_params(p), bias_dev, topk_ids_dev, topk_w_dev,
                                       err, static_cast<cudaStream_t>(stream)));
}

nvfp4_status moe_route_topk_backward(const void* logits_dev, int type, int64_t T, int E, int64_t ld,
                                     const moe_route_params* params, const int32_t* topk_ids_dev, const float* dw_dev,
                                     void* dlogits_dev, int64_t ld_out, void* stream) {
    if (!params) return NVFP4_ERR_INVALID_ARG;
    if (T < 0 || T >= kMaxTokens || E < 1 || E > 1024 || ld < E || ld_out < E || !rows_ok(T, ld) ||
        !rows_ok(T, ld_out) || !type_ok(type) || !route_params_ok(*params, E))
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return NVFP4_OK;
    if (!logits_dev || !topk_ids_dev || !dw_dev || !dlogits_dev || !aligned(logits_dev, type_size(type)) ||
        !aligned(dlogits_dev, type_size(type)) || !aligned(topk_ids_dev, 4) || !aligned(dw_dev, 4))
        return NVFP4_ERR_INVALID_ARG;
    // a row's zeros go out before its logits come in
    const int64_t size = type_size(type);
    if (rows_overlap(logits_dev, ld * size, E * size, dlogits_dev, ld_out * size, E * size, T)) return NVFP4_ERR_INVALID_ARG;
    int* err = device_error_ptr();
    if (!err) return NVFP4_ERR_CUDA;
    return from_cuda(launch_route_topk_backward(logits_dev, type, T, E, ld, route_params(*params), topk_ids_dev, dw_dev,
                                                dlogits_dev, ld_out, err, static_cast<cudaStream_t>(stream)));
}

// ---- balance loss of a router

namespace {

// What both calls refuse by shape; T == 0 has its outputs too.
bool balance_shape_ok(int type, int64_t T, int E, int64_t ld, int score, int k, const int32_t* offsets, int64_t S) {
    return T >= 0 && T < kMaxTokens && E >= 1 && E <= 1024 && ld >= E && rows_ok(T, ld) && type_ok(type) &&
           (score == MOE_SCORE_SOFTMAX || score == MOE_SCORE_SIGMOID) && k >= 1 && k <= 32 && k <= E && S >= 1 &&
           S < (int64_t(1) << 27) && (offsets || S == 1);
}

}  // namespace

size_t moe_balance_workspace_bytes(int64_t T, int E, int64_t S) {
    return T >= 0 && T < kMaxTokens && E >= 1 && E <= 1024 && S >= 1 && S < (int64_t(1) << 27) ? balance_workspace(T, E, S) : 0;
}

nvfp4_status moe_balance_loss(const void* logits_dev, int type, int64_t T, int E, int64_t ld, int score,
                              const int32_t* topk_ids_dev, int k, const uint8_t* mask_dev,
                              const int32_t* seq_offsets_dev, int64_t S, float* loss_dev, int32_t* counts_dev,
                              float* probs_dev, int32_t* tokens_dev, void* ws_dev, size_t ws_bytes, void* stream) {
    if (!balance_shape_ok(type, T, E, ld, score, k, seq_offsets_dev, S)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    const size_t need = balance_workspace(T, E, S);
    if ((need && !ws_dev) || !aligned(ws_dev, 256) || (T > 0 && (!logits_dev || !topk_ids_dev)) || !loss_dev || !counts_dev || !probs_dev || !tokens_dev ||
        !aligned(logits_dev, type_size(type)) || !aligned(topk_ids_dev, 4) || !aligned(seq_offsets_dev, 4) ||
        !aligned(loss_dev, 4) || !aligned(counts_dev, 4) || !aligned(probs_dev, 4) || !aligned(tokens_dev, 4))
        return NVFP4_ERR_INVALID_ARG;
    if (ws_bytes < need) return NVFP4_ERR_WORKSPACE_TOO_SMALL;
    int* err = device_error_ptr();
    if (!err) return NVFP4_ERR_CUDA;
    return from_cuda(launch_balance_loss(logits_dev, type, {T, E, ld, score, k, topk_ids_dev, mask_dev, seq_offsets_dev, S},
                                         loss_dev, counts_dev, probs_dev, tokens_dev, ws_dev, err,
                                         static_cast<cudaStream_t>(stream)));
}

nvfp4_status moe_balance_loss_backward(const void* logits_dev, int type, int64_t T, int E, int64_t ld, int score, int k,
                                       const uint8_t* mask_dev, const int32_t* seq_offsets_dev, int64_t S,
                                       const int32_t* counts_dev, const int32_t* tokens_dev, const float* dloss_dev,
                                       void* dlogits_dev, int64_t ld_out, int accumulate, void* stream) {
    if (!balance_shape_ok(type, T, E, ld, score, k, seq_offsets_dev, S) || ld_out < E || !rows_ok(T, ld_out) ||
        (accumulate != 0 && accumulate != 1))
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return NVFP4_OK;
    if (!logits_dev || !counts_dev || !tokens_dev || !dloss_dev || !dlogits_dev || !aligned(logits_dev, type_size(type)) ||
        !aligned(dlogits_dev, type_size(type)) || !aligned(seq_offsets_dev, 4) || !aligned(counts_dev, 4) ||
        !aligned(tokens_dev, 4) || !aligned(dloss_dev, 4))
        return NVFP4_ERR_INVALID_ARG;
    const int64_t size = type_size(type);
    if (rows_overlap(logits_dev, ld * size, E * size, dlogits_dev, ld_out * size, E * size, T)) return NVFP4_ERR_INVALID_ARG;
    int* err = device_error_ptr();
    if (!err) return NVFP4_ERR_CUDA;
    return from_cuda(launch_balance_loss_backward(logits_dev, type, {T, E, ld, score, k, nullptr, mask_dev, seq_offsets_dev, S},
                                                  counts_dev, tokens_dev, dloss_dev, dlogits_dev, ld_out, accumulate != 0, err,
                                                  static_cast<cudaStream_t>(stream)));
}

size_t mxfp4_sf_bytes(int64_t rows, int64_t cols) {
    if (!mx_shape_ok(rows, cols)) return 0;
    return static_cast<size_t>(nvfp4_rows_padded(rows) / kTileM) * mx_sf_tiles(cols) * kSfAtomBytes;
}

nvfp4_status mxfp4_quantize_rows(const void* x_dev, int type, int64_t rows, int64_t cols, int64_t ld, void* codes_dev,
                                 void* sf_dev, void* stream) {
    if (!mx_shape_ok(rows, cols) || ld < cols || !rows_ok(rows, ld) || !type_ok(type)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return NVFP4_OK;
    if (!x_dev || !codes_dev || !sf_dev || !aligned(x_dev, type_size(type)) || !aligned(codes_dev, 16) ||
        !aligned(sf_dev, 16))
        return NVFP4_ERR_INVALID_ARG;
    int* err = device_error_ptr();
    if (!err) return NVFP4_ERR_CUDA;
    return from_cuda(launch_mxfp4_quantize_rows(x_dev, type, rows, cols, ld, static_cast<uint8_t*>(codes_dev),
                                                static_cast<uint8_t*>(sf_dev), err,
                                                static_cast<cudaStream_t>(stream)));
}

nvfp4_status mxfp4_dequantize_rows(const void* codes_dev, const void* sf_dev, int64_t rows, int64_t cols, void* out_dev,
                                   int type, int64_t ld, void* stream) {
    if (!mx_shape_ok(rows, cols) || ld < cols || !rows_ok(rows, ld) ||
        (type != NVFP4_TYPE_F32 && type != NVFP4_TYPE_BF16))
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return NVFP4_OK;
    if (!codes_dev || !sf_dev || !out_dev || !aligned(codes_dev, 16) || !aligned(sf_dev, 16) ||
        !aligned(out_dev, type_size(type)))
        return NVFP4_ERR_INVALID_ARG;
    return from_cuda(launch_mxfp4_dequantize_rows(static_cast<const uint8_t*>(codes_dev),
                                                  static_cast<const uint8_t*>(sf_dev), rows, cols, out_dev, type, ld,
                                                  static_cast<cudaStream_t>(stream)));
}

size_t nvfp4_linear_workspace_bytes(int64_t T, int64_t K) {
    return nv_shape_ok(T, K) ? linear_layout(false, T, K).total : 0;
}
size_t mxfp4_linear_workspace_bytes(int64_t T, int64_t K) {
    return mx_shape_ok(T, K) ? linear_layout(true, T, K).total : 0;
}

nvfp4_status nvfp4_linear(const fp4_linear_weights* w, const void* x_dev, int64_t T, int64_t ldx, const float* bias_dev,
                          void* out_dev, int out_type, int64_t ldo, void* ws_dev, size_t ws_bytes, void* stream) {
    return linear_impl(false, w, x_dev, NVFP4_TYPE_BF16, T, ldx, bias_dev, out_dev, out_type, ldo, ws_dev, ws_bytes,
                       static_cast<cudaStream_t>(stream));
}
nvfp4_status mxfp4_linear(const fp4_linear_weights* w, const void* x_dev, int x_type, int64_t T, int64_t ldx,
                          const float* bias_dev, void* out_dev, int out_type, int64_t ldo, void* ws_dev,
                          size_t ws_bytes, void* stream) {
    return linear_impl(true, w, x_dev, x_type, T, ldx, bias_dev, out_dev, out_type, ldo, ws_dev, ws_bytes,
                       static_cast<cudaStream_t>(stream));
}

// ---- low-rank adapters

namespace {

// What both calls refuse of the adapters, first by shape, then by pointer.
bool adapters_shape_ok(const lora_adapters& a) {
    return (a.type == NVFP4_TYPE_BF16 || a.type == NVFP4_TYPE_F16) && a.L >= 1 && a.L <= 1024 && a.R >= 8 && a.R <= 128 &&
           a.R % 8 == 0 && a.K >= 8 && a.K <= (int64_t(1) << 20) && a.K % 8 == 0 && a.N >= 1 && a.N <= (int64_t(1) << 20);
}
bool adapters_ok(const lora_adapters& a) {
    return a.down && a.up && aligned(a.down, 16) && aligned(a.up, 16) && aligned(a.scale, 4);
}

}  // namespace

size_t lora_add_workspace_bytes(int64_t T, int L) {
    return T >= 0 && T < kMaxTokens && L >= 1 && L <= 1024 ? lora_workspace(T, L) : 0;
}
size_t lora_add_backward_workspace_bytes(int64_t T, int L, int R, int64_t K, int64_t N) {
    const lora_adapters a = {nullptr, nullptr, nullptr, NVFP4_TYPE_BF16, L, R, K, N};
    return T > 0 && T < kMaxTokens && adapters_shape_ok(a) ? lora_backward_workspace(T, L, R, K, N) : 0;
}

nvfp4_status lora_add(const lora_adapters* adapters, const void* x_dev, int64_t T, int64_t ldx,
                      const int32_t* adapter_ids_dev, const void* y_dev, int64_t ldy, void* out_dev, int64_t ldo,
                      int out_type, float* h_dev, void* ws_dev, size_t ws_bytes, void* stream) {
    if (!adapters) return NVFP4_ERR_INVALID_ARG;
    const lora_adapters& a = *adapters;
    if (!adapters_shape_ok(a) || T < 0 || T >= kMaxTokens || ldx < a.K || ldx % 8 || ldy < a.N || ldo < a.N || !type_ok(out_type) ||
        !rows_ok(T, ldx) || !rows_ok(T, ldy) || !rows_ok(T, ldo))
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (!adapters_ok(a)) return NVFP4_ERR_INVALID_ARG;
    if (T == 0) return NVFP4_OK;
    const size_t need = lora_workspace(T, a.L);
    const int64_t out_size = type_size(out_type);
    if (!x_dev || !adapter_ids_dev || !y_dev || !out_dev || (need && !ws_dev) || !aligned(x_dev, 16) ||
        !aligned(adapter_ids_dev, 4) || !aligned(y_dev, out_size) || !aligned(out_dev, out_size) || !aligned(h_dev, 16) ||
        !aligned(ws_dev, 256))
        return NVFP4_ERR_INVALID_ARG;
    if (ws_bytes < need) return NVFP4_ERR_WORKSPACE_TOO_SMALL;
    const bool in_place = y_dev == out_dev && ldy == ldo;
    if ((!in_place && rows_overlap(y_dev, ldy * out_size, a.N * out_size, out_dev, ldo * out_size, a.N * out_size, T)) ||
        rows_overlap(x_dev, ldx * 2, a.K * 2, out_dev, ldo * out_size, a.N * out_size, T))
        return NVFP4_ERR_INVALID_ARG;
    int* err = device_error_ptr();
    if (!err) return NVFP4_ERR_CUDA;
    return from_cuda(launch_lora_add({x_dev, T, ldx, a.type, a.down, a.up, a.scale, adapter_ids_dev, a.L, a.R, a.K, a.N, y_dev, ldy,
                                      out_dev, ldo, out_type, h_dev, ws_dev, err},
                                     static_cast<cudaStream_t>(stream)));
}

nvfp4_status lora_add_backward(const lora_adapters* adapters, const void* dy_dev, int64_t lddy, const void* x_dev,
                               int64_t ldx, const float* h_dev, const int32_t* adapter_ids_dev, int64_t T, void* dx_dev,
                               int64_t lddx, int dx_type, int accumulate, float* ddown_dev, float* dup_dev, void* ws_dev,
                               size_t ws_bytes, void* stream) {
    if (!adapters) return NVFP4_ERR_INVALID_ARG;
    const lora_adapters& a = *adapters;
    if (!adapters_shape_ok(a) || a.type != NVFP4_TYPE_BF16 || T < 0 || T >= kMaxTokens || lddy < a.N || ldx < a.K || ldx % 8 ||
        lddx < a.K || !type_ok(dx_type) || (accumulate != 0 && accumulate != 1) || !rows_ok(T, lddy) || !rows_ok(T, ldx) ||
        !rows_ok(T, lddx))
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (!adapters_ok(a) || !ddown_dev || !dup_dev || !aligned(ddown_dev, 4) || !aligned(dup_dev, 4)) return NVFP4_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        const size_t down = sizeof(float) * a.L * a.R * a.K, up = sizeof(float) * a.L * a.R * a.N;
        const nvfp4_status s = from_cuda(cudaMemsetAsync(ddown_dev, 0, down, st));
        return s != NVFP4_OK ? s : from_cuda(cudaMemsetAsync(dup_dev, 0, up, st));
    }
    const int64_t dx_size = type_size(dx_type);
    if (!dy_dev || !x_dev || !h_dev || !adapter_ids_dev || !dx_dev || !ws_dev || !aligned(dy_dev, 2) || !aligned(x_dev, 16) ||
        !aligned(h_dev, 16) || !aligned(adapter_ids_dev, 4) || !aligned(dx_dev, dx_size) || !aligned(ws_dev, 256))
        return NVFP4_ERR_INVALID_ARG;
    if (ws_bytes < lora_backward_workspace(T, a.L, a.R, a.K, a.N)) return NVFP4_ERR_WORKSPACE_TOO_SMALL;
    if (rows_overlap(dy_dev, lddy * 2, a.N * 2, dx_dev, lddx * dx_size, a.K * dx_size, T) ||
        rows_overlap(x_dev, ldx * 2, a.K * 2, dx_dev, lddx * dx_size, a.K * dx_size, T))
        return NVFP4_ERR_INVALID_ARG;
    int* err = device_error_ptr();
    if (!err) return NVFP4_ERR_CUDA;
    return from_cuda(launch_lora_add_backward({dy_dev, x_dev, T, lddy, ldx, h_dev, a.down, a.up, a.scale, adapter_ids_dev, a.L, a.R,
                                               a.K, a.N, dx_dev, lddx, dx_type, accumulate != 0, ddown_dev, dup_dev, ws_dev, err},
                                              st));
}

int nvfp4_last_cuda_error(void) { return static_cast<int>(t_last_cuda_error); }

const char* nvfp4_cuda_error_name(int error) { return cudaGetErrorName(static_cast<cudaError_t>(error)); }

nvfp4_status nvfp4_silu_table(float* out_dev, void* stream) {
    if (!out_dev || !aligned(out_dev, 4)) return NVFP4_ERR_INVALID_ARG;
    return from_cuda(copy_silu_table(out_dev, static_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_get_device_error(void* stream, int* device_status) {
    if (!device_status) return NVFP4_ERR_INVALID_ARG;
    *device_status = NVFP4_OK;
    if (from_cuda(cudaStreamSynchronize(static_cast<cudaStream_t>(stream))) != NVFP4_OK) return NVFP4_ERR_CUDA;
    int v = 0;
    if (from_cuda(cudaMemcpyFromSymbol(&v, g_device_error, sizeof(int))) != NVFP4_OK) return NVFP4_ERR_CUDA;
    if (v != 0) {
        const int zero = 0;
        if (from_cuda(cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int))) != NVFP4_OK) return NVFP4_ERR_CUDA;
    }
    *device_status = v;
    return NVFP4_OK;
}

}  // extern "C"
