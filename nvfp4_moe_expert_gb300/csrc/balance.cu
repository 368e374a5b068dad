// The router's balance loss (balance.cuh says what is computed).
//
// Two ways to the sums of p and the counts of each sequence.  Few tokens: one cluster of 8 or 16 CTAs to a sequence, which join
// their sums through shared memory: one launch, no workspace (128 x 128 5.5 us, 4096 x 128 BF16 14: a chain of latencies).  More: the rows in equal stretches to about three CTAs an SM,
// whatever sequences they hold; where a sequence ends in a stretch, or the stretch does, the CTA writes what it has of the
// sequence to slot (CTA + sequence) of the workspace, which no other pair shares, as each step of the walk moves one of
// the two on.  A second kernel adds a sequence's slots in their order.  No float atomics: the same bits for the same call.
// 65537 x 256 FP32, sigmoid, in 37 sequences take 22 + 6 us.  The rows' kernel is bound by instruction issue
// (72% of the slots, 257 warp instructions a row: an exponential, a quotient and a sum for each logit), 67 MB at 3.0 TB/s;
// the second one by its start and three trips to memory.
#include <atomic>

#include "balance.cuh"

namespace nvfp4 {
namespace balance {
namespace {

constexpr int kSplit = 8;                 // CTAs of a cluster; twice as many where there are few sequences

// What a CTA holds of a sequence: sums of p (a lane's elements of its rows), counts in shared memory, tokens.
template <int kPer>
struct Held {
    float sum[kPer];
    int tokens;
    __device__ void clear() {
#pragma unroll
        for (int i = 0; i < kPer; ++i) sum[i] = 0.0f;
        tokens = 0;
    }
};

template <typename T, int kPer, int kLanes, int kN>
__device__ __forceinline__ void add_rows(const T* __restrict__ logits, const BalanceParams& p, int64_t begin, int64_t end,
                                         int* s_count, Held<kPer>& held) {
    constexpr int kGroups = 32 / kLanes, kStep = kWarps * kGroups;
    const int lane = threadIdx.x & 31, sub = lane % kLanes, E = p.E;
    int64_t t = begin + threadIdx.x / kLanes;
    // the next row's logits and ids are on their way while a row is worked on
    float next[kPer];
    int next_id = -1;
    bool next_real;
    const auto fetch = [&](int64_t at) {
        next_real = at < end && (p.mask == nullptr || p.mask[at] != 0);
        if (next_real) {
            load_row<T, kPer, kLanes, kN>(logits + at * p.ld, E, sub, next);
            if (sub < p.k) next_id = p.ids[at * p.k + sub];
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) next[i] = 0.0f;     // adds nothing, and takes no warp out of its way
        }
    };
    const auto count = [&](int id) {
        if (static_cast<unsigned>(id) < static_cast<unsigned>(E)) atomicAdd(s_count + id, 1);
        else set_device_error(p.err, NVFP4_ERR_BAD_EXPERT_ID);
    };
    fetch(t);
    for (int64_t base = begin; base < end; base += kStep, t += kStep) {
        float v[kPer], none[1];
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = next[i];
        const int id = next_id;
        const bool real = next_real;
        if (base + kStep < end) fetch(t + kStep);
        bool bad;
        const float r = row_terms<kPer, kLanes, false>(p.score, v, none, bad), mine = real ? r : 0.0f;
        if (bad) set_device_error(p.err, NVFP4_ERR_NONFINITE);
#pragma unroll
        for (int i = 0; i < kPer; ++i) held.sum[i] = fmaf(v[i], mine, held.sum[i]);
        if (real) {
            held.tokens += sub == 0;
            if (sub < p.k) count(id);
            for (int j = sub + kLanes; j < p.k; j += kLanes) count(p.ids[t * p.k + j]);
        }
    }
}

// The lanes' sums joined: s_sum[e] (of [kWarps][E]) holds the CTA's.  Ends with the sums written, before a barrier.
template <int kPer, int kLanes, int kN>
__device__ __forceinline__ void join_rows(Held<kPer>& held, int E, float* s_sum, int* s_tokens) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o >= kLanes; o >>= 1) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) held.sum[i] += __shfl_xor_sync(kAll, held.sum[i], o);
    }
    if (lane < kLanes) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = expert_of<kLanes, kN>(i, lane);
            if (e < E) s_sum[warp * E + e] = held.sum[i];
        }
    }
    if (held.tokens) atomicAdd(s_tokens, held.tokens);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) {
        float sum = s_sum[e];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) sum += s_sum[w * E + e];
        s_sum[e] = sum;
    }
}

struct Outputs {
    float* loss;
    int32_t* counts;
    float* probs;
    int32_t* tokens;
};

__device__ __forceinline__ float loss_of(float sum, int n, int E, int k) {
    return n > 0 ? sum * (static_cast<float>(E) / (static_cast<float>(k) * static_cast<float>(n))) : 0.0f;
}

// ------------------------------------------------------------------ few tokens: a cluster to a sequence
template <typename T, int kPer, int kLanes, int kN>
__global__ void __launch_bounds__(kThreads) sequence_kernel(const T* __restrict__ logits, const BalanceParams p, const Outputs out) {
    extern __shared__ float s_sum[];                        // [kWarps][E], then [E] counts
    __shared__ int s_tokens;
    __shared__ float s_loss, s_part[kWarps];
    const int E = p.E, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int* s_count = reinterpret_cast<int*>(s_sum + kWarps * E);
    const int rank = static_cast<int>(cluster_rank()), split = static_cast<int>(cluster_size());
    const int64_t s = blockIdx.x / split;
    int64_t begin, end;
    sequence_rows(p.offsets, s, p.T, begin, end);
    const int64_t share = (end - begin + split - 1) / split;
    begin = min(begin + rank * share, end);
    end = min(begin + share, end);
    for (int e = threadIdx.x; e < E; e += kThreads) s_count[e] = 0;
    if (threadIdx.x == 0) s_tokens = 0;
    __syncthreads();
    Held<kPer> held;
    held.clear();
    add_rows<T, kPer, kLanes, kN>(logits, p, begin, end, s_count, held);
    join_rows<kPer, kLanes, kN>(held, E, s_sum, &s_tokens);
    cluster_barrier();

    int n = 0;
#pragma unroll 8
    for (int c = 0; c < split; ++c) n += cluster_load_s32(cluster_addr(&s_tokens, c));
    const int part = (E + split - 1) / split;             // at most 128
    const int e = rank * part + static_cast<int>(threadIdx.x);
    float term = 0.0f;
    if (static_cast<int>(threadIdx.x) < part && e < E) {
        int count = 0;
        float sum = 0.0f;
#pragma unroll 8
        for (int c = 0; c < split; ++c) {
            count += cluster_load_s32(cluster_addr(s_count + e, c));
            sum += cluster_load_f32(cluster_addr(s_sum + e, c));
        }
        const float mean = n > 0 ? sum / static_cast<float>(n) : 0.0f;
        out.counts[s * E + e] = count;
        out.probs[s * E + e] = mean;
        term = static_cast<float>(count) * mean;
    }
    term = lanes_sum<32>(term);
    if (lane == 0) s_part[warp] = term;
    __syncthreads();
    if (threadIdx.x == 0) {
        s_loss = 0.0f;
        for (int w = 0; w < kWarps; ++w) s_loss += s_part[w];
    }
    cluster_barrier();
    if (rank == 0 && threadIdx.x == 0) {
        float sum = 0.0f;
        for (int c = 0; c < split; ++c) sum += cluster_load_f32(cluster_addr(&s_loss, c));
        out.loss[s] = loss_of(sum, n, E, p.k);
        out.tokens[s] = n;
    }
    cluster_barrier();                                      // no CTA leaves while another reads its shared memory
}

// Launches a kernel in clusters of `split` CTAs; wide: the devices on which it may ask for more than 8.
template <typename... P, typename... A>
cudaError_t launch_clusters(void (*kernel)(P...), unsigned split, int64_t clusters, int threads, size_t smem, cudaStream_t st,
                            std::atomic<uint64_t>& wide, A... args) {
    if (split > 8) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        if (!(wide.load() >> dev & 1)) {
            e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            wide.fetch_or(uint64_t(1) << dev);
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * split));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ------------------------------------------------------------------ more: stretches of rows, then the slots
struct Slots {
    float* sums;          // [slots][E]
    int32_t* counts;      // [slots][E]
    int32_t* tokens;      // [slots]
    int64_t rows;         // of a stretch
};

template <typename T, int kPer, int kLanes, int kN>
__global__ void __launch_bounds__(kThreads, kPer <= 16 ? 3 : 2) stretch_kernel(const T* __restrict__ logits, const BalanceParams p, const Slots w) {
    extern __shared__ float s_sum[];                        // [kWarps][E], then [E] counts
    __shared__ int s_tokens;
    const int E = p.E;
    int* s_count = reinterpret_cast<int*>(s_sum + kWarps * E);
    const int64_t cta = blockIdx.x, end = min((cta + 1) * w.rows, p.T);
    int64_t row = cta * w.rows, s = find_sequence(p.offsets, p.S, row);
    if (s < 0) {                                            // in front of the first
        s = 0;
        row = max(row, static_cast<int64_t>(p.offsets[0]));
    }
    while (row < end && s < p.S) {
        const int64_t stop = p.offsets == nullptr ? end : min(end, static_cast<int64_t>(p.offsets[s + 1]));
        if (stop <= row) {                                  // empty, as any number behind it may be
            s = max(s + 1, find_sequence(p.offsets, p.S, row));
            continue;
        }
        for (int e = threadIdx.x; e < E; e += kThreads) s_count[e] = 0;
        if (threadIdx.x == 0) s_tokens = 0;
        __syncthreads();
        Held<kPer> held;
        held.clear();
        add_rows<T, kPer, kLanes, kN>(logits, p, row, stop, s_count, held);
        join_rows<kPer, kLanes, kN>(held, E, s_sum, &s_tokens);
        const int64_t at = cta + s;
        for (int e = threadIdx.x; e < E; e += kThreads) {   // the experts this thread joined
            w.sums[at * E + e] = s_sum[e];
            w.counts[at * E + e] = s_count[e];
        }
        if (threadIdx.x == 0) w.tokens[at] = s_tokens;
        __syncthreads();
        row = stop;
        ++s;
    }
    pdl_launch_dependents();              // not earlier: the join's CTAs would take this kernel's room
}

constexpr int kJoinThreads = 512;

// A sequence to a cluster (of 1 to 8 CTAs, a part of the experts each): an expert to a thread, the threads that are left
// over take every second, fourth, ... slot.
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const BalanceParams p, const Slots w, const Outputs out) {
    __shared__ float s_sum[kJoinThreads], s_loss[kJoinThreads / 32];
    __shared__ int s_count[kJoinThreads], s_tokens;
    const int E = p.E, thread = threadIdx.x;
    const int rank = static_cast<int>(cluster_rank()), parts = static_cast<int>(cluster_size());
    const int64_t s = blockIdx.x / parts;
    int64_t begin, end;
    sequence_rows(p.offsets, s, p.T, begin, end);
    const int64_t first = begin / w.rows + s, last = end > begin ? (end - 1) / w.rows + s : first - 1;
    const int part = (E + parts - 1) / parts, e0 = rank * part, e1 = min(e0 + part, E);
    int wide = 32;                        // experts at a time, a power of two
    while (wide < part && wide < kJoinThreads) wide *= 2;
    const int apart = kJoinThreads / wide, turn = thread / wide, mine = thread & (wide - 1);
    if (thread == 0) s_tokens = 0;
    __syncthreads();
    pdl_wait();
    int tokens = 0;
    for (int64_t at = first + thread; at <= last; at += kJoinThreads) tokens += w.tokens[at];
    if (tokens) atomicAdd(&s_tokens, tokens);
    float loss = 0.0f;
    for (int base = e0; base < e1; base += wide) {
        const int e = base + mine;
        float sum = 0.0f;
        int count = 0;
        if (e < e1) {
#pragma unroll 8
            for (int64_t at = first + turn; at <= last; at += apart) {
                sum += w.sums[at * E + e];
                count += w.counts[at * E + e];
            }
        }
        s_sum[thread] = sum;
        s_count[thread] = count;
        __syncthreads();
        if (turn == 0) {
            for (int i = 1; i < apart; ++i) {
                sum += s_sum[i * wide + mine];
                count += s_count[i * wide + mine];
            }
            const int n = s_tokens;
            const float mean = n > 0 ? sum / static_cast<float>(n) : 0.0f;
            if (e < e1) {
                out.counts[s * E + e] = count;
                out.probs[s * E + e] = mean;
            }
            loss += static_cast<float>(count) * mean;
        }
        __syncthreads();
    }
    loss = lanes_sum<32>(loss);
    if ((thread & 31) == 0) s_loss[thread >> 5] = loss;
    cluster_barrier();
    if (rank == 0 && thread == 0) {
        float sum = 0.0f;
        for (int c = 0; c < parts; ++c) {
            float own = 0.0f;
            for (int i = 0; i < wide / 32; ++i) own += cluster_load_f32(cluster_addr(s_loss + i, c));   // warps of turn 0
            sum += own;
        }
        out.loss[s] = loss_of(sum, s_tokens, E, p.k);
        out.tokens[s] = s_tokens;
    }
    cluster_barrier();
}

// Whether a cluster to a sequence takes no longer than two kernels, with the second launch and the workspace, which take the host
// about 8 us.  us on the device from the first kernel's start, E = 128, BF16, a cluster and two kernels:
//     tokens        512          1024          2048          4096          8192
//     1 sequence    5.9 * 13     7.4 * 13      9.4 * 13      14 * 14       27 13 *
//     4             6.3 * 9.4    6.3 * 9.4     6.5 * 9.6     8.0 * 10      14 11 *
//     32            6.2 * 12     6.0 * 10      6.2 * 10      6.2 * 10      6.5 9.6 *
// and 1 sequence with E = 256 7.5 * 8.7, 10 * 9.3, 15 * 10, 23 13 * (a call of 4096 x 128 20 us instead of 26; behind queued work or
// in a graph, where the host's part does not count, two kernels would be sooner where their figure above is the lower one).  The host does
// not know the lengths: they are taken to be even.  More than 32 clusters wait for each other (64: 11 us, two kernels 9).
bool few(int64_t T, int E, int64_t S) { return S <= 32 && T * (E > 128 ? E : 128) <= int64_t(1) << 19; }
// CTAs of such a cluster: 16 where there are few sequences and more than 512 rows of 128 experts (4096 x 128 14 us with 16, 22 with 8;
// 128 x 128 a microsecond more with 16).
unsigned split_of(int64_t T, int E, int64_t S) { return S < 8 && T * (E > 128 ? E : 128) > int64_t(1) << 16 ? 2 * kSplit : kSplit; }
int rows_at_once(int E) { return E <= 128 ? 32 : E <= 256 ? 16 : 8; }   // of a CTA
// Stretches: three to an SM, of whole turns of a CTA.
int64_t stretch_rows(int64_t T, int E) {
    constexpr int64_t kStretches = 3 * 152;
    const int64_t at_once = rows_at_once(E), turns = (T + at_once * kStretches - 1) / (at_once * kStretches);
    return at_once * (turns < 1 ? 1 : turns);
}
int64_t stretches(int64_t T, int E) { return T == 0 ? 0 : (T + stretch_rows(T, E) - 1) / stretch_rows(T, E); }
size_t align_256(size_t n) { return (n + 255) / 256 * 256; }

Slots slots(void* ws, int64_t T, int E, int64_t S) {
    const size_t n = static_cast<size_t>(stretches(T, E) + S), each = align_256(n * E * 4);
    uint8_t* b = static_cast<uint8_t*>(ws);
    return {reinterpret_cast<float*>(b), reinterpret_cast<int32_t*>(b + each), reinterpret_cast<int32_t*>(b + 2 * each),
            stretch_rows(T, E)};
}

template <typename T>
cudaError_t forward(const void* logits, const BalanceParams& p, const Outputs& out, void* ws, cudaStream_t st) {
    const size_t smem = static_cast<size_t>(p.E) * (kWarps + 1) * sizeof(float);
    const T* l = static_cast<const T*>(logits);
    return by_experts(p.E, [&](auto per, auto lanes) {
        return by_width<T>(load_width<T>(logits, p.ld, p.E), [&](auto width) {
            constexpr int kPer = decltype(per)::value, kLanes = decltype(lanes)::value, kN = decltype(width)::value;
            if (few(p.T, p.E, p.S)) {
                static std::atomic<uint64_t> wide{0};
                return launch_clusters(sequence_kernel<T, kPer, kLanes, kN>, split_of(p.T, p.E, p.S), p.S, kThreads, smem, st,
                                       wide, l, p, out);
            }
            const Slots w = slots(ws, p.T, p.E, p.S);
            return launch_pdl(false, stretch_kernel<T, kPer, kLanes, kN>, dim3(static_cast<unsigned>(stretches(p.T, p.E))),
                              dim3(kThreads), smem, st, l, p, w);
        });
    });
}

}  // namespace
}  // namespace balance

size_t balance_workspace(int64_t T, int E, int64_t S) {
    using namespace balance;
    if (few(T, E, S)) return 0;
    const size_t n = static_cast<size_t>(stretches(T, E) + S);
    return 2 * align_256(n * E * 4) + align_256(n * 4);
}

cudaError_t launch_balance_loss(const void* logits, int type, const BalanceArgs& a, float* loss, int32_t* counts, float* probs,
                                int32_t* tokens, void* ws, int* err, cudaStream_t st) {
    using namespace balance;
    const BalanceParams p = {a.T, a.E, a.ld, a.score, a.k, a.ids, a.mask, a.offsets, a.S, err};
    const Outputs out = {loss, counts, probs, tokens};
    const bool two = !few(a.T, a.E, a.S), rows = !two || a.T > 0;
    if (rows) {
        const cudaError_t e = type == NVFP4_TYPE_F32    ? forward<float>(logits, p, out, ws, st)
                              : type == NVFP4_TYPE_BF16 ? forward<__nv_bfloat16>(logits, p, out, ws, st)
                                                        : forward<__half>(logits, p, out, ws, st);
        if (e != cudaSuccess || !two) return e;
    }
    // CTAs to a sequence: as many as an SM each allows.  One sequence has up to 456 slots, which 8 CTAs read sooner; with 8 for each
    // of 64 sequences the call took 16 us, with one 9
    unsigned parts = kSplit;
    while (parts > 1 && a.S * parts > 152) parts /= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.S * parts));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = parts;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = rows ? 2 : 1;          // behind the rows' kernel
    return cudaLaunchKernelEx(&cfg, join_kernel, p, slots(ws, a.T, a.E, a.S), out);
}

}  // namespace nvfp4
