// C ABI of the operators around a fine-tuning step's dense layers
// (include/lora_step.h, lora_embedding.h, lora_qk_rope.h, lora_distill.h):
// argument checks, workspace layout and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <mutex>
#include <vector>

#include "lora_distill.h"
#include "lora_embedding.h"
#include "lora_qk_rope.h"
#include "distill.cuh"
#include "embedding.cuh"
#include "qk_rope.cuh"

using namespace lmlp::step;

namespace {

#define STEP_TRY(expr)                       \
    do {                                     \
        const int rc_ = (expr);              \
        if (rc_ != LORA_MLP_OK) return rc_;  \
    } while (0)

constexpr int kMaxDevices = 64;
constexpr size_t kAlign = 256;

__device__ int g_step_status;

std::atomic<int64_t> g_launches{0};

constexpr long long kWaitLimitCycles = 4000000000LL;  // about 2 s
std::atomic<long long> g_wait_limit{kWaitLimitCycles};
std::atomic<int> g_force_timeout{0};

// ----------------------------------------------------------------------------- device info
struct DevInfo {
    bool checked, ok;
    int sms;
    int* status;
};
DevInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

int device_info(DevInfo* out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return LORA_MLP_ERR_CUDA;
    std::lock_guard<std::mutex> lk(g_dev_mu);
    DevInfo& di = g_dev[dev];
    if (!di.checked) {
        int major = 0, minor = 0, sms = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return LORA_MLP_ERR_CUDA;
        di.ok = major == 10 && minor == 0;
        di.sms = sms;
        void* addr = nullptr;
        if (di.ok && cudaGetSymbolAddress(&addr, g_step_status) != cudaSuccess) return LORA_MLP_ERR_CUDA;
        di.status = static_cast<int*>(addr);
        di.checked = true;
    }
    *out = di;
    return di.ok ? LORA_MLP_OK : LORA_MLP_ERR_UNSUPPORTED_ARCH;
}

// ----------------------------------------------------------------------------- argument checks
struct Arg {
    const void* p;
    size_t align;
};

// Null pointers, then alignment (both found without CUDA).
int check_args(std::initializer_list<Arg> as) {
    for (const Arg& a : as)
        if (a.p == nullptr) return LORA_MLP_ERR_INVALID_ARG;
    for (const Arg& a : as)
        if (reinterpret_cast<uintptr_t>(a.p) % a.align) return LORA_MLP_ERR_MISALIGNED;
    return LORA_MLP_OK;
}

// Pointers that may be null.
int check_optional(std::initializer_list<Arg> as) {
    for (const Arg& a : as)
        if (reinterpret_cast<uintptr_t>(a.p) % a.align) return LORA_MLP_ERR_MISALIGNED;
    return LORA_MLP_OK;
}

// Memory of the current device (after every other check of the arguments).
int check_memory(std::initializer_list<Arg> as) {
    for (const Arg& a : as)
        if (a.p != nullptr) STEP_TRY(lora_mlp_check_pointer(a.p, 1));
    return LORA_MLP_OK;
}

// ----------------------------------------------------------------------------- timing
struct TimingRec {
    const char* name;
    cudaEvent_t beg, end;
};
std::mutex g_time_mu;
std::atomic<int> g_timing{0};
std::vector<TimingRec> g_recs;

struct LaunchScope {
    TimingRec rec;
    cudaStream_t st;
    LaunchScope(const char* n, cudaStream_t s) : rec{n, nullptr, nullptr}, st(s) {
        g_launches.fetch_add(1, std::memory_order_relaxed);
        if (!g_timing.load(std::memory_order_relaxed)) return;
        if (cudaEventCreate(&rec.beg) != cudaSuccess || cudaEventCreate(&rec.end) != cudaSuccess) {
            cudaGetLastError();
            drop();
            return;
        }
        cudaEventRecord(rec.beg, st);
    }
    ~LaunchScope() {
        if (rec.end == nullptr) return;
        cudaEventRecord(rec.end, st);
        try {
            std::lock_guard<std::mutex> lk(g_time_mu);
            g_recs.push_back(rec);
        } catch (...) {  // no memory for the record: the launch stands, its time is lost
            drop();
        }
    }
    void drop() {
        if (rec.beg != nullptr) cudaEventDestroy(rec.beg);
        if (rec.end != nullptr) cudaEventDestroy(rec.end);
        rec.beg = rec.end = nullptr;
    }
};

// One launch.  `after_own`: the kernel before it in the stream is one of this
// call's, which lets it start early and which it waits for itself
// (programmatic dependent launch).  `cluster`: blocks of a thread-block cluster.
template <class... P, class... A>
int launch(const char* name, void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
           bool after_own, int cluster, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2] = {};
    cfg.attrs = attr;
    if (after_own) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs++].val.clusterDim = {static_cast<unsigned>(cluster), 1u, 1u};
    }
    LaunchScope scope(name, st);
    if (cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) != cudaSuccess) {
        cudaGetLastError();
        return LORA_MLP_ERR_CUDA;
    }
    return LORA_MLP_OK;
}

// Raises a kernel's dynamic shared memory limit.
template <class K>
int allow_smem(K* kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) ==
                   cudaSuccess
               ? LORA_MLP_OK
               : LORA_MLP_ERR_CUDA;
}

// Clusters of a kernel that the current device holds at once.  CUDA takes
// several microseconds to say; the last few answers are kept.
struct Residency {
    int dev;
    const void* kernel;
    int threads, cluster;
    size_t smem;
    int count;
};
constexpr int kResidencies = 16;
Residency g_residency[kResidencies];
int g_residency_next = 0;
std::mutex g_residency_mu;

template <class... P>
int resident_clusters(void (*kernel)(P...), size_t max_smem, int threads, size_t smem, int cluster, int* count) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return LORA_MLP_ERR_CUDA;
    const void* key = reinterpret_cast<const void*>(kernel);
    std::lock_guard<std::mutex> lk(g_residency_mu);
    for (const Residency& r : g_residency)
        if (r.kernel == key && r.dev == dev && r.threads == threads && r.cluster == cluster && r.smem == smem) {
            *count = r.count;
            return LORA_MLP_OK;
        }
    STEP_TRY(allow_smem(kernel, max_smem));
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {static_cast<unsigned>(cluster), 1u, 1u};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(cluster));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(count, kernel, &cfg) != cudaSuccess || *count < 1) {
        cudaGetLastError();
        return LORA_MLP_ERR_CUDA;
    }
    g_residency[g_residency_next] = {dev, key, threads, cluster, smem, *count};
    g_residency_next = (g_residency_next + 1) % kResidencies;
    return LORA_MLP_OK;
}

struct Carver {
    size_t off = 0;
    size_t take(size_t bytes) {
        const size_t at = off;
        off += (bytes + kAlign - 1) / kAlign * kAlign;
        return at;
    }
};

int ceil_log2(uint64_t x) {
    int b = 0;
    while ((uint64_t{1} << b) < x) ++b;
    return b;
}

}  // namespace

extern "C" {

int lora_step_device_status(void* stream, int* status) {
    if (status == nullptr) return LORA_MLP_ERR_INVALID_ARG;
    DevInfo di;
    STEP_TRY(device_info(&di));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int v = 0;
    const int zero = 0;
    if (cudaMemcpyAsync(&v, di.status, sizeof(int), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaMemcpyAsync(di.status, &zero, sizeof(int), cudaMemcpyHostToDevice, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return LORA_MLP_ERR_CUDA;
    *status = v;
    return LORA_MLP_OK;
}

int lora_step_timing_enable(int enable) {
    g_timing.store(enable ? 1 : 0);
    return LORA_MLP_OK;
}

int lora_step_timing_collect(lora_mlp_kernel_time* out, int max, int* count) {
    std::lock_guard<std::mutex> lk(g_time_mu);
    int n = 0, rc = LORA_MLP_OK;
    for (const TimingRec& rec : g_recs) {
        float ms = 0.0f;
        if (cudaEventSynchronize(rec.end) != cudaSuccess || cudaEventElapsedTime(&ms, rec.beg, rec.end) != cudaSuccess)
            rc = LORA_MLP_ERR_CUDA;
        if (out != nullptr && n < max) out[n] = {rec.name, ms};
        ++n;
        cudaEventDestroy(rec.beg);
        cudaEventDestroy(rec.end);
    }
    g_recs.clear();
    if (count) *count = n;
    return rc;
}

int64_t lora_step_launch_count(void) { return g_launches.load(); }

int lora_step_debug_force_timeout(int enable, int64_t wait_cycles) {
    if (enable && wait_cycles < 1) return LORA_MLP_ERR_INVALID_ARG;
    g_wait_limit.store(enable ? static_cast<long long>(wait_cycles) : kWaitLimitCycles);
    g_force_timeout.store(enable ? 1 : 0);
    return LORA_MLP_OK;
}

}  // extern "C"

// ============================================================================= embedding

namespace {

constexpr int64_t kEmbMaxN = int64_t{1} << 30;

int validate_embedding(int64_t N, int64_t V, int64_t d) {
    if (N < 1 || V < 1 || d < 1) return LORA_MLP_ERR_INVALID_ARG;
    if (d % 8 || N > kEmbMaxN || d > kEmbMaxN || V > INT32_MAX - 1) return LORA_MLP_ERR_UNSUPPORTED_SHAPE;
    return LORA_MLP_OK;
}

struct EmbPlan {
    int nv, slices, log_worker, log_group, nchunks, bits, passes, ntiles, tile;
    bool small;
    size_t key[2], val[2], hist, counters, part, total;
};

EmbPlan make_emb_plan(int64_t N, int64_t V, int64_t d) {
    EmbPlan p{};
    p.nv = static_cast<int>(d / 8);
    p.log_worker = std::max(5, ceil_log2(static_cast<uint64_t>(std::min((p.nv + 1) / 2, kEmbThreads))));
    p.nchunks = static_cast<int>(N / kEmbChunk);
    // Narrow slices, for many groups a block and few tokens a share, unless
    // there are so many chunks that most of their blocks find nothing to do.
    p.log_group = 5;
    while (p.log_group < p.log_worker && int64_t{p.nchunks} * (p.nv >> (p.log_group + 1)) > 1024) ++p.log_group;
    p.slices = (p.nv + (2 << p.log_group) - 1) >> (p.log_group + 1);
    const int key_bits = std::max(1, ceil_log2(static_cast<uint64_t>(V) + 1));  // keys 0 .. V
    p.passes = (key_bits + kSortMaxBits - 1) / kSortMaxBits;
    p.bits = (key_bits + p.passes - 1) / p.passes;
    p.small = N <= kSortSmall;
    // a tile a multiprocessor as far as that goes; four times as wide beyond,
    // as every tile reads every tile's counts
    p.tile = kSortThreads * (N <= int64_t{128} * kSortThreads ? 1 : 4);
    p.ntiles = static_cast<int>((N + p.tile - 1) / p.tile);
    Carver c;
    for (int i = 0; i < 2; ++i) {
        p.key[i] = c.take(static_cast<size_t>(N) * 4);
        p.val[i] = c.take(static_cast<size_t>(N) * 4);
    }
    p.hist = c.take(p.small ? 0 : static_cast<size_t>(p.passes) * p.ntiles * (size_t{4} << p.bits));
    p.counters = c.take(static_cast<size_t>(p.nchunks) * p.slices * 4);
    p.part = c.take(static_cast<size_t>(p.nchunks) * static_cast<size_t>(d) * 4);
    p.total = c.off;
    return p;
}

}  // namespace

extern "C" {

int lora_embedding_forward(int64_t N, int64_t V, int64_t d, float scale, const int64_t* ids, const void* E,
                           void* out, void* stream) {
    STEP_TRY(validate_embedding(N, V, d));
    if (!std::isfinite(scale)) return LORA_MLP_ERR_INVALID_ARG;
    STEP_TRY(check_args({{ids, 8}, {E, 16}, {out, 16}}));
    STEP_TRY(check_memory({{ids, 8}, {E, 16}, {out, 16}}));
    DevInfo di;
    STEP_TRY(device_info(&di));
    EmbFwdArgs a{};
    a.ids = reinterpret_cast<const long long*>(ids);
    a.E = static_cast<const __nv_bfloat16*>(E);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.N = N;
    a.V = V;
    a.nv = static_cast<int>(d / 8);
    // Few tokens: a thread for each vector of a row.  Many: kEmbLoads vectors a
    // thread, so that enough bytes are on their way.
    const bool many = N * a.nv >= int64_t{kEmbLoads} * kEmbThreads * 8 * di.sms;
    const int per = many ? kEmbLoads : 1;
    a.log_tpr = ceil_log2(static_cast<uint64_t>(std::min((a.nv + per - 1) / per, kEmbThreads)));
    a.scale = scale;
    a.status = di.status;
    const int rows = kEmbThreads >> a.log_tpr;
    return launch("EMB_fwd", embed_fwd_kernel, dim3(static_cast<unsigned>((N + rows - 1) / rows)), kEmbThreads, 0,
                  static_cast<cudaStream_t>(stream), false, 1, a);
}

int lora_embedding_sizes(int64_t N, int64_t V, int64_t d, size_t* workspace_bytes) {
    STEP_TRY(validate_embedding(N, V, d));
    if (workspace_bytes) *workspace_bytes = make_emb_plan(N, V, d).total;
    return LORA_MLP_OK;
}

int lora_embedding_backward(int64_t N, int64_t V, int64_t d, float scale, int64_t padding_idx, int grad_type,
                            const int64_t* ids, const void* dOut, void* dE, void* workspace,
                            size_t workspace_bytes, void* stream) {
    STEP_TRY(validate_embedding(N, V, d));
    if (!std::isfinite(scale)) return LORA_MLP_ERR_INVALID_ARG;
    if (grad_type != LORA_EMBEDDING_GRAD_BF16 && grad_type != LORA_EMBEDDING_GRAD_FP32) return LORA_MLP_ERR_INVALID_ARG;
    STEP_TRY(check_args({{ids, 8}, {dOut, 16}, {dE, 16}, {workspace, 16}}));
    const EmbPlan p = make_emb_plan(N, V, d);
    const bool f32 = grad_type == LORA_EMBEDDING_GRAD_FP32;
    const int64_t zeros = V * d / 8 * (f32 ? 2 : 1), zero_blocks = (zeros + kZeroBlock - 1) / kZeroBlock;
    const int64_t workers = kEmbThreads >> p.log_worker;
    const int64_t blocks = (N + workers - 1) / workers + static_cast<int64_t>(p.nchunks) * p.slices;
    if (zero_blocks > INT32_MAX || blocks > INT32_MAX) return LORA_MLP_ERR_UNSUPPORTED_SHAPE;
    if (workspace_bytes < p.total) return LORA_MLP_ERR_WORKSPACE_TOO_SMALL;
    STEP_TRY(check_memory({{ids, 8}, {dOut, 16}, {dE, 16}, {workspace, 16}}));
    DevInfo di;
    STEP_TRY(device_info(&di));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);

    SortArgs s{};
    s.ids = reinterpret_cast<const long long*>(ids);
    s.N = static_cast<int>(N);
    s.V = static_cast<int>(V);
    s.padding = padding_idx;
    s.bits = p.bits;
    s.passes = p.passes;
    s.ntiles = p.ntiles;
    s.tile = p.tile;
    for (int i = 0; i < 2; ++i) {
        s.key[i] = reinterpret_cast<uint32_t*>(ws + p.key[i]);
        s.val[i] = reinterpret_cast<uint32_t*>(ws + p.val[i]);
    }
    s.hist = reinterpret_cast<uint32_t*>(ws + p.hist);
    s.counters = reinterpret_cast<uint32_t*>(ws + p.counters);
    s.ncounters = p.nchunks * p.slices;
    s.status = di.status;
    if (p.small) {
        const int items = N <= kSortThreads ? 1 : N <= 2 * kSortThreads ? 2 : N <= 4 * kSortThreads ? 4 : 8;
        auto kernel = items == 1   ? embed_sort_small_kernel<1>
                      : items == 2 ? embed_sort_small_kernel<2>
                      : items == 4 ? embed_sort_small_kernel<4>
                                   : embed_sort_small_kernel<8>;
        const size_t smem = sizeof(SortShared) + 2 * sizeof(uint32_t) * kSortThreads * items;
        STEP_TRY(allow_smem(kernel, smem));
        STEP_TRY(launch("EMB_sort", kernel, dim3(1), kSortThreads, smem, st, false, 1, s));
    } else {
        const dim3 grid(static_cast<unsigned>(p.ntiles));
        STEP_TRY(launch("EMB_sort_count", embed_sort_count_kernel, grid, kSortThreads, 0, st, false, 1, s));
        for (int i = 0; i < p.passes; ++i)
            STEP_TRY(launch("EMB_sort_scatter",
                            p.tile == kSortThreads ? embed_sort_scatter_kernel<1> : embed_sort_scatter_kernel<4>, grid,
                            kSortThreads, sizeof(SortShared), st, true, 1, s, i));
    }

    EmbBwdArgs a{};
    a.key = s.key[p.passes & 1];
    a.val = s.val[p.passes & 1];
    a.dOut = static_cast<const __nv_bfloat16*>(dOut);
    a.dE = dE;
    a.part = reinterpret_cast<float*>(ws + p.part);
    a.counters = s.counters;
    a.N = s.N;
    a.V = s.V;
    a.nv = p.nv;
    a.slices = p.slices;
    a.log_group = p.log_group;
    a.log_worker = p.log_worker;
    a.scale = scale;
    const dim3 grid(static_cast<unsigned>(blocks));
    STEP_TRY(launch("EMB_zero", embed_zero_kernel, dim3(static_cast<unsigned>(zero_blocks)),
                    kZeroThreads, 0, st, true, 1, static_cast<uint4*>(dE), static_cast<long long>(zeros)));
    if (f32) return launch("EMB_grad", embed_bwd_kernel<true>, grid, kEmbThreads, 0, st, true, 1, a);
    return launch("EMB_grad", embed_bwd_kernel<false>, grid, kEmbThreads, 0, st, true, 1, a);
}

}  // extern "C"

// ============================================================================= queries' and keys' norm and rotation

namespace {

int validate_qk(const lora_qk_shape* sh) {
    if (sh == nullptr) return LORA_MLP_ERR_INVALID_ARG;
    if (sh->B < 1 || sh->S < 1 || sh->Hq < 1 || sh->Hk < 1 || sh->P < 1 || sh->rot < 1 || sh->rot > sh->D ||
        sh->position_stride < 0)
        return LORA_MLP_ERR_INVALID_ARG;
    if (!std::isfinite(sh->eps) || sh->eps < 0.0f) return LORA_MLP_ERR_INVALID_ARG;
    if (sh->D % 16 || sh->rot % 16 || sh->D > 512) return LORA_MLP_ERR_UNSUPPORTED_SHAPE;
    const int64_t lim = INT32_MAX;
    if (sh->B > lim || sh->S > lim || sh->Hq > 65536 || sh->Hk > 65536 || sh->P > lim || sh->B * sh->S > lim ||
        sh->B * sh->S * ((sh->Hq + 1) / 2 + (sh->Hk + 1) / 2) > lim)
        return LORA_MLP_ERR_UNSUPPORTED_SHAPE;
    return LORA_MLP_OK;
}

int check_view(const lora_qk_view* v) {
    if (v == nullptr || v->data == nullptr) return LORA_MLP_ERR_INVALID_ARG;
    if (v->stride_b % 8 || v->stride_s % 8 || v->stride_h % 8) return LORA_MLP_ERR_UNSUPPORTED_SHAPE;
    return reinterpret_cast<uintptr_t>(v->data) % 16 ? LORA_MLP_ERR_MISALIGNED : LORA_MLP_OK;
}

// A written view's strides nest: in ascending order, each is at least what the
// axes before it span, so that no two of its elements are one.
int check_written(const lora_qk_view* v, const lora_qk_shape* sh, int64_t heads) {
    struct Axis {
        uint64_t stride;
        int64_t n;
    } axes[3] = {{0, heads}, {0, sh->S}, {0, sh->B}};
    const int64_t strides[3] = {v->stride_h, v->stride_s, v->stride_b};
    for (int i = 0; i < 3; ++i)
        axes[i].stride = strides[i] < 0 ? 0 - static_cast<uint64_t>(strides[i]) : static_cast<uint64_t>(strides[i]);
    for (int i : {0, 1, 0})
        if (axes[i].stride > axes[i + 1].stride) std::swap(axes[i], axes[i + 1]);
    unsigned __int128 span = static_cast<uint64_t>(sh->D);
    for (const Axis& x : axes) {
        if (x.n == 1) continue;
        if (x.stride < span) return LORA_MLP_ERR_UNSUPPORTED_SHAPE;
        span += static_cast<unsigned __int128>(x.n - 1) * x.stride;
    }
    return LORA_MLP_OK;
}

// Two views that begin at one address: whether they are the same, stride by
// stride (those of axes of one entry are never used).
bool same_begin(const lora_qk_view* x, const lora_qk_view* y) { return x->data == y->data; }
bool same_view(const lora_qk_view* x, const lora_qk_view* y, const lora_qk_shape* sh, int64_t heads) {
    return (sh->B == 1 || x->stride_b == y->stride_b) && (sh->S == 1 || x->stride_s == y->stride_s) &&
           (heads == 1 || x->stride_h == y->stride_h);
}

// `out` written in place of `in`, or not over its beginning.
int check_in_place(const lora_qk_view* out, const lora_qk_view* in, const lora_qk_shape* sh, int64_t heads) {
    return same_begin(out, in) && !same_view(out, in, sh, heads) ? LORA_MLP_ERR_INVALID_ARG : LORA_MLP_OK;
}

QkView qk_view(const lora_qk_view* v) {
    return {static_cast<uint4*>(v->data), v->stride_b / 8, v->stride_s / 8, v->stride_h / 8};
}

QkDivisor qk_divisor(int64_t d) {
    const int l = ceil_log2(static_cast<uint64_t>(d));
    return {static_cast<uint32_t>(d), static_cast<uint32_t>(((uint64_t{1} << 32) * ((uint64_t{1} << l) - d)) / d + 1), l};
}

QkArgs qk_args(const lora_qk_shape* sh, const void* q_gain, const void* k_gain, const float* cos, const float* sin,
               const int64_t* positions, int* status, int unroll) {
    QkArgs a{};
    a.gain[0] = static_cast<const uint4*>(q_gain);
    a.gain[1] = static_cast<const uint4*>(k_gain);
    a.cos = cos;
    a.sin = sin;
    a.pos = reinterpret_cast<const long long*>(positions);
    a.pos_stride = sh->position_stride;
    a.T = sh->B * sh->S;
    a.seq = qk_divisor(sh->S);
    a.P = sh->P;
    a.H[0] = static_cast<int>(sh->Hq);
    a.H[1] = static_cast<int>(sh->Hk);
    a.D = static_cast<int>(sh->D);
    a.nslot = a.D / 16;
    a.nrot = static_cast<int>(sh->rot / 16);
    a.half = static_cast<int>(sh->rot / 2);
    a.log_group = ceil_log2(static_cast<uint64_t>(a.nslot));
    a.eps = sh->eps;
    a.inv_d = 1.0f / static_cast<float>(a.D);
    a.turn = 1.0f;
    a.status = status;
    const int heads = (32 >> a.log_group) * unroll;
    // Units of several tokens where units of one would be half empty or more:
    // 80270 tokens of 4 + 1 heads of 96 forward, 61 us against 169.  Where units
    // are full they cost more, by the angles of each row: 4096 tokens of 32 + 8
    // heads of 128 both ways, 66 us against 60 with the keys alone so.
    const int64_t each[2] = {(a.H[0] + heads - 1) / heads, (a.H[1] + heads - 1) / heads}, all = a.H[0] + a.H[1];
    a.flat = 2 * all <= (each[0] + each[1]) * heads && a.T * all + 2 * heads <= INT32_MAX;
    for (int i = 0; i < 2; ++i) {
        a.by[i] = qk_divisor(a.flat ? a.H[i] : each[i]);
        a.units[i] = static_cast<uint32_t>(a.flat ? (a.T * a.H[i] + heads - 1) / heads : a.T * each[i]);
    }
    a.per_token = qk_divisor(each[0] + each[1]);
    return a;
}

template <bool FLAT, bool IN_PLACE>
auto pick_qk(bool norm, bool inter) {
    return norm ? (inter ? qk_rope_kernel<true, true, FLAT, IN_PLACE> : qk_rope_kernel<true, false, FLAT, IN_PLACE>)
                : (inter ? qk_rope_kernel<false, true, FLAT, IN_PLACE> : qk_rope_kernel<false, false, FLAT, IN_PLACE>);
}
template <bool IN_PLACE>
auto pick_qk_bwd(bool inter, bool flat) {
    return inter ? (flat ? qk_rope_bwd_kernel<true, true, IN_PLACE> : qk_rope_bwd_kernel<true, false, IN_PLACE>)
                 : (flat ? qk_rope_bwd_kernel<false, true, IN_PLACE> : qk_rope_bwd_kernel<false, false, IN_PLACE>);
}

// Both passes without the norm, and the forward with it: one unit a warp.
int launch_qk(const char* name, const QkArgs& a, bool norm, bool inter, bool in_place, cudaStream_t st) {
    const int64_t units = int64_t{a.units[0]} + a.units[1];
    const int64_t blocks = (units + kQkWarps - 1) / kQkWarps;
    auto kernel = in_place ? (a.flat ? pick_qk<true, true>(norm, inter) : pick_qk<false, true>(norm, inter))
                           : (a.flat ? pick_qk<true, false>(norm, inter) : pick_qk<false, false>(norm, inter));
    return launch(name, kernel, dim3(static_cast<unsigned>(blocks)), kQkThreads, 0, st, false, 1, a);
}

// Blocks of the backward through the norm for queries and keys: together at
// most kQkBwdBlocks, shared in proportion to their units.  A B200's 148
// multiprocessors are written out, as the workspace is sized by them, and
// lora_qk_rope_sizes needs no device; where there are fewer, blocks wait.
constexpr int64_t kQkBwdBlocks = 148 * kQkBwdBlocksPerSm;

void qk_bwd_blocks(const QkArgs& a, int64_t (&blocks)[2]) {
    const int64_t uq = a.units[0], uk = a.units[1];
    const int64_t q = std::max<int64_t>(1, kQkBwdBlocks * uq / (uq + uk));
    blocks[0] = std::min((uq + kQkWarps - 1) / kQkWarps, std::min(q, kQkBwdBlocks - 1));
    blocks[1] = std::min((uk + kQkWarps - 1) / kQkWarps, std::max<int64_t>(1, kQkBwdBlocks - q));
}

}  // namespace

extern "C" {

int lora_qk_rope_forward(const lora_qk_shape* shape, const lora_qk_view* q, const lora_qk_view* k,
                         const void* q_gain, const void* k_gain, const float* cos, const float* sin,
                         const int64_t* positions, const lora_qk_view* q_out, const lora_qk_view* k_out,
                         void* stream) {
    STEP_TRY(validate_qk(shape));
    if ((q_gain == nullptr) != (k_gain == nullptr)) return LORA_MLP_ERR_INVALID_ARG;
    if (positions == nullptr && shape->S > shape->P) return LORA_MLP_ERR_INVALID_ARG;
    for (const lora_qk_view* v : {q, k, q_out, k_out}) STEP_TRY(check_view(v));
    STEP_TRY(check_args({{cos, 16}, {sin, 16}}));
    STEP_TRY(check_optional({{q_gain, 16}, {k_gain, 16}, {positions, 8}}));
    STEP_TRY(check_written(q_out, shape, shape->Hq));
    STEP_TRY(check_written(k_out, shape, shape->Hk));
    STEP_TRY(check_in_place(q_out, q, shape, shape->Hq));
    STEP_TRY(check_in_place(k_out, k, shape, shape->Hk));
    if (same_begin(q_out, k) || same_begin(k_out, q) || same_begin(q_out, k_out)) return LORA_MLP_ERR_INVALID_ARG;
    STEP_TRY(check_memory({{q->data, 16}, {k->data, 16}, {q_out->data, 16}, {k_out->data, 16}, {q_gain, 16},
                           {k_gain, 16}, {cos, 16}, {sin, 16}, {positions, 8}}));
    DevInfo di;
    STEP_TRY(device_info(&di));
    QkArgs a = qk_args(shape, q_gain, k_gain, cos, sin, positions, di.status,
                       q_gain != nullptr ? kQkUnroll : kQkRopeUnroll);
    a.in[0] = qk_view(q);
    a.in[1] = qk_view(k);
    a.out[0] = qk_view(q_out);
    a.out[1] = qk_view(k_out);
    return launch_qk("QK_rope_fwd", a, q_gain != nullptr, shape->interleaved != 0,
                     same_begin(q_out, q) || same_begin(k_out, k), static_cast<cudaStream_t>(stream));
}

int lora_qk_rope_sizes(const lora_qk_shape* shape, size_t* workspace_bytes) {
    STEP_TRY(validate_qk(shape));
    if (workspace_bytes) *workspace_bytes = static_cast<size_t>(kQkBwdBlocks) * static_cast<size_t>(shape->D) * 4;
    return LORA_MLP_OK;
}

int lora_qk_rope_backward(const lora_qk_shape* shape, const lora_qk_view* q, const lora_qk_view* k,
                          const void* q_gain, const void* k_gain, const float* cos, const float* sin,
                          const int64_t* positions, const lora_qk_view* dq_out, const lora_qk_view* dk_out,
                          const lora_qk_view* dq, const lora_qk_view* dk, float* dq_gain, float* dk_gain,
                          void* workspace, size_t workspace_bytes, void* stream) {
    STEP_TRY(validate_qk(shape));
    const bool norm = q_gain != nullptr, gains = dq_gain != nullptr;
    if (norm != (k_gain != nullptr) || gains != (dk_gain != nullptr) || (gains && !norm)) return LORA_MLP_ERR_INVALID_ARG;
    if (positions == nullptr && shape->S > shape->P) return LORA_MLP_ERR_INVALID_ARG;
    for (const lora_qk_view* v : {dq_out, dk_out, dq, dk}) STEP_TRY(check_view(v));
    if (norm)
        for (const lora_qk_view* v : {q, k}) STEP_TRY(check_view(v));
    STEP_TRY(check_args({{cos, 16}, {sin, 16}}));
    STEP_TRY(check_optional({{q_gain, 16}, {k_gain, 16}, {positions, 8}, {dq_gain, 4}, {dk_gain, 4}}));
    if (gains) {
        STEP_TRY(check_args({{workspace, 16}}));
        size_t need = 0;
        STEP_TRY(lora_qk_rope_sizes(shape, &need));
        if (workspace_bytes < need) return LORA_MLP_ERR_WORKSPACE_TOO_SMALL;
    }
    STEP_TRY(check_written(dq, shape, shape->Hq));
    STEP_TRY(check_written(dk, shape, shape->Hk));
    STEP_TRY(check_in_place(dq, dq_out, shape, shape->Hq));
    STEP_TRY(check_in_place(dk, dk_out, shape, shape->Hk));
    if (same_begin(dq, dk_out) || same_begin(dk, dq_out) || same_begin(dq, dk)) return LORA_MLP_ERR_INVALID_ARG;
    if (norm) {
        STEP_TRY(check_in_place(dq, q, shape, shape->Hq));
        STEP_TRY(check_in_place(dk, k, shape, shape->Hk));
        if (same_begin(dq, k) || same_begin(dk, q)) return LORA_MLP_ERR_INVALID_ARG;
    }
    STEP_TRY(check_memory({{norm ? q->data : nullptr, 16}, {norm ? k->data : nullptr, 16}, {dq_out->data, 16},
                           {dk_out->data, 16}, {dq->data, 16}, {dk->data, 16}, {q_gain, 16}, {k_gain, 16}, {cos, 16},
                           {sin, 16}, {positions, 8}, {dq_gain, 4}, {dk_gain, 4}, {gains ? workspace : nullptr, 16}}));
    DevInfo di;
    STEP_TRY(device_info(&di));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    QkArgs a = qk_args(shape, q_gain, k_gain, cos, sin, positions, di.status, norm ? kQkBwdUnroll : kQkRopeUnroll);
    a.in[0] = qk_view(dq_out);
    a.in[1] = qk_view(dk_out);
    a.out[0] = qk_view(dq);
    a.out[1] = qk_view(dk);
    a.turn = -1.0f;
    const bool in_place = same_begin(dq, dq_out) || same_begin(dk, dk_out) ||
                          (norm && (same_begin(dq, q) || same_begin(dk, k)));
    if (!norm) return launch_qk("QK_rope_bwd", a, false, shape->interleaved != 0, in_place, st);
    a.x[0] = qk_view(q);
    a.x[1] = qk_view(k);
    a.part = gains ? static_cast<float*>(workspace) : nullptr;
    int64_t blocks[2];
    qk_bwd_blocks(a, blocks);
    a.blocks_q = static_cast<int>(blocks[0]);
    const int all = static_cast<int>(blocks[0] + blocks[1]);
    auto kernel = in_place ? pick_qk_bwd<true>(shape->interleaved != 0, a.flat != 0)
                           : pick_qk_bwd<false>(shape->interleaved != 0, a.flat != 0);
    STEP_TRY(launch("QK_norm_rope_bwd", kernel,
                    dim3(static_cast<unsigned>(all)), kQkThreads, 0, st, false, 1, a));
    if (!gains) return LORA_MLP_OK;
    return launch("QK_gain_grads", qk_gain_kernel, dim3(static_cast<unsigned>((a.D + 31) / 32), 2), dim3(32, 32), 0, st,
                  true, 1, static_cast<const float*>(a.part), a.D, a.blocks_q, all, dq_gain, dk_gain);
}

}  // extern "C"

// ============================================================================= distillation

namespace {

constexpr size_t kDsMaxSmem = 226 * 1024;  // a block's, beside its static part
constexpr int kDsMaxCluster = 8;
constexpr int64_t kDsMaxV = 5 << 16;  // what eight blocks hold with kDsMaxK teacher's entries

int validate_distill(const lora_distill_shape* sh) {
    if (sh == nullptr) return LORA_MLP_ERR_INVALID_ARG;
    if (sh->N < 1 || sh->V < 1 || sh->K < 1 || sh->ld < sh->V) return LORA_MLP_ERR_INVALID_ARG;
    if (!std::isfinite(sh->temperature) || !(sh->temperature > 0.0f)) return LORA_MLP_ERR_INVALID_ARG;
    if (!std::isfinite(sh->logit_scale) || sh->logit_scale == 0.0f) return LORA_MLP_ERR_INVALID_ARG;
    if (!std::isfinite(sh->softcap) || sh->softcap < 0.0f) return LORA_MLP_ERR_INVALID_ARG;
    // the kernel's factors of an exponent, and of the teacher's
    const double T = sh->temperature, cap = sh->softcap, scale = std::fabs(static_cast<double>(sh->logit_scale));
    const double unit = cap > 0.0 ? std::max(2.0 * cap / T, 2.0 * scale / cap) : scale / T;
    if (!(std::max(unit, 1.0 / T) < 1e38)) return LORA_MLP_ERR_INVALID_ARG;
    if (sh->values_type != LORA_DISTILL_VALUES_BF16 && sh->values_type != LORA_DISTILL_VALUES_FP32)
        return LORA_MLP_ERR_INVALID_ARG;
    if (sh->ids_type != LORA_DISTILL_IDS_INT32 && sh->ids_type != LORA_DISTILL_IDS_INT64)
        return LORA_MLP_ERR_INVALID_ARG;
    if (sh->ld % 8 || sh->K > kDsMaxK || sh->V > kDsMaxV || sh->N > INT32_MAX / kDsMaxCluster)
        return LORA_MLP_ERR_UNSUPPORTED_SHAPE;
    return LORA_MLP_OK;
}

int ds_cap_form(const lora_distill_shape* sh) {
    if (!(sh->softcap > 0.0f)) return kDsNoCap;
    return sh->softcap / sh->temperature > kDsWide ? kDsWideCap : kDsCap;
}

DsArgs ds_args(const lora_distill_shape* sh, const void* logits, const void* values, const void* ids,
               const int64_t* labels, int* status) {
    DsArgs a{};
    a.z = static_cast<const __nv_bfloat16*>(logits);
    a.ld = sh->ld;
    a.V = sh->V;
    a.N = sh->N;
    a.K = static_cast<int>(sh->K);
    a.log_table = std::max(5, ceil_log2(2 * static_cast<uint64_t>(a.K)));
    a.values = values;
    a.ids = ids;
    a.values_f32 = sh->values_type == LORA_DISTILL_VALUES_FP32;
    a.ids_i64 = sh->ids_type == LORA_DISTILL_IDS_INT64;
    a.labels = reinterpret_cast<const long long*>(labels);
    a.ignore = sh->ignore_index;
    a.T = sh->temperature;
    a.inv_T = 1.0f / sh->temperature;
    a.scale = sh->logit_scale;
    a.sign = sh->logit_scale < 0.0f ? -1.0f : 1.0f;
    a.cap = sh->softcap;
    a.form = ds_cap_form(sh);
    constexpr double kLog2e = 1.4426950408889634;
    double kn = 1.0 * sh->logit_scale / sh->temperature;
    if (sh->softcap > 0.0f) {
        const double ratio = 1.0 * sh->logit_scale / sh->softcap;
        kn = (ds_cap_form(sh) == kDsWideCap ? 1.0 : 2.0 * sh->softcap) / sh->temperature;
        a.cap2 = static_cast<float>(2.0 * ratio * kLog2e);
        a.ratio2 = std::fabs(ratio) < 0x1p-60 ? 0x1p-60f : 1.0f;
        a.ratio = static_cast<float>(ratio / a.ratio2);
    }
    a.k = static_cast<float>(kn * kLog2e);
    a.status = status;
    a.wait_limit = g_wait_limit.load();
    a.force_timeout = g_force_timeout.load();
    return a;
}

// A launch that is settled but for its call, so that a refusal comes before the
// first kernel of an entry.
struct DsLaunch {
    DsArgs a;
    void (*kernel)(DsArgs);
    int threads, cluster;
    int64_t clusters;
    size_t smem;
};

// T threads for a slice, chunks of at most B vectors each.  The smallest
// cluster whose blocks hold their slice and the chunks around it in shared
// memory; a larger one where there are too few rows for the multiprocessors.
template <bool GRAD, int T, int B>
int plan_distill_by(const DsArgs& args, int sms, DsLaunch& l) {
    constexpr int64_t widest = T * B;  // vectors of a chunk
    l.a = args;
    DsArgs& a = l.a;
    l.threads = T + 32 * kDsTeachers;
    const auto fixed = [&](int lc) {
        return kDsTeachers * ((static_cast<size_t>(a.K) + 3) / 4 * 4 * kDsEntryBytes + (size_t{4} << a.log_table)) +
               static_cast<size_t>(kDsDepth + 2) * (T / 32 * 8 << lc);
    };
    const auto slice = [&](int lc) { return (((a.V + (1 << lc) - 1) >> lc) + 7) / 8; };
    const auto chunks = [&](int lc) { return (slice(lc) + widest - 1) / widest; };
    const auto chunk = [&](int lc) { return (slice(lc) + chunks(lc) - 1) / chunks(lc); };
    const auto most = [&](int lc) { return static_cast<int64_t>((kDsMaxSmem - fixed(lc)) / (chunk(lc) * 16)); };
    int lc = 0;
    while ((1 << lc) < kDsMaxCluster && ((GRAD && chunks(lc) + 1 + kDsAhead > most(lc)) ||
                                         ((a.N << lc) * 2 <= sms && chunks(lc) > 1)))
        ++lc;
    a.log_cluster = lc;
    a.slice = static_cast<int>(slice(lc) * 8);
    a.chunks = static_cast<int>(chunks(lc));
    a.chunk = static_cast<int>(chunk(lc));
    // a chunk more than the row's, where there is room: the sums' way to the
    // other blocks is then hidden behind it
    a.lag = a.chunks + (a.chunks > 1 && (!GRAD || a.chunks + 2 + kDsAhead <= most(lc)) ? 2 : 1);
    a.slots = (GRAD ? a.lag : 0) + kDsAhead;
    if (a.slots > most(lc)) return LORA_MLP_ERR_UNSUPPORTED_SHAPE;
    l.cluster = 1 << lc;
    l.smem = std::max(static_cast<size_t>(a.slots) * a.chunk * 16 + fixed(lc),
                      static_cast<size_t>(l.threads) * 12);  // 12: the reduction's sums and counts
    l.kernel = a.form == kDsNoCap ? distill_kernel<GRAD, kDsNoCap, T, B>
               : a.form == kDsCap ? distill_kernel<GRAD, kDsCap, T, B>
                                  : distill_kernel<GRAD, kDsWideCap, T, B>;
    // As many clusters as run at once; each takes every so many-th row.
    int at_once = 0;
    STEP_TRY(resident_clusters(l.kernel, kDsMaxSmem, l.threads, l.smem, l.cluster, &at_once));
    l.clusters = std::min<int64_t>(a.N, at_once);
    return LORA_MLP_OK;
}

// The gradient takes an SM for each block: 512 threads and chunks of 24 KB (453
// us at 4096 rows of 128256; 460 with 16 KB), which do not fit where a row is
// long and K large.  The loss alone needs no row resident: blocks of 256
// threads, two an SM, 24 KB a chunk (107 us there; 111 with 16 KB).  Short rows
// take blocks of 64 threads, so that a thread has work to overlap.
int plan_distill(const DsArgs& a, int sms, DsLaunch& l) {
    const bool grad = a.dz != nullptr;
    if (a.V <= 4096) return grad ? plan_distill_by<true, 64, 4>(a, sms, l) : plan_distill_by<false, 64, 4>(a, sms, l);
    if (!grad) return plan_distill_by<false, 256, 6>(a, sms, l);
    const int rc = plan_distill_by<true, 512, 3>(a, sms, l);
    return rc == LORA_MLP_ERR_UNSUPPORTED_SHAPE ? plan_distill_by<true, 512, 2>(a, sms, l) : rc;
}

int launch_distill(const char* name, const DsLaunch& l, cudaStream_t st, bool after_own) {
    return launch(name, l.kernel, dim3(static_cast<unsigned>(l.clusters * l.cluster)), dim3(l.threads), l.smem, st,
                  after_own, l.cluster, l.a);
}

int check_distill(const lora_distill_shape* sh, const void* logits, const void* values, const void* ids,
                  const int64_t* labels) {
    const size_t va = sh->values_type == LORA_DISTILL_VALUES_FP32 ? 4 : 2;
    const size_t ia = sh->ids_type == LORA_DISTILL_IDS_INT64 ? 8 : 4;
    STEP_TRY(check_args({{logits, 16}, {values, va}, {ids, ia}}));
    return check_optional({{labels, 8}});
}

}  // namespace

extern "C" {

int lora_distill_forward(const lora_distill_shape* shape, const void* logits, const void* values, const void* ids,
                         const int64_t* labels, float* loss, void* stream) {
    STEP_TRY(validate_distill(shape));
    STEP_TRY(check_distill(shape, logits, values, ids, labels));
    STEP_TRY(check_args({{loss, 4}}));
    STEP_TRY(check_memory({{logits, 1}, {values, 1}, {ids, 1}, {labels, 1}, {loss, 1}}));
    DevInfo di;
    STEP_TRY(device_info(&di));
    DsArgs a = ds_args(shape, logits, values, ids, labels, di.status);
    a.loss = loss;
    DsLaunch l;
    STEP_TRY(plan_distill(a, di.sms, l));
    return launch_distill("DISTILL_fwd", l, static_cast<cudaStream_t>(stream), false);
}

int lora_distill_backward(const lora_distill_shape* shape, const void* logits, const void* values, const void* ids,
                          const int64_t* labels, const float* dloss, void* dlogits, void* stream) {
    STEP_TRY(validate_distill(shape));
    STEP_TRY(check_distill(shape, logits, values, ids, labels));
    STEP_TRY(check_args({{dloss, 4}, {dlogits, 16}}));
    STEP_TRY(check_memory({{logits, 1}, {values, 1}, {ids, 1}, {labels, 1}, {dloss, 1}, {dlogits, 1}}));
    DevInfo di;
    STEP_TRY(device_info(&di));
    DsArgs a = ds_args(shape, logits, values, ids, labels, di.status);
    a.dloss = dloss;
    a.dloss_stride = 1;
    a.dz = static_cast<__nv_bfloat16*>(dlogits);
    DsLaunch l;
    STEP_TRY(plan_distill(a, di.sms, l));
    return launch_distill("DISTILL_bwd", l, static_cast<cudaStream_t>(stream), false);
}

int lora_distill_backward_reduced(const lora_distill_shape* shape, const void* logits, const void* values,
                                  const void* ids, const int64_t* labels, const float* dout, const float* fwd_out,
                                  void* dlogits, void* stream) {
    STEP_TRY(validate_distill(shape));
    STEP_TRY(check_distill(shape, logits, values, ids, labels));
    STEP_TRY(check_args({{dout, 4}, {fwd_out, 8}, {dlogits, 16}}));
    STEP_TRY(check_memory({{logits, 1}, {values, 1}, {ids, 1}, {labels, 1}, {dout, 1}, {fwd_out, 1}, {dlogits, 1}}));
    DevInfo di;
    STEP_TRY(device_info(&di));
    DsArgs a = ds_args(shape, logits, values, ids, labels, di.status);
    a.dloss = dout;
    a.factor = fwd_out;
    a.dz = static_cast<__nv_bfloat16*>(dlogits);
    DsLaunch l;
    STEP_TRY(plan_distill(a, di.sms, l));
    return launch_distill("DISTILL_bwd", l, static_cast<cudaStream_t>(stream), false);
}

int lora_distill_sizes(const lora_distill_shape* shape, size_t* workspace_bytes) {
    STEP_TRY(validate_distill(shape));
    if (workspace_bytes) *workspace_bytes = kAlign + static_cast<size_t>(shape->N) * 4;
    return LORA_MLP_OK;
}

int lora_distill_loss(const lora_distill_shape* shape, const void* logits, const void* values, const void* ids,
                      const int64_t* labels, int reduction, float* out, void* dlogits, void* workspace,
                      size_t workspace_bytes, void* stream) {
    STEP_TRY(validate_distill(shape));
    if (reduction != LORA_DISTILL_REDUCTION_SUM && reduction != LORA_DISTILL_REDUCTION_MEAN)
        return LORA_MLP_ERR_INVALID_ARG;
    STEP_TRY(check_distill(shape, logits, values, ids, labels));
    STEP_TRY(check_args({{out, 8}, {workspace, 16}}));
    STEP_TRY(check_optional({{dlogits, 16}}));
    size_t need = 0;
    STEP_TRY(lora_distill_sizes(shape, &need));
    if (workspace_bytes < need) return LORA_MLP_ERR_WORKSPACE_TOO_SMALL;
    STEP_TRY(check_memory({{logits, 1}, {values, 1}, {ids, 1}, {labels, 1}, {out, 1}, {dlogits, 1}, {workspace, 1}}));
    DevInfo di;
    STEP_TRY(device_info(&di));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool mean = reduction == LORA_DISTILL_REDUCTION_MEAN;
    DsArgs a = ds_args(shape, logits, values, ids, labels, di.status);
    a.counter = static_cast<uint32_t*>(workspace);
    a.loss = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kAlign);
    a.dz = static_cast<__nv_bfloat16*>(dlogits);
    a.out = out;
    a.factor = out;
    a.mean = mean;
    DsLaunch l;
    STEP_TRY(plan_distill(a, di.sms, l));
    STEP_TRY(launch("DISTILL_count", distill_count_kernel, dim3(1), kDsCountThreads, 0, st, false, 1, a.labels, a.N,
                    a.ignore, a.mean, out, a.counter));
    return launch_distill(dlogits != nullptr ? "DISTILL_loss_grad" : "DISTILL_fwd", l, st, true);
}

}  // extern "C"
