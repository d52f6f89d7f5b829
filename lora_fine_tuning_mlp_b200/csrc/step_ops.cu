// C ABI of the operators around a fine-tuning step's dense layers
// (include/lora_step.h, lora_embedding.h): argument checks, workspace layout
// and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <mutex>
#include <vector>

#include "lora_embedding.h"
#include "embedding.cuh"

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
// (programmatic dependent launch).
template <class... P, class... A>
int launch(const char* name, void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st,
           bool after_own, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = after_own ? 1 : 0;
    LaunchScope scope(name, st);
    if (cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) != cudaSuccess) {
        cudaGetLastError();
        return LORA_MLP_ERR_CUDA;
    }
    return LORA_MLP_OK;
}

// Raises a kernel's dynamic shared memory limit, once a device.
template <class K>
int allow_smem(K* kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) ==
                   cudaSuccess
               ? LORA_MLP_OK
               : LORA_MLP_ERR_CUDA;
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
    int nv, slices, nchunks, bits, passes, ntiles;
    bool small;
    size_t key[2], val[2], hist, counters, part, total;
};

EmbPlan make_emb_plan(int64_t N, int64_t V, int64_t d) {
    EmbPlan p{};
    p.nv = static_cast<int>(d / 8);
    p.slices = (p.nv + kEmbThreads - 1) / kEmbThreads;
    p.nchunks = static_cast<int>(N / kEmbChunk);
    const int key_bits = std::max(1, ceil_log2(static_cast<uint64_t>(V) + 1));  // keys 0 .. V
    p.passes = (key_bits + kSortMaxBits - 1) / kSortMaxBits;
    p.bits = (key_bits + p.passes - 1) / p.passes;
    p.small = N <= kSortSmall;
    p.ntiles = static_cast<int>((N + kSortTile - 1) / kSortTile);
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
    a.log_tpr = ceil_log2(static_cast<uint64_t>(std::min(a.nv, kEmbThreads)));
    a.scale = scale;
    a.status = di.status;
    const int rows = kEmbThreads >> a.log_tpr;
    return launch("EMB_fwd", embed_fwd_kernel, dim3(static_cast<unsigned>((N + rows - 1) / rows)), kEmbThreads, 0,
                  static_cast<cudaStream_t>(stream), false, a);
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
    for (int i = 0; i < 2; ++i) {
        s.key[i] = reinterpret_cast<uint32_t*>(ws + p.key[i]);
        s.val[i] = reinterpret_cast<uint32_t*>(ws + p.val[i]);
    }
    s.hist = reinterpret_cast<uint32_t*>(ws + p.hist);
    s.counters = reinterpret_cast<uint32_t*>(ws + p.counters);
    s.ncounters = p.nchunks * p.slices;
    s.status = di.status;
    if (p.small) {
        const size_t smem = sizeof(SortShared) + 2 * sizeof(uint32_t) * kSortSmall;
        STEP_TRY(allow_smem(embed_sort_small_kernel, smem));
        STEP_TRY(launch("EMB_sort", embed_sort_small_kernel, dim3(1), kSortThreads, smem, st, false, s));
    } else {
        const dim3 grid(static_cast<unsigned>(p.ntiles));
        STEP_TRY(launch("EMB_sort_count", embed_sort_count_kernel, grid, kSortThreads, 0, st, false, s));
        for (int i = 0; i < p.passes; ++i)
            STEP_TRY(launch("EMB_sort_scatter", embed_sort_scatter_kernel, grid, kSortThreads, sizeof(SortShared), st,
                            true, s, i));
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
    a.log_worker = std::max(5, ceil_log2(static_cast<uint64_t>(std::min(p.nv, kEmbThreads))));
    a.scale = scale;
    // Rows of a worker: about kEmbBlockBytes of dE a block, but eight blocks a
    // multiprocessor where the vocabulary is small.
    const bool f32 = grad_type == LORA_EMBEDDING_GRAD_FP32;
    const int64_t workers = kEmbThreads >> a.log_worker, row_bytes = d * (f32 ? 4 : 2);
    const int64_t by_bytes = kEmbBlockBytes / (row_bytes * workers), spread = int64_t{8} * di.sms * workers;
    a.rows_w = static_cast<int>(std::max<int64_t>(1, std::min(by_bytes, (V + spread - 1) / spread)));
    const int64_t nrow = (V + a.rows_w * workers - 1) / (a.rows_w * workers);
    const int64_t blocks = nrow + static_cast<int64_t>(p.nchunks) * p.slices;
    if (blocks > INT32_MAX) return LORA_MLP_ERR_UNSUPPORTED_SHAPE;
    a.first_wave = static_cast<int>(std::min<int64_t>(nrow, int64_t{kEmbBlocksPerSm} * di.sms));
    const dim3 grid(static_cast<unsigned>(blocks));
    if (f32) return launch("EMB_grad", embed_bwd_kernel<true>, grid, kEmbThreads, 0, st, true, a);
    return launch("EMB_grad", embed_bwd_kernel<false>, grid, kEmbThreads, 0, st, true, a);
}

}  // extern "C"
