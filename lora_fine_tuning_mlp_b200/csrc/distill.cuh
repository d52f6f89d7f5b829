// Distillation from a teacher's top logits, loss and gradient
// (include/lora_distill.h).
//
//   x = t(z) / T,  q = softmax(x),  p = softmax(a / T) over the K entries
//   loss = T^2 sum p_i (log p_i - log q_ci),   dz_j = g T (q_j - p_j) dt/dz
//
// The gradient needs the row's softmax sum before its first element, so a
// kernel that streams rows from HBM has to read them twice.  Here a row stays
// on the chip: a cluster of 1, 2, 4 or 8 blocks holds it in shared memory as
// the bf16 it came in, a slice each, the blocks exchange their (maximum, sum)
// through distributed shared memory, and the gradient is formed from the
// resident slice: 2 bytes a logit in, 2 out, nothing else.  Several blocks to
// a multiprocessor overlap one's loads with another's arithmetic.
//
// Every thread copies the 16-byte vectors that it later reads (cp.async), so
// the loads need no barrier.  Sums are taken of 2^((z - m) k) with the
// difference formed first: exact next to the maximum, and rows filled with
// bf16's lowest value or with large logits neither overflow nor vanish.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "f32x2.cuh"
#include "vec8.cuh"

namespace lmlp {
namespace step {

constexpr int kDsMaxThreads = 256;
constexpr int kDsMaxCluster = 8;
constexpr int kDsMaxK = 1024;
constexpr float kDsLowest = -3.3895313892515355e38f;  // bf16's lowest finite value

struct DsArgs {
    const __nv_bfloat16* z;
    __nv_bfloat16* dz;
    long long ld, V, N;
    int K;
    int slice;  // logits of a block: a multiple of 8
    int log_cluster;
    const void *values, *ids;
    int values_f32, ids_i64;
    const long long* labels;  // may be null
    long long ignore;
    float inv_T, T;
    float scale, cap;     // s with its sign taken off (see flip), cap or 0
    uint32_t flip;        // 0x80008000 where s is negative: z and dz change sign
    float k;              // log2(e) / T, times s without softcapping: exponents in base 2 per unit of z (of t)
    float kn;             // the same per unit, base e
    float cap2;           // 2 s / cap * log2(e)
    float* loss;          // may be null
    const float* dloss;   // [N], stride 0 or 1 (null: 1)
    long long dloss_stride;
    const float* factor;  // factor[1] multiplies it (null: 1)
    int* status;
};

__device__ __forceinline__ float ds_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float ds_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t ds_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void ds_cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void ds_cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// What exponents are taken of: z itself, or t = cap tanh(s z / cap) = cap -
// 2 cap / (1 + 2^(cap2 z)), whose reciprocal saturates to 0 or 1 where tanh is
// +-1.
template <bool CAP>
__device__ __forceinline__ float ds_t(const DsArgs& a, float z) {
    return CAP ? fmaf(ds_rcp(1.0f + ds_ex2(a.cap2 * z)), -2.0f * a.cap, a.cap) : z;
}

// (m, s) := (max, sum of 2^((x - max) k)) of the union of two sets.
__device__ __forceinline__ void ds_merge(float& m, float& s, float m2, float s2, float k) {
    const float M = fmaxf(m, m2);
    s = s * ds_ex2((m - M) * k) + s2 * ds_ex2((m2 - M) * k);
    m = M;
}

struct DsShared {
    float2 warp[kDsMaxThreads / 32];
    float2 all[kDsMaxCluster];  // written by every block of the cluster
    float red[kDsMaxThreads / 32];
    int bad;
};

// Sum over the block, the same bits for every thread.
__device__ __forceinline__ float ds_block_sum(DsShared& s, float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = s.red[0];
    for (int w = 1; w < static_cast<int>(blockDim.x >> 5); ++w) v += s.red[w];
    return v;
}
__device__ __forceinline__ float ds_block_max(DsShared& s, float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = s.red[0];
    for (int w = 1; w < static_cast<int>(blockDim.x >> 5); ++w) v = fmaxf(v, s.red[w]);
    return v;
}

template <bool CAP>
__device__ __forceinline__ void ds_load8(const DsArgs& a, uint4 v, float (&z)[8]) {
    v.x ^= a.flip, v.y ^= a.flip, v.z ^= a.flip, v.w ^= a.flip;
    widen8(v, z);
    if (CAP) {
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = ds_t<true>(a, z[e]);
    }
}

// One row a cluster.
template <bool GRAD, bool CAP>
__global__ void __launch_bounds__(kDsMaxThreads) distill_kernel(const DsArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    __shared__ DsShared sh;
    let_next();
    const int T = blockDim.x, tid = threadIdx.x;
    const uint32_t rank = ds_rank();
    const long long row = blockIdx.x >> a.log_cluster;
    const long long c0 = static_cast<long long>(rank) * a.slice;
    const int n = static_cast<int>(max(0LL, min(static_cast<long long>(a.slice), a.V - c0)));  // this block's logits
    const int nvec = (n + 7) >> 3, nfull = n >> 3;
    uint4* slice = reinterpret_cast<uint4*>(raw);
    float* tp = reinterpret_cast<float*>(raw + static_cast<size_t>(a.slice) * 2);  // teacher's p
    float* tx = tp + a.K;                                                         // rank 0: log q + its constant
    int* tc = reinterpret_cast<int*>(tx + a.K);                                   // teacher's ids
    const __nv_bfloat16* z = a.z + row * a.ld + c0;
    const bool ignored = a.labels != nullptr && a.labels[row] == a.ignore;
    if (ignored) {  // the same for the whole cluster
        wait_prior();
        if (GRAD) {
            __nv_bfloat16* dz = a.dz + row * a.ld + c0;
            for (int j = tid; j < nfull; j += T) reinterpret_cast<uint4*>(dz)[j] = make_uint4(0u, 0u, 0u, 0u);
            if (tid < n - 8 * nfull) dz[8 * nfull + tid] = __float2bfloat16(0.0f);
        }
        if (a.loss != nullptr && rank == 0 && tid == 0) a.loss[row] = 0.0f;
        return;
    }
    ds_cluster_arrive();
    const uint32_t sbase = static_cast<uint32_t>(__cvta_generic_to_shared(slice));
    for (int j = tid; j < nfull; j += T)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sbase + 16u * j), "l"(z + 8 * j) : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (nfull < nvec && tid == nfull % T) {  // the thread that reads the last, partial vector: V need not be a
        uint16_t* last = reinterpret_cast<uint16_t*>(slice + nfull);  // multiple of 8, nor the row padded
        for (int e = 0; e < 8; ++e)
            last[e] = e < n - 8 * nfull ? __bfloat16_as_ushort(z[8 * nfull + e]) : static_cast<uint16_t>(0);
    }

    // The teacher's softmax over its entries, by every block for itself; block
    // 0 also fetches the student's logits at them for the loss.
    if (tid == 0) sh.bad = 0;
    __syncthreads();
    float amax = -3.4028234663852886e38f;  // fp32's lowest, which a teacher's mask may hold
    bool any = false;
    for (int i = tid; i < a.K; i += T) {
        const long long at = row * a.K + i;
        const long long id = a.ids_i64 ? static_cast<const long long*>(a.ids)[at] : static_cast<const int*>(a.ids)[at];
        const float v = a.values_f32 ? static_cast<const float*>(a.values)[at]
                                     : __bfloat162float(static_cast<const __nv_bfloat16*>(a.values)[at]);
        const bool in = id >= 0 && id < a.V;
        if (id < -1 || id >= a.V) sh.bad = 1;
        tc[i] = in ? static_cast<int>(id) : -1;
        tp[i] = v;
        if (in) {
            amax = fmaxf(amax, v);
            any = any || !(v == -INFINITY);
        }
        if (rank == 0 && in) {
            float zc = __bfloat162float(a.z[row * a.ld + id]);
            if (a.flip) zc = -zc;
            tx[i] = CAP ? a.cap * tanhf(a.scale / a.cap * zc) : zc;
        }
    }
    const float A = ds_block_max(sh, amax);
    const bool live = __syncthreads_or(any);
    float psum = 0.0f;
    for (int i = tid; i < a.K; i += T)
        if (tc[i] >= 0) psum += expf((tp[i] - A) * a.inv_T);
    psum = ds_block_sum(sh, psum);
    const float logp0 = logf(psum), inv_psum = 1.0f / psum;

    // The slice's maximum and sum.
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    float m = kDsLowest, s = 0.0f;
    {
        uint32_t m2 = 0xFF7FFF7Fu;  // two of bf16's lowest
        for (int j = tid; j < nvec; j += T) {
            const uint4 v = slice[j];
            const uint32_t w[4] = {v.x ^ a.flip, v.y ^ a.flip, v.z ^ a.flip, v.w ^ a.flip};
            if (j < nfull) {
#pragma unroll
                for (int i = 0; i < 4; ++i) asm("max.bf16x2 %0, %0, %1;" : "+r"(m2) : "r"(w[i]));
            } else {
                for (int e = 0; e < n - 8 * nfull; ++e)
                    m = fmaxf(m, __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16));
            }
        }
        m = fmaxf(m, fmaxf(__uint_as_float(m2 << 16), __uint_as_float(m2 & 0xFFFF0000u)));
        if (CAP) m = ds_t<true>(a, m);
    }
    for (int j = tid; j < nvec; j += T) {
        float x[8];
        ds_load8<CAP>(a, slice[j], x);
        if (j >= nfull)
            for (int e = 0; e < 8; ++e)
                if (e >= n - 8 * nfull) x[e] = -INFINITY;
        const uint64_t mm = f2_packf(m, m), kk = f2_packf(a.k, a.k);
        float part[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lo, hi;
            f2_unpack(f2_mul(f2_sub(f2_packf(x[2 * i], x[2 * i + 1]), mm), kk), lo, hi);
            part[i] = ds_ex2(lo) + ds_ex2(hi);
        }
        s += (part[0] + part[1]) + (part[2] + part[3]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
        ds_merge(m, s, m2, s2, a.k);
    }
    if ((tid & 31) == 0) sh.warp[tid >> 5] = make_float2(m, s);
    __syncthreads();
    ds_cluster_wait();  // every block of the cluster runs: its shared memory may be written
    const uint32_t cluster = 1u << a.log_cluster;
    if (tid < static_cast<int>(cluster)) {
        m = sh.warp[0].x, s = sh.warp[0].y;
        for (int w = 1; w < T / 32; ++w) ds_merge(m, s, sh.warp[w].x, sh.warp[w].y, a.k);
        uint32_t to;
        const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(&sh.all[rank]));
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(mine), "r"(tid));
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(m), "f"(s) : "memory");
    }
    ds_cluster_arrive();
    ds_cluster_wait();
    m = sh.all[0].x, s = sh.all[0].y;
    for (uint32_t r = 1; r < cluster; ++r) ds_merge(m, s, sh.all[r].x, sh.all[r].y, a.k);

    wait_prior();  // the factor may come from the kernel before
    if (rank == 0 && a.loss != nullptr) {
        const float logq0 = logf(s);
        float part = 0.0f;
        for (int i = tid; i < a.K; i += T) {
            if (tc[i] < 0) continue;
            const float la = (tp[i] - A) * a.inv_T - logp0, p = expf((tp[i] - A) * a.inv_T) * inv_psum;
            if (p != 0.0f) part += p * (la - ((tx[i] - m) * a.kn - logq0));
        }
        part = ds_block_sum(sh, part);
        if (tid == 0) {
            const bool bad = sh.bad != 0;
            if (bad) atomicExch(a.status, -1);
            a.loss[row] = bad ? __int_as_float(0x7fc00000) : (live ? a.T * a.T * part : 0.0f);
        }
    } else if (rank == 0 && tid == 0 && sh.bad) {
        atomicExch(a.status, -1);
    }
    if (!GRAD) return;

    float g = a.T * a.scale;
    if (a.flip) g = -g;
    if (a.dloss != nullptr) g *= a.dloss[row * a.dloss_stride];
    if (a.factor != nullptr) g *= a.factor[1];
    if (!live) g = 0.0f;
    const float gs = live ? g / s : 0.0f;
    const float inv_cap = CAP ? 1.0f / a.cap : 0.0f;
    __nv_bfloat16* dz = a.dz + row * a.ld + c0;
    for (int j = tid; j < nvec; j += T) {
        float x[8], d[8];
        ds_load8<CAP>(a, slice[j], x);
        const uint64_t mm = f2_packf(m, m), kk = f2_packf(a.k, a.k), gg = f2_packf(gs, gs);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t x2 = f2_packf(x[2 * i], x[2 * i + 1]);
            float lo, hi;
            f2_unpack(f2_mul(f2_sub(x2, mm), kk), lo, hi);
            uint64_t d2 = f2_mul(f2_packf(ds_ex2(lo), ds_ex2(hi)), gg);
            if (CAP) {  // times 1 - (t / cap)^2
                const uint64_t th = f2_mul(x2, f2_packf(inv_cap, inv_cap));
                const uint64_t nth = f2_mul(x2, f2_packf(-inv_cap, -inv_cap));
                d2 = f2_mul(d2, f2_fma(th, nth, f2_packf(1.0f, 1.0f)));
            }
            f2_unpack(d2, d[2 * i], d[2 * i + 1]);
        }
        if (!live)
            for (int e = 0; e < 8; ++e) d[e] = 0.0f;
        const uint4 o = round8(d);
        if (j < nfull) {
            __stcs(reinterpret_cast<uint4*>(dz) + j, o);
        } else {
            const uint32_t w[4] = {o.x, o.y, o.z, o.w};
            for (int e = 0; e < n - 8 * nfull; ++e)
                dz[8 * j + e] = __ushort_as_bfloat16(static_cast<uint16_t>(e & 1 ? w[e >> 1] >> 16 : w[e >> 1]));
        }
    }
    if (!live) return;
    __syncthreads();  // the elements below are written a second time
    for (int i = tid; i < a.K; i += T) {
        const int c = tc[i];
        const long long at = c - c0;
        if (c < 0 || at < 0 || at >= n) continue;
        bool first = true;
        float p = 0.0f;
        for (int o = 0; o < a.K; ++o) {
            if (tc[o] != c) continue;
            if (o < i) first = false;
            p += expf((tp[o] - A) * a.inv_T) * inv_psum;
        }
        if (!first) continue;  // the first entry of an id writes for all of them
        float x = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(slice)[at]);
        if (a.flip) x = -x;
        x = ds_t<CAP>(a, x);
        float d = (ds_ex2((x - m) * a.k) / s - p) * g;
        if (CAP) d *= 1.0f - (x * inv_cap) * (x * inv_cap);
        dz[at] = __float2bfloat16(d);
    }
}

// factor[1] = 1 / (rows whose label is not ignore_index) for the mean, else 1.
constexpr int kDsReduceThreads = 1024;
__global__ void __launch_bounds__(kDsReduceThreads) distill_count_kernel(const long long* labels, long long N,
                                                                         long long ignore, bool mean, float* out) {
    let_next();
    __shared__ int cnt[kDsReduceThreads / 32];
    int c = 0;
    if (mean)
        for (long long r = threadIdx.x; r < N; r += kDsReduceThreads) c += labels == nullptr || labels[r] != ignore;
    c = __reduce_add_sync(0xffffffffu, c);
    if ((threadIdx.x & 31) == 0) cnt[threadIdx.x >> 5] = c;
    __syncthreads();
    if (threadIdx.x == 0) {
        long long all = 0;
        for (int w = 0; w < kDsReduceThreads / 32; ++w) all += cnt[w];
        out[1] = mean ? static_cast<float>(1.0 / static_cast<double>(all > 0 ? all : 1)) : 1.0f;
    }
}

// out[0] = factor * sum of the rows' losses, in fp64: each thread adds every
// 1024th row, then a fixed tree adds the threads.
__global__ void __launch_bounds__(kDsReduceThreads) distill_reduce_kernel(const float* loss, long long N,
                                                                          const long long* labels, long long ignore,
                                                                          bool mean, float* out) {
    __shared__ double sum[kDsReduceThreads];
    __shared__ int cnt[kDsReduceThreads];
    wait_prior();
    double v = 0.0;
    int c = 0;
    for (long long r = threadIdx.x; r < N; r += kDsReduceThreads) {
        v += static_cast<double>(loss[r]);
        c += labels == nullptr || labels[r] != ignore;
    }
    sum[threadIdx.x] = v;
    cnt[threadIdx.x] = c;
    __syncthreads();
    for (int h = kDsReduceThreads / 2; h > 0; h >>= 1) {
        if (static_cast<int>(threadIdx.x) < h) {
            sum[threadIdx.x] += sum[threadIdx.x + h];
            cnt[threadIdx.x] += cnt[threadIdx.x + h];
        }
        __syncthreads();
    }
    if (threadIdx.x == 0)
        out[0] = static_cast<float>(mean ? sum[0] / static_cast<double>(cnt[0] > 0 ? cnt[0] : 1) : sum[0]);
}

}  // namespace step
}  // namespace lmlp
