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
// the loads need no barrier, and takes them up in four parts as they arrive;
// one warp beside them takes the teacher's softmax.  Exponents are in base 2
// and relative to fl(m k) for the maximum m: fma(z, k, -fl(m k)) rounds once,
// and sums relative to that very number are exact in it.  Where m k is out of
// fma's range (rows filled with bf16's lowest value, say) the difference z - m
// is formed first.  With softcapping, t = cap tanh(s z / cap) = cap - 2 cap r
// with r = 1 / (1 + 2^(cap2 z)): exponents are taken of -r, dt/dz = 4 s r (1 -
// r) has no cancellation where tanh saturates, and four logits share one
// reciprocal.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "f32x2.cuh"
#include "vec8.cuh"

namespace lmlp {
namespace step {

constexpr int kDsMaxThreads = 256;  // that work on the slice; a warp for the teacher comes on top
constexpr int kDsMaxCluster = 8;
constexpr int kDsMaxK = 1024;
constexpr int kDsParts = 4;   // of a thread's vectors, waited for one after the other
constexpr int kDsBatch = 4;   // vectors taken up together
constexpr int kDsEntryBytes = 16;  // of shared memory for a teacher's entry
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
    float k;              // base-2 exponent of a unit of z: s log2(e) / T; of a unit of -r: 2 cap log2(e) / T
    float cap2;           // 2 s / cap * log2(e)
    float* loss;          // may be null
    float* out;           // the reduced loss, or null
    uint32_t* counter;    // rows done, zero before the launch (with out)
    int mean;
    int threads;          // that work on the slice
    int Kp;               // K rounded up to 4
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

// What exponents are taken of: z, or -r (see above).  2^(cap2 z) is held to
// 2^30, where tanh is 1 in fp32 already, so that a product of four
// denominators stays in range; min keeps a NaN.
__device__ __forceinline__ float ds_denominator(const DsArgs& a, float z) {
    float e;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(e) : "f"(a.cap2 * z), "f"(30.0f));
    return 1.0f + ds_ex2(e);
}
template <bool CAP>
__device__ __forceinline__ float ds_arg(const DsArgs& a, float z) {
    return CAP ? -ds_rcp(ds_denominator(a, z)) : z;
}
template <bool CAP>
__device__ __forceinline__ void ds_args8(const DsArgs& a, const uint4& v, float (&x)[8]) {
    widen8(v, x);
    if constexpr (CAP) {
#pragma unroll
        for (int h = 0; h < 8; h += 4) {
            float d[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = ds_denominator(a, x[h + i]);
            const float d01 = d[0] * d[1], d23 = d[2] * d[3], r = ds_rcp(d01 * d23);
            const float n01 = -r * d23, n23 = -r * d01;
            x[h] = n01 * d[1], x[h + 1] = n01 * d[0], x[h + 2] = n23 * d[3], x[h + 3] = n23 * d[2];
        }
    }
}

__device__ __forceinline__ float ds_warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float ds_warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The vector with its signs as the scale's magnitude wants them.
__device__ __forceinline__ uint4 ds_signed(const DsArgs& a, uint4 v) {
    if (a.flip) v = make_uint4(v.x ^ a.flip, v.y ^ a.flip, v.z ^ a.flip, v.w ^ a.flip);
    return v;
}
__device__ __forceinline__ void ds_max(uint32_t& m2, const uint4& v) {
    asm("max.bf16x2 %0, %0, %1;" : "+r"(m2) : "r"(v.x));
    asm("max.bf16x2 %0, %0, %1;" : "+r"(m2) : "r"(v.y));
    asm("max.bf16x2 %0, %0, %1;" : "+r"(m2) : "r"(v.z));
    asm("max.bf16x2 %0, %0, %1;" : "+r"(m2) : "r"(v.w));
}

// Whether m k is out of the range in which z k - fl(m k) is formed by one fma.
template <bool CAP>
__device__ __forceinline__ bool ds_far(float m, float k) {
    return !CAP && !(fabsf(m * k) < 1.0e30f);
}
// A term of a sum that is relative to m.
template <bool CAP>
__device__ __forceinline__ float ds_rel(float x, float m, float k) {
    return ds_far<CAP>(m, k) ? ds_ex2((x - m) * k) : ds_ex2(fmaf(x, k, -__fmul_rn(m, k)));
}
// What turns a sum relative to m into one relative to M >= m: 2^(fl(m k) -
// fl(M k)), both products rounded (1 where m = M).
template <bool CAP>
__device__ __forceinline__ float ds_shift(float m, float M, float k) {
    return ds_far<CAP>(M, k) ? ds_ex2((m - M) * k) : ds_ex2(__fmul_rn(m, k) - __fmul_rn(M, k));
}

struct DsShared {
    float2 warp[32];            // (max, sum) of each warp
    float2 all[kDsMaxCluster];  // ... of each block of the cluster, written by all of them
    float inv_psum;             // teacher: 1 / sum of exp((a - max) / T)
    int live;                   // it has an entry that counts
    int last;                   // this block reduces the rows' losses
};

// The teacher's entries of the row, by one warp: ids to tc, exp((a - max) / T)
// to tp, its exponent to tl, and for the loss (`student`) what the student's
// exponents are taken of at them to tx.
struct DsTeacher {
    float *tp, *tl, *tx;
    int* tc;
    float log_psum;
    bool bad;
};

template <bool CAP>
__device__ __forceinline__ void ds_teacher(const DsArgs& a, DsShared& sh, DsTeacher& t, long long row, bool student) {
    const int lane = threadIdx.x & 31;
    float amax = -3.4028234663852886e38f;  // fp32's lowest, which a teacher's mask may hold
    bool any = false, bad = false;
#pragma unroll 4
    for (int i = lane; i < a.Kp; i += 32) {
        const long long at = row * a.K + min(i, a.K - 1);
        const long long id = a.ids_i64 ? static_cast<const long long*>(a.ids)[at] : static_cast<const int*>(a.ids)[at];
        const float v = a.values_f32 ? static_cast<const float*>(a.values)[at]
                                     : __bfloat162float(static_cast<const __nv_bfloat16*>(a.values)[at]);
        const bool in = i < a.K && id >= 0 && id < a.V;
        bad = bad || id < -1 || id >= a.V;
        t.tc[i] = in ? static_cast<int>(id) : -1;
        t.tl[i] = v;
        if (in) {
            amax = fmaxf(amax, v);
            any = any || !(v == -INFINITY);
            if (student) {
                float z = __bfloat162float(a.z[row * a.ld + id]);
                if (a.flip) z = -z;
                t.tx[i] = CAP ? -1.0f / (1.0f + expf(2.0f * (a.scale / a.cap * z))) : z;
            }
        }
    }
    amax = ds_warp_max(amax);
    float psum = 0.0f;
    for (int i = lane; i < a.Kp; i += 32) {
        const float l = (t.tl[i] - amax) * a.inv_T, e = t.tc[i] >= 0 ? expf(l) : 0.0f;
        t.tl[i] = l;
        t.tp[i] = e;
        psum += e;
    }
    psum = ds_warp_sum(psum);
    t.log_psum = logf(psum);
    t.bad = __any_sync(0xffffffffu, bad);
    any = __any_sync(0xffffffffu, any);
    if (lane == 0) {
        sh.inv_psum = 1.0f / psum;
        sh.live = any;
    }
}

// A batch's exponentials added up: sum of 2^(x k - m k) over the vectors j0, j0
// + T, ... below `stop`.
template <bool CAP, bool FAR>
__device__ __forceinline__ float ds_batch_sum(const DsArgs& a, const uint4 (&v)[kDsBatch], int j0, int stop, float m) {
    const float c = FAR ? m : -__fmul_rn(m, a.k);
    float s = 0.0f;
#pragma unroll
    for (int b = 0; b < kDsBatch; ++b) {
        if (j0 + b * a.threads >= stop) break;
        float x[8];
        ds_args8<CAP>(a, v[b], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = ds_ex2(FAR ? (x[e] - c) * a.k : fmaf(x[e], a.k, c));
        s += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
    }
    return s;
}

// The gradient of the whole vectors, the teacher's part left out: gs 2^(x k -
// m k) dt/dz.  The factor gs goes into the exponent (its sign apart): it is
// off by 2^-24 of that exponent, far below the rounding to bf16.
template <bool CAP, bool FAR>
__device__ __forceinline__ void ds_grad(const DsArgs& a, const uint4* slice, uint4* dz, int nfull, float m, float gs) {
    const float c = FAR ? m : log2f(fabsf(CAP ? 4.0f * gs : gs)) - __fmul_rn(m, a.k);
    const uint32_t sign = !FAR && ((gs < 0.0f) != CAP) ? 0x80008000u : 0u;  // x^2 + x below is negative
#pragma unroll 2
    for (int j = threadIdx.x; j < nfull; j += a.threads) {
        float x[8];
        ds_args8<CAP>(a, ds_signed(a, slice[j]), x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (FAR) {
                x[e] = ds_ex2((x[e] - c) * a.k) * gs;
            } else {
                const float y = ds_ex2(fmaf(x[e], a.k, c));
                x[e] = CAP ? y * fmaf(x[e], x[e], x[e]) : y;  // r (1 - r) = -(x^2 + x)
            }
        }
        uint4 o = round8(x);
        if (sign) o = make_uint4(o.x ^ sign, o.y ^ sign, o.z ^ sign, o.w ^ sign);
        __stcs(dz + j, o);
    }
}

// The rows' losses reduced by one block, in fp64 and a fixed order.
__device__ __forceinline__ void ds_reduce(const DsArgs& a, double* sum) {
    const int T = blockDim.x, tid = threadIdx.x;
    int* cnt = reinterpret_cast<int*>(sum + T);
    __threadfence();
    double v = 0.0;
    int c = 0;
#pragma unroll 4
    for (long long r = tid; r < a.N; r += T) {
        v += static_cast<double>(__ldcg(a.loss + r));
        if (a.mean) c += a.labels == nullptr || a.labels[r] != a.ignore;
    }
    sum[tid] = v;
    cnt[tid] = c;
    __syncthreads();
    if (tid < 32) {
        for (int i = tid + 32; i < T; i += 32) v += sum[i], c += cnt[i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            v += __shfl_xor_sync(0xffffffffu, v, o);
            c += __shfl_xor_sync(0xffffffffu, c, o);
        }
        if (tid == 0) a.out[0] = static_cast<float>(a.mean ? v / static_cast<double>(c > 0 ? c : 1) : v);
    }
}

// One row a cluster.
template <bool GRAD, bool CAP>
__global__ void __launch_bounds__(kDsMaxThreads + 32, 3) distill_kernel(const DsArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    __shared__ DsShared sh;
    let_next();
    const int T = a.threads, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool teaches = tid >= T;  // the last warp
    const uint32_t rank = ds_rank(), cluster = 1u << a.log_cluster;
    const long long row = blockIdx.x >> a.log_cluster;
    const long long c0 = static_cast<long long>(rank) * a.slice;
    const int n = static_cast<int>(max(0LL, min(static_cast<long long>(a.slice), a.V - c0)));  // this block's logits
    const int nfull = n >> 3, ntail = n & 7;
    const int part = (nfull + T * kDsParts - 1) / (T * kDsParts);  // a thread's vectors of a part
    uint4* slice = reinterpret_cast<uint4*>(raw);
    const __nv_bfloat16* z = a.z + row * a.ld + c0;
    if (!teaches) {
        const uint32_t sbase = static_cast<uint32_t>(__cvta_generic_to_shared(slice));
#pragma unroll
        for (int g = 0; g < kDsParts; ++g) {
            for (int i = 0; i < part; ++i) {
                const int j = tid + (g * part + i) * T;
                if (j < nfull)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sbase + 16u * j), "l"(z + 8 * j)
                                 : "memory");
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    }
    ds_cluster_arrive();
    const bool ignored = a.labels != nullptr && a.labels[row] == a.ignore;  // the same for the whole cluster
    const bool wants_loss = rank == 0 && a.loss != nullptr;
    __nv_bfloat16* dz = GRAD ? a.dz + row * a.ld + c0 : nullptr;
    bool zeros = ignored;
    if (ignored) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        wait_prior();
        ds_cluster_wait();
        if (wants_loss && tid == 0) a.loss[row] = 0.0f;
    } else {
        DsTeacher t{};
        t.tp = reinterpret_cast<float*>(raw + static_cast<size_t>(a.slice) * 2);
        t.tl = t.tp + a.Kp;
        t.tx = t.tl + a.Kp;
        t.tc = reinterpret_cast<int*>(t.tx + a.Kp);
        float m = CAP ? -1.0f : kDsLowest, s = 0.0f, xt = 0.0f;
        if (teaches) {
            ds_teacher<CAP>(a, sh, t, row, wants_loss);
        } else {
            // V need not be a multiple of 8, nor the row padded: the logits
            // behind the last whole vector go to one thread each
            if (tid < ntail) {
                const __nv_bfloat16 zt = z[8 * nfull + tid];
                reinterpret_cast<__nv_bfloat16*>(slice)[8 * nfull + tid] = zt;
                xt = ds_arg<CAP>(a, a.flip ? -__bfloat162float(zt) : __bfloat162float(zt));
                m = fmaxf(m, xt);
                s = ds_rel<CAP>(xt, m, a.k);
            }
            // The slice's maximum and sum.  A batch's maximum comes first, so
            // that the running sum is rescaled at most once a batch.
#pragma unroll
            for (int g = 0; g < kDsParts; ++g) {
                if (g == 0) asm volatile("cp.async.wait_group 3;" ::: "memory");
                if (g == 1) asm volatile("cp.async.wait_group 2;" ::: "memory");
                if (g == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
                if (g == 3) asm volatile("cp.async.wait_group 0;" ::: "memory");
                const int stop = min(nfull, tid + (g + 1) * part * T);  // of this part
                for (int j0 = tid + g * part * T; j0 < stop; j0 += kDsBatch * T) {
                    uint4 v[kDsBatch];
                    uint32_t m2 = 0xFF7FFF7Fu;  // two of bf16's lowest
#pragma unroll
                    for (int b = 0; b < kDsBatch; ++b) {
                        if (j0 + b * T >= stop) break;
                        v[b] = ds_signed(a, slice[j0 + b * T]);
                        ds_max(m2, v[b]);
                    }
                    const float xb = ds_arg<CAP>(a, fmaxf(__uint_as_float(m2 << 16), __uint_as_float(m2 & 0xFFFF0000u)));
                    if (xb > m) {
                        s *= ds_shift<CAP>(m, xb, a.k);
                        m = xb;
                    }
                    s += ds_far<CAP>(m, a.k) ? ds_batch_sum<CAP, true>(a, v, j0, stop, m)
                                             : ds_batch_sum<CAP, false>(a, v, j0, stop, m);
                }
            }
        }
        float M = ds_warp_max(m);
        s = ds_warp_sum(s * ds_shift<CAP>(m, M, a.k));
        if (lane == 0) sh.warp[warp] = make_float2(M, s);
        __syncthreads();
        ds_cluster_wait();  // every block of the cluster runs: its shared memory may be written
        if (warp == 0) {
            const float2 w = lane <= T / 32 ? sh.warp[lane] : make_float2(CAP ? -1.0f : kDsLowest, 0.0f);
            M = ds_warp_max(w.x);
            s = ds_warp_sum(w.y * ds_shift<CAP>(w.x, M, a.k));
            if (lane < static_cast<int>(cluster)) {
                uint32_t to;
                const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(&sh.all[rank]));
                asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(mine), "r"(lane));
                asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(M), "f"(s) : "memory");
            }
            __syncwarp();
        }
        ds_cluster_arrive();
        ds_cluster_wait();
        m = sh.all[0].x;
        for (uint32_t r = 1; r < cluster; ++r) m = fmaxf(m, sh.all[r].x);
        s = 0.0f;
        for (uint32_t r = 0; r < cluster; ++r) s += sh.all[r].y * ds_shift<CAP>(sh.all[r].x, m, a.k);

        wait_prior();  // the factor may come from the kernel before
        const bool live = sh.live != 0, far = ds_far<CAP>(m, a.k);
        zeros = !live;
        if (teaches) {
            if (wants_loss) {
                const float log_s = logf(s), inv_psum = sh.inv_psum;
                constexpr float kLn2 = 0.6931471805599453f;
                float sum = 0.0f;
                for (int i = lane; i < a.K; i += 32) {
                    const float p = t.tp[i] * inv_psum;
                    const float x = far ? (t.tx[i] - m) * a.k : fmaf(t.tx[i], a.k, -__fmul_rn(m, a.k));
                    if (p != 0.0f) sum += p * ((t.tl[i] - t.log_psum) - (x * kLn2 - log_s));
                }
                sum = ds_warp_sum(sum);
                if (lane == 0)
                    a.loss[row] = t.bad ? __int_as_float(0x7fc00000) : (live ? a.T * a.T * sum : 0.0f);
            }
            if (t.bad && rank == 0 && lane == 0) atomicExch(a.status, -1);
        }
        if (GRAD && live) {
            float g = a.T * (a.flip ? -a.scale : a.scale);
            if (a.dloss != nullptr) g *= a.dloss[row * a.dloss_stride];
            if (a.factor != nullptr) g *= a.factor[1];
            if (!teaches) {
                if (far)
                    ds_grad<CAP, true>(a, slice, reinterpret_cast<uint4*>(dz), nfull, m, g / s);
                else
                    ds_grad<CAP, false>(a, slice, reinterpret_cast<uint4*>(dz), nfull, m, g / s);
            }
            const auto one = [&](float x, float p) {
                const float d = (ds_rel<CAP>(x, m, a.k) / s - p) * g;
                return __float2bfloat16(CAP ? -4.0f * d * fmaf(x, x, x) : d);
            };
            if (tid < ntail) dz[8 * nfull + tid] = one(xt, 0.0f);
            __syncthreads();  // the teacher's elements are written a second time
            const float inv_psum = sh.inv_psum;
            for (int i = tid; i < a.K; i += T + 32) {
                const int c = t.tc[i];
                const long long at = c - c0;
                if (c < 0 || at < 0 || at >= n) continue;
                bool first = true;  // the first entry of an id writes for all of them
                float p = 0.0f;
                for (int o = 0; o < a.Kp; o += 4) {
                    const int4 q = *reinterpret_cast<const int4*>(t.tc + o);
                    if (q.x != c && q.y != c && q.z != c && q.w != c) continue;
                    const int is[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (is[e] == c) {
                            first = first && o + e >= i;
                            p += t.tp[o + e] * inv_psum;
                        }
                }
                if (!first) continue;
                const float zc = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(slice)[at]);
                dz[at] = one(ds_arg<CAP>(a, a.flip ? -zc : zc), p);
            }
        }
    }
    if (GRAD && zeros) {
        for (int j = tid; j < nfull; j += T + 32) reinterpret_cast<uint4*>(dz)[j] = make_uint4(0u, 0u, 0u, 0u);
        if (tid < ntail) dz[8 * nfull + tid] = __float2bfloat16(0.0f);
    }
    if (a.out == nullptr || rank != 0) return;
    __syncthreads();  // this row's loss is written
    if (tid == 0) {
        __threadfence();
        sh.last = atomicAdd(a.counter, 1u) == static_cast<uint32_t>(a.N - 1);
    }
    __syncthreads();
    if (sh.last) ds_reduce(a, reinterpret_cast<double*>(raw));
}

// out[1] = d out[0] / d loss of a row that takes part: 1 / (rows whose label
// is not ignore_index) for the mean, else 1; and the counter of rows done.
constexpr int kDsCountThreads = 1024;
__global__ void __launch_bounds__(kDsCountThreads) distill_count_kernel(const long long* labels, long long N,
                                                                        long long ignore, int mean, float* out,
                                                                        uint32_t* counter) {
    let_next();
    __shared__ int cnt[kDsCountThreads / 32];
    int c = 0;
    if (mean)
        for (long long r = threadIdx.x; r < N; r += kDsCountThreads) c += labels == nullptr || labels[r] != ignore;
    c = __reduce_add_sync(0xffffffffu, c);
    if ((threadIdx.x & 31) == 0) cnt[threadIdx.x >> 5] = c;
    __syncthreads();
    if (threadIdx.x == 0) {
        long long all = 0;
        for (int w = 0; w < kDsCountThreads / 32; ++w) all += cnt[w];
        out[1] = mean ? static_cast<float>(1.0 / static_cast<double>(all > 0 ? all : 1)) : 1.0f;
        *counter = 0u;
    }
}

}  // namespace step
}  // namespace lmlp
