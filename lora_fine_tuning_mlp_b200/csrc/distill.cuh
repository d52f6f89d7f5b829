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
// resident slice: 2 bytes a logit in, 2 out, nothing else.
//
// Clusters stay and take row after row, about three blocks to a multiprocessor
// so that one's exchange falls into another's arithmetic.  Every thread copies
// the 16-byte vectors that it later reads (cp.async), so the loads need no
// barrier: it takes them up in four parts as they arrive, and asks for the next
// row's part as soon as it has used this row's for the last time.  A warp of
// its own takes the teacher's softmax and the loss, and corrects the gradient
// at the teacher's entries when the others are through with the row and on
// their way into the next.  Exponents are in base 2
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

constexpr int kDsMaxThreads = 256, kDsMinThreads = 64;  // that work on the slice; a warp for the teacher on top
constexpr int kDsMaxCluster = 8;
constexpr int kDsMaxK = 1024;
constexpr int kDsParts = 4;   // of a thread's vectors, waited for one after the other
constexpr int kDsBatch = 4;   // vectors taken up together
constexpr int kDsEntryBytes = 32;  // of shared memory for a teacher's entry, two rows' in turn; 4 for each place of the table of ids
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
    float scale, cap;     // s, cap or 0
    float sign;           // of s: the largest exponent is that of the largest sign * z
    float k;              // base-2 exponent of a unit of z: s log2(e) / T; of a unit of -r: 2 cap log2(e) / T
    float cap2;           // 2 s / cap * log2(e)
    float* loss;          // may be null
    float* out;           // the reduced loss, or null
    uint32_t* counter;    // clusters done, zero before the launch (with out)
    int mean;
    int log_table;        // places of the table of a row's ids: at least 2 K
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

// Maxima m are kept as sign * z (as -r with softcapping), so that more is more
// whatever the sign of k; |k| m is their exponent.
template <bool CAP>
__device__ __forceinline__ float ds_exponent(const DsArgs& a, float m) {
    return __fmul_rn(m, fabsf(a.k));
}
// Whether it is out of the range in which x k - fl(|k| m) is formed by one fma.
template <bool CAP>
__device__ __forceinline__ bool ds_far(const DsArgs& a, float m) {
    return !CAP && !(fabsf(ds_exponent<CAP>(a, m)) < 1.0e30f);
}
// A term of a sum that is relative to m.
template <bool CAP>
__device__ __forceinline__ float ds_rel(const DsArgs& a, float x, float m) {
    return ds_far<CAP>(a, m) ? ds_ex2((x - a.sign * m) * a.k) : ds_ex2(fmaf(x, a.k, -ds_exponent<CAP>(a, m)));
}
// What turns a sum relative to m into one relative to M >= m: 2 to the
// difference of their exponents, both rounded (1 where m = M).
template <bool CAP>
__device__ __forceinline__ float ds_shift(const DsArgs& a, float m, float M) {
    return ds_far<CAP>(a, M) ? ds_ex2((m - M) * fabsf(a.k))
                             : ds_ex2(ds_exponent<CAP>(a, m) - ds_exponent<CAP>(a, M));
}

constexpr int kDsMaxWarps = kDsMaxThreads / 32;
struct DsShared {
    // (max, sum) of every warp of the cluster, written by all its blocks; the
    // next row's go to the other half, so that a block may still read this one's
    float2 all[2][kDsMaxCluster * kDsMaxWarps];
    int live[2];  // the teacher has an entry that counts in this row
    int last;     // this block reduces the rows' losses
};

// The teacher's entries of a row, in one warp's hands: ids to tc, exp((a -
// max) / T) to tp, its exponent to tl, and to tx what the student's exponents
// are taken of at the ids of this block's slice, for the loss (`all`) at every
// id.
struct DsTeacher {
    float *tp, *tl, *tx;
    int *tc, *table;
    float inv_psum, log_psum;
    bool bad, live, twice;  // twice: an id stands more than once
};

template <bool CAP>
__device__ __forceinline__ void ds_teacher(const DsArgs& a, DsTeacher& t, long long row, long long c0, int n, bool all) {
    const int lane = threadIdx.x & 31, places = 1 << a.log_table;
    for (int i = lane; i < places; i += 32) t.table[i] = -1;
    __syncwarp();
    float amax = -3.4028234663852886e38f;  // fp32's lowest, which a teacher's mask may hold
    bool any = false, bad = false, twice = false;
#pragma unroll 2
    for (int i = lane; i < a.K; i += 32) {
        const long long at = row * a.K + i;
        const long long id = a.ids_i64 ? static_cast<const long long*>(a.ids)[at] : static_cast<const int*>(a.ids)[at];
        const float v = a.values_f32 ? static_cast<const float*>(a.values)[at]
                                     : __bfloat162float(static_cast<const __nv_bfloat16*>(a.values)[at]);
        const bool in = id >= 0 && id < a.V;
        bad = bad || id < -1 || id >= a.V;
        t.tc[i] = in ? static_cast<int>(id) : -1;
        t.tl[i] = v;
        if (in) {
            amax = fmaxf(amax, v);
            any = any || !(v == -INFINITY);
            if (all || (id >= c0 && id < c0 + n)) {
                const float z = __bfloat162float(a.z[row * a.ld + id]);
                t.tx[i] = CAP ? -1.0f / (1.0f + expf(2.0f * (a.scale / a.cap * z))) : z;
            }
            // at most K ids for at least 2 K places: a free one is found
            const int c = static_cast<int>(id);
            int at_table = static_cast<int>((static_cast<uint32_t>(c) * 2654435769u) >> (32 - a.log_table));
            for (int tries = 0; tries < places; ++tries) {
                const int seen = atomicCAS(t.table + at_table, -1, c);
                twice = twice || seen == c;
                if (seen == -1 || seen == c) break;
                at_table = (at_table + 1) & (places - 1);
            }
        }
    }
    amax = ds_warp_max(amax);
    float psum = 0.0f;
    for (int i = lane; i < a.K; i += 32) {
        const float l = (t.tl[i] - amax) * a.inv_T, e = t.tc[i] >= 0 ? expf(l) : 0.0f;
        t.tl[i] = l;
        t.tp[i] = e;
        psum += e;
    }
    psum = ds_warp_sum(psum);
    t.log_psum = logf(psum);
    t.inv_psum = 1.0f / psum;
    t.bad = __any_sync(0xffffffffu, bad);
    t.live = __any_sync(0xffffffffu, any);
    t.twice = __any_sync(0xffffffffu, twice);
    __syncwarp();
}

// The largest sign * z of the first `count` of a batch's vectors.
__device__ __forceinline__ float ds_batch_max(const DsArgs& a, const uint4 (&v)[kDsBatch], int count) {
    uint32_t m2;
    if (a.sign > 0.0f) {
        m2 = 0xFF7FFF7Fu;  // two of bf16's lowest
#pragma unroll
        for (int b = 0; b < kDsBatch; ++b) {
            if (b >= count) break;
            const uint32_t w[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) asm("max.bf16x2 %0, %0, %1;" : "+r"(m2) : "r"(w[i]));
        }
        return fmaxf(__uint_as_float(m2 << 16), __uint_as_float(m2 & 0xFFFF0000u));
    }
    m2 = 0x7F7F7F7Fu;  // two of its largest
#pragma unroll
    for (int b = 0; b < kDsBatch; ++b) {
        if (b >= count) break;
        const uint32_t w[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("min.bf16x2 %0, %0, %1;" : "+r"(m2) : "r"(w[i]));
    }
    return -fminf(__uint_as_float(m2 << 16), __uint_as_float(m2 & 0xFFFF0000u));
}

// The exponentials of the first `count` of a batch's vectors added up,
// relative to m.
template <bool CAP, bool FAR>
__device__ __forceinline__ float ds_batch_sum(const DsArgs& a, const uint4 (&v)[kDsBatch], int count, float m) {
    const float c = FAR ? a.sign * m : -ds_exponent<CAP>(a, m);
    float s = 0.0f;
#pragma unroll
    for (int b = 0; b < kDsBatch; ++b) {
        if (b >= count) break;
        float x[8];
        ds_args8<CAP>(a, v[b], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = ds_ex2(FAR ? (x[e] - c) * a.k : fmaf(x[e], a.k, c));
        s += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
    }
    return s;
}

// A batch taken into the running (m, s).  Its maximum comes first, so that the
// sum is rescaled at most once a batch.
template <bool CAP>
__device__ __forceinline__ void ds_take(const DsArgs& a, const uint4 (&v)[kDsBatch], int count, float& m, float& s) {
    float mb = ds_batch_max(a, v, count);
    if (CAP) mb = ds_arg<CAP>(a, a.sign * mb);
    if (mb > m) {
        s *= ds_shift<CAP>(a, m, mb);
        m = mb;
    }
    s += ds_far<CAP>(a, m) ? ds_batch_sum<CAP, true>(a, v, count, m) : ds_batch_sum<CAP, false>(a, v, count, m);
}

// The gradient of a vector, the teacher's part left out: gs 2^(x k - |k| m)
// dt/dz.  Where gs is positive it goes into the exponent: the result is off by
// 2^-24 of that exponent, far below its rounding to bf16.
template <bool CAP, bool PLAIN>
__device__ __forceinline__ uint4 ds_grad8(const DsArgs& a, const uint4& v, float m, float c, float gs) {
    float x[8];
    ds_args8<CAP>(a, v, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float y = PLAIN ? ds_rel<CAP>(a, x[e], m) * gs : ds_ex2(fmaf(x[e], a.k, c));
        x[e] = CAP ? y * fmaf(-x[e], x[e], -x[e]) : y;  // r (1 - r) = -x^2 - x
    }
    return round8(x);
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

// Waits for part g of the row at hand.  Behind it in the queue are the row's
// other parts and, without a gradient, those of the next row asked for since:
// three in all.
template <bool GRAD>
__device__ __forceinline__ void ds_wait_part(int g) {
    if (!GRAD || g == 0) asm volatile("cp.async.wait_group 3;" ::: "memory");
    if (GRAD && g == 1) asm volatile("cp.async.wait_group 2;" ::: "memory");
    if (GRAD && g == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    if (GRAD && g == 3) asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <bool GRAD, bool CAP, int T>
__global__ void __launch_bounds__(T + 32, T == kDsMaxThreads ? 3 : 8) distill_kernel(const DsArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    __shared__ DsShared sh;
    let_next();
    constexpr int W = T / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool teaches = tid >= T;  // the last warp
    const uint32_t rank = ds_rank(), cluster = 1u << a.log_cluster;
    const long long stride = gridDim.x >> a.log_cluster;
    const long long c0 = static_cast<long long>(rank) * a.slice;
    const int n = static_cast<int>(max(0LL, min(static_cast<long long>(a.slice), a.V - c0)));  // this block's logits
    const int nfull = n >> 3, ntail = n & 7;
    const int part = (nfull + T * kDsParts - 1) / (T * kDsParts);  // a thread's vectors of a part
    uint4* slice = reinterpret_cast<uint4*>(raw);
    const uint32_t sbase = static_cast<uint32_t>(__cvta_generic_to_shared(slice));
    const bool wants_loss = rank == 0 && a.loss != nullptr;
    const auto ignored = [&](long long row) { return a.labels != nullptr && row < a.N && a.labels[row] == a.ignore; };

    // Part g of a row into this thread's places of the slice.
    const auto ask = [&](int g, long long row) {
        if (row < a.N) {
            const __nv_bfloat16* z = a.z + row * a.ld + c0;
            const int stop = min(nfull, (g + 1) * part * T);
#pragma unroll 4
            for (int j = tid + g * part * T; j < stop; j += T)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sbase + 16u * j), "l"(z + 8 * j)
                             : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const auto write_zeros = [&](long long row) {
        __nv_bfloat16* dz = a.dz + row * a.ld + c0;
        for (int j = tid; j < nfull; j += T) __stcs(reinterpret_cast<uint4*>(dz) + j, make_uint4(0u, 0u, 0u, 0u));
        if (tid < ntail) dz[8 * nfull + tid] = __float2bfloat16(0.0f);
    };
    // The first row from `row` on that takes part; those passed over are
    // finished here (labels are the same for the whole cluster).
    const auto taking_part = [&](long long row, bool skip) {
        while (skip) {
            if (GRAD && !teaches) write_zeros(row);
            if (wants_loss && tid == T) a.loss[row] = 0.0f;
            row += stride;
            skip = ignored(row);
        }
        return row;
    };

    long long row = blockIdx.x >> a.log_cluster;
    row = taking_part(row, ignored(row));
    if (!teaches) {
#pragma unroll
        for (int g = 0; g < kDsParts; ++g) ask(g, row);
    }
    ds_cluster_arrive();
    // The teacher's warp prepares a row while the others write the gradient of
    // the one before it.
    DsTeacher t{}, ahead{};
    const auto prepare = [&](DsTeacher& d, int turn, long long row) {
        float* at = reinterpret_cast<float*>(raw + static_cast<size_t>(a.slice) * 2);
        d.table = reinterpret_cast<int*>(at + 8 * a.K);
        at += turn * 4 * a.K;
        d.tp = at;
        d.tl = at + a.K;
        d.tx = at + 2 * a.K;
        d.tc = reinterpret_cast<int*>(at + 3 * a.K);
        ds_teacher<CAP>(a, d, row, c0, n, wants_loss);
        if (lane == 0) sh.live[turn] = d.live;
        __syncwarp();
    };
    if (teaches && row < a.N) prepare(t, 0, row);
    const float up = a.T * a.scale;
    ds_cluster_wait();  // every block of the cluster runs: its shared memory may be written
    for (int turn = 0; row < a.N; turn ^= 1) {
        const bool skip = ignored(row + stride);
        long long next = GRAD ? 0 : taking_part(row + stride, skip);
        float m = CAP ? -1.0f : kDsLowest, s = 0.0f, xt = 0.0f;
        if (!teaches) {
            // V need not be a multiple of 8, nor the row padded: the logits
            // behind the last whole vector go to one thread each
            if (tid < ntail) {
                const float zt = __bfloat162float(a.z[row * a.ld + c0 + 8 * nfull + tid]);
                xt = ds_arg<CAP>(a, zt);
                m = fmaxf(m, CAP ? xt : a.sign * xt);
                s = ds_rel<CAP>(a, xt, m);
            }
            // the slice's maximum and sum
#pragma unroll
            for (int g = 0; g < kDsParts; ++g) {
                ds_wait_part<GRAD>(g);
                const int stop = min(nfull, (g + 1) * part * T);
#pragma unroll 1
                for (int j0 = tid + g * part * T; j0 < stop; j0 += kDsBatch * T) {
                    uint4 v[kDsBatch];
                    if (j0 + (kDsBatch - 1) * T < stop) {
#pragma unroll
                        for (int b = 0; b < kDsBatch; ++b) v[b] = slice[j0 + b * T];
                        ds_take<CAP>(a, v, kDsBatch, m, s);
                    } else {
                        for (int j = j0; j < stop; j += T) {
                            v[0] = slice[j];
                            ds_take<CAP>(a, v, 1, m, s);
                        }
                    }
                }
                if (!GRAD) ask(g, next);
            }
            const float M = ds_warp_max(m);
            s = ds_warp_sum(s * ds_shift<CAP>(a, m, M));
            if (lane < static_cast<int>(cluster)) {
                uint32_t to;
                const uint32_t mine =
                    static_cast<uint32_t>(__cvta_generic_to_shared(&sh.all[turn][rank * W + warp]));
                asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(mine), "r"(lane));
                asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(M), "f"(s) : "memory");
            }
        }
        __syncwarp();
        ds_cluster_arrive();
        ds_cluster_wait();
        {
            // each warp merges all warps' sums, in the same order everywhere
            const int entries = static_cast<int>(cluster) * W;
            const float2 none = make_float2(CAP ? -1.0f : kDsLowest, 0.0f);
            const float2 w0 = lane < entries ? sh.all[turn][lane] : none;
            const float2 w1 = lane + 32 < entries ? sh.all[turn][lane + 32] : none;
            m = ds_warp_max(fmaxf(w0.x, w1.x));
            s = ds_warp_sum(w0.y * ds_shift<CAP>(a, w0.x, m) + w1.y * ds_shift<CAP>(a, w1.x, m));
        }
        const bool live = sh.live[turn] != 0, far = ds_far<CAP>(a, m);
        wait_prior();  // the factor may come from the kernel before
        float g = up;
        if (GRAD) {
            next = taking_part(row + stride, skip);
            if (a.dloss != nullptr) g *= a.dloss[row * a.dloss_stride];
            if (a.factor != nullptr) g *= a.factor[1];
        }
        __nv_bfloat16* dz = GRAD ? a.dz + row * a.ld + c0 : nullptr;
        const auto one = [&](float x, float p) {
            const float d = (ds_rel<CAP>(a, x, m) / s - p) * g;
            return __float2bfloat16(CAP ? 4.0f * d * fmaf(-x, x, -x) : d);
        };
        if (!teaches) {
            if (GRAD) {
                if (tid < ntail) dz[8 * nfull + tid] = live ? one(xt, 0.0f) : __float2bfloat16(0.0f);
                uint4* o = reinterpret_cast<uint4*>(dz);
                const float gs = (CAP ? 4.0f : 1.0f) * (g / s);
                const float c = log2f(gs) - ds_exponent<CAP>(a, m);
#pragma unroll 1
                for (int q = 0; q < kDsParts; ++q) {
                    const int from = tid + q * part * T, stop = min(nfull, (q + 1) * part * T);
                    if (live && !far && gs > 0.0f) {
#pragma unroll 4
                        for (int j = from; j < stop; j += T) __stcs(o + j, ds_grad8<CAP, false>(a, slice[j], m, c, gs));
                    } else {
                        for (int j = from; j < stop; j += T)
                            __stcs(o + j, live ? ds_grad8<CAP, true>(a, slice[j], m, c, gs) : make_uint4(0u, 0u, 0u, 0u));
                    }
                    ask(q, next);
                }
                __syncwarp();
                asm volatile("bar.arrive 1, %0;" ::"r"(T + 32) : "memory");
            }
        } else {
            if (wants_loss) {
                const float log_s = logf(s);
                constexpr float kLn2 = 0.6931471805599453f;
                float sum = 0.0f;
                for (int i = lane; i < a.K; i += 32) {
                    const float p = t.tp[i] * t.inv_psum;
                    if (p == 0.0f || t.tc[i] < 0) continue;
                    const float x = far ? (t.tx[i] - a.sign * m) * a.k
                                        : fmaf(t.tx[i], a.k, -ds_exponent<CAP>(a, m));
                    sum += p * ((t.tl[i] - t.log_psum) - (x * kLn2 - log_s));
                }
                sum = ds_warp_sum(sum);
                if (lane == 0)
                    a.loss[row] = t.bad ? __int_as_float(0x7fc00000) : (live ? a.T * a.T * sum : 0.0f);
            }
            if (t.bad && rank == 0 && lane == 0) atomicExch(a.status, -1);
            if (next < a.N) prepare(ahead, turn ^ 1, next);
            if (GRAD) {
                asm volatile("bar.sync 1, %0;" ::"r"(T + 32) : "memory");  // the row's gradient is written
                for (int i = lane; live && i < a.K; i += 32) {
                    const int c = t.tc[i];
                    const long long at = c - c0;
                    if (c < 0 || at < 0 || at >= n) continue;
                    float p = t.tp[i];
                    if (t.twice) {  // the first entry of an id writes for all of them
                        bool first = true;
                        p = 0.0f;
                        for (int o = 0; o < a.K; ++o) {
                            if (t.tc[o] != c) continue;
                            first = first && o >= i;
                            p += t.tp[o];
                        }
                        if (!first) continue;
                    }
                    dz[at] = one(t.tx[i], p * t.inv_psum);
                }
                __syncwarp();
            }
            t = ahead;
        }
        row = next;
    }
    wait_prior();  // in every block, whatever rows it had
    if (a.out == nullptr || rank != 0) return;
    __syncthreads();  // this block's losses are written
    if (tid == 0) {
        __threadfence();
        sh.last = atomicAdd(a.counter, 1u) == static_cast<uint32_t>(stride - 1);
    }
    __syncthreads();
    if (sh.last) ds_reduce(a, reinterpret_cast<double*>(raw));
}

// out[1] = d out[0] / d loss of a row that takes part: 1 / (rows whose label
// is not ignore_index) for the mean, else 1; and the counter of clusters done.
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
