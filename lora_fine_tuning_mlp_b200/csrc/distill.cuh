// Distillation from a teacher's top logits, loss and gradient
// (include/lora_distill.h).
//
//   x = t(z) / T,  q = softmax(x),  p = softmax(a / T) over the K entries
//   loss = T^2 sum p_i (log p_i - log q_ci),   dz_j = g T (q_j - p_j) dt/dz
//
// The gradient needs the row's softmax sum before its first element, so a
// kernel that streams rows from HBM has to read them twice.  Here a row stays
// on the chip between its two passes: a cluster of 1, 2, 4 or 8 blocks holds
// it in shared memory as the bf16 it came in, a slice each, and the gradient is
// formed from the resident slice: 2 bytes a logit in, 2 out, nothing else.
//
// The clusters stay and take row after row as one stream of chunks (B vectors
// for each thread) through a ring of shared memory.  In step k a thread adds
// chunk k into its row's sum, turns chunk k - lag into gradient, and asks
// (cp.async) for chunk k + kDsAhead in the place that this sets free.  It only
// ever touches vectors of its own, so the ring needs no barrier.  The lag is a
// row and one or two chunks: when a row's second pass begins, the sums that
// its warps stored in all blocks of the cluster have arrived.  Three
// more warps take the teacher's softmax and the loss, a row each in turn, and
// correct the gradient at the teacher's entries once the row is written.
//
// One exponential a logit and pass is what the special-function unit can
// deliver in about the time that HBM takes, so the passes do little else.  In
// particular they look for no maximum: sums are taken relative to a reference
// m that stays from row to row (0 at first), 2^(z k - E) with one fma, E = fl(m
// k).  A row whose sum leaves the middle of fp32's range (its largest logit far
// from m, infinities, a vocabulary masked whole) is summed again, after a
// search for its maximum, which is the reference from then on.  E's rounding is
// in the row's sum as in its terms and leaves no trace in the softmax, as long
// as it is small itself: from |E| = 2^20 on (logits of 10^6, a temperature of
// 10^-6) exponents are formed of the difference z - m, and the reference is not
// kept for other rows.  Either way an exponent is off by 2^-23 of its distance
// from the reference, which is fp32's own precision of it.
//
// With softcapping, t = cap tanh(s z / cap) = cap - 2 cap r with r = 1 / (1 + e),
// e = 2^(cap2 z): exponents are taken of -r, dt/dz = 4 s e r^2 has no
// cancellation where tanh saturates on either side, and four logits share one
// reciprocal.  t / T is off by 2^-22 cap / T so, however small t is: fp32 holds
// r, near 1/2, to 2^-24.  That is a choice for speed up to cap / T = 128 (3e-5;
// 1024 rows of 256000 take 415 us so, 746 us with tanhf).  Above it t itself is
// what exponents are taken of, to fp32's precision of t, and rows are else
// treated as without softcapping.
//
// On a B200: 4096 rows of 128256 logits, loss and gradient, 455 us (4.6 TB/s; the
// same stream of chunks merely copied takes 390, the exponentials' unit 248); the
// loss of 2047 rows alone 104 to 110 us (4.9 TB/s); 1024 rows of 256000 with
// softcapping 415 us.  There the unit has 4.5 operations a logit in the two
// passes, 280 us if all multiprocessors did nothing else: clusters of four leave
// 16 of 148 idle (312 us), and on the others it is 73 % busy, the rest being
// waits for results of fixed latency and for its queue.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "f32x2.cuh"
#include "ptx.cuh"
#include "vec8.cuh"

namespace lmlp {
namespace step {

constexpr int kDsAhead = 3;     // chunks asked for ahead of their first use
constexpr int kDsMaxK = 1024;
constexpr int kDsDepth = 8;     // rows under way (see DsShared)
constexpr int kDsTeachers = 3;  // warps that take the teacher's part, a row each in turn
constexpr int kDsTimeout = -7;  // LORA_MLP_ERR_DEVICE_TIMEOUT
constexpr int kDsEntryBytes = 16;  // of shared memory for a teacher's entry, and 4 for each place of the table of ids
// How exponents are formed: of z, of -r, of t (the kernel's parameter CAP).
constexpr int kDsNoCap = 0, kDsCap = 1, kDsWideCap = 2;
constexpr float kDsWide = 128.0f;  // cap / T above which t is formed
constexpr float kDsLowest = -3.3895313892515355e38f;  // bf16's lowest finite value

struct DsArgs {
    const __nv_bfloat16* z;
    __nv_bfloat16* dz;
    long long ld, V, N;
    int K;
    int slice;  // logits of a block: a multiple of 8
    int log_cluster;
    int chunks;  // of a slice
    int chunk;   // vectors of a chunk
    int lag;     // chunks between a chunk's two uses
    int slots;   // chunks of the ring
    long long wait_limit;  // SM cycles that a wait may take before the kernel gives up
    int force_timeout;     // test hook: no wait is ever over
    const void *values, *ids;
    int values_f32, ids_i64;
    const long long* labels;  // may be null
    long long ignore;
    float inv_T, T;
    float scale, cap;     // s, cap or 0
    int form;             // kDsNoCap, kDsCap, kDsWideCap (the host's; the kernel has it as a parameter)
    float sign;           // of s: the largest exponent is that of the largest sign * z
    float k;              // base-2 exponent of a unit of z: s log2(e) / T; of -r: 2 cap log2(e) / T; of t: log2(e) / T
    float cap2;           // 2 s / cap * log2(e)
    float ratio, ratio2;  // their product is s / cap: two, as it may be below fp32's normal numbers
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

// What exponents are taken of: z, -r or t (see above).  2^(cap2 z) is held to
// 2^30, where tanh is 1 in fp32 already (and dt/dz below 2^-28 s), so that a
// product of four denominators stays in range; min keeps a NaN.
__device__ __forceinline__ float ds_cap_exp(float power) {
    float e;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(e) : "f"(power), "f"(30.0f));
    return ds_ex2(e);
}
// s z / cap, t and dt/dz / s = 1 / cosh^2(s z / cap).
__device__ __forceinline__ float ds_wide_arg(const DsArgs& a, float z) { return z * a.ratio * a.ratio2; }
__device__ __forceinline__ float ds_wide(const DsArgs& a, float u) { return a.cap * tanhf(u); }
__device__ __forceinline__ float ds_wide_slope(float u) {
    constexpr float kLog2e = 1.4426950408889634f;
    const float e = ds_ex2(-2.0f * kLog2e * fabsf(u)), r = ds_rcp(1.0f + e);
    return 4.0f * e * r * r;
}
template <int CAP>
__device__ __forceinline__ float ds_arg(const DsArgs& a, float z) {
    if (CAP == kDsWideCap) return ds_wide(a, ds_wide_arg(a, z));
    return CAP ? -ds_rcp(1.0f + ds_cap_exp(a.cap2 * z)) : z;
}
// The same of single logits, and dt/dz / s, by CUDA's own functions.
template <int CAP>
__device__ __forceinline__ float ds_arg_one(const DsArgs& a, float z) {
    return CAP == kDsCap ? -1.0f / (1.0f + expf(2.0f * ds_wide_arg(a, z))) : ds_arg<CAP>(a, z);
}
template <int CAP>
__device__ __forceinline__ float ds_slope_one(const DsArgs& a, float z) {
    if (!CAP) return 1.0f;
    const float e = expf(-2.0f * fabsf(ds_wide_arg(a, z)));
    return 4.0f * e / ((1.0f + e) * (1.0f + e));
}
// Of eight, as packed fp32 pairs: neighbours, or of -r elements (0, 2), (1, 3),
// (4, 6), (5, 7); and what dt/dz takes of each, e of -r, the slope of t.
__device__ __forceinline__ uint64_t ds_pair(float v) { return f2_packf(v, v); }
template <int CAP>
__device__ __forceinline__ void ds_args8(const DsArgs& a, const uint4& v, uint64_t (&x)[4], uint64_t (&e)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int h = 0; h < 4; h += 2) {
        if constexpr (CAP != kDsCap) {
            x[h] = f2_pack(w[h] << 16, w[h] & 0xFFFF0000u);
            x[h + 1] = f2_pack(w[h + 1] << 16, w[h + 1] & 0xFFFF0000u);
            if constexpr (CAP == kDsWideCap) {
#pragma unroll
                for (int i = h; i < h + 2; ++i) {
                    float lo, hi;
                    f2_unpack(x[i], lo, hi);
                    lo = ds_wide_arg(a, lo), hi = ds_wide_arg(a, hi);
                    x[i] = f2_packf(ds_wide(a, lo), ds_wide(a, hi));
                    e[i] = f2_packf(ds_wide_slope(lo), ds_wide_slope(hi));
                }
            }
        } else {
            x[h] = f2_pack(w[h] << 16, w[h + 1] << 16);
            x[h + 1] = f2_pack(w[h] & 0xFFFF0000u, w[h + 1] & 0xFFFF0000u);
            uint64_t d[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float lo, hi;
                f2_unpack(f2_mul(x[h + i], ds_pair(a.cap2)), lo, hi);
                e[h + i] = f2_packf(ds_cap_exp(lo), ds_cap_exp(hi));
                d[i] = f2_add(e[h + i], ds_pair(1.0f));
            }
            float d01, d23;
            f2_unpack(f2_mul(d[0], d[1]), d01, d23);
            const uint64_t n = f2_mul(ds_pair(-ds_rcp(d01 * d23)), f2_packf(d23, d01));
            x[h] = f2_mul(n, d[1]), x[h + 1] = f2_mul(n, d[0]);
        }
    }
}
template <int CAP>
__device__ __forceinline__ uint4 ds_round8(const uint64_t (&x)[4]) {
    float f[8];
#pragma unroll
    for (int h = 0; h < 4; h += 2) {
        f2_unpack(x[h], f[2 * h], f[2 * h + (CAP == kDsCap ? 2 : 1)]);
        f2_unpack(x[h + 1], f[2 * h + (CAP == kDsCap ? 1 : 2)], f[2 * h + 3]);
    }
    return round8(f);
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

// References m are kept as sign * z (as -r or t with softcapping), so that more is
// more whatever the sign of k; |k| m is their exponent.
__device__ __forceinline__ float ds_exponent(const DsArgs& a, float m) { return __fmul_rn(m, fabsf(a.k)); }
// Whether it is so large that its rounding alone (2^-24 of it) shifts the sums
// of a row by a part that counts: at 2^20 a sixteenth of a power of two, at
// 2^32 out of fp32.
constexpr float kDsFar = 0x1p20f;
__device__ __forceinline__ bool ds_far(const DsArgs& a, float m) { return !(fabsf(ds_exponent(a, m)) < kDsFar); }
// m as what exponents are taken of.
template <int CAP>
__device__ __forceinline__ float ds_origin(const DsArgs& a, float m) {
    return CAP ? m : a.sign * m;
}
// The exponent of a term of a sum that is relative to m.
template <int CAP>
__device__ __forceinline__ float ds_power(const DsArgs& a, float x, float m) {
    return ds_far(a, m) ? (x - ds_origin<CAP>(a, m)) * a.k : fmaf(x, a.k, -ds_exponent(a, m));
}
template <int CAP>
__device__ __forceinline__ float ds_rel(const DsArgs& a, float x, float m) {
    return ds_ex2(ds_power<CAP>(a, x, m));
}

// The warps of a cluster that work on its slices tell one another a number
// each, in an 8-byte store to every block's shared memory together with a tag,
// which is how the readers know it has come.  Sums of row i (i = 0, 1, ... of
// the cluster's) have the tag i + 1 and buffer i mod kDsDepth, which is free
// again in time: the lag is at most chunks + 1, or chunks + 2 where a slice has
// two chunks or more, so a warp that sends row x's sum has received row x -
// 3's, and the warps that sent those had received row x - 6's.  Exchanges for
// rows that are summed again are counted by themselves and use two buffers in
// turn: a warp that sends number f has received f - 1, sent by warps that had
// received f - 2.
//
// A row's teacher sets `ready` when it has prepared the row, having finished
// with row i - 3; block 0's sets `read` in all blocks.  The first warp tells it
// the row's reference and sum in `told`.
struct DsShared {
    float reference[kDsDepth];  // that row i's sums are relative to
    int ready[kDsDepth];  // 2 (i + 1), + 1 where the teacher has an entry that counts
    int read[kDsDepth];   // i + 1 when block 0's teacher reads the logits of row i no more
    float told[kDsDepth][2];
    int told_row[kDsDepth];       // i + 1
    uint64_t done[kDsTeachers];   // mbarriers: a row's gradient is written
    int gave_up;                  // a wait ran out
    int last;                     // this block reduces the rows' losses
};

__device__ __forceinline__ uint32_t ds_smem(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ uint32_t ds_remote(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
template <class V>
__device__ __forceinline__ V ds_look(const V* p) {
    return *static_cast<const volatile V*>(p);
}

// Polls until `here` holds in every lane of the warp, for a limited time; false
// where it ran out here or for another of the block's warps.
template <class F>
__device__ __forceinline__ bool ds_wait(const DsArgs& a, DsShared& sh, F here) {
    if (!a.force_timeout && __all_sync(0xffffffffu, here())) return true;
    const long long begin = clock64();
    for (;;) {
        __nanosleep(300);  // polls without a pause take issue slots from the warps that work: 3 % of the kernel's time
        if (!a.force_timeout && __all_sync(0xffffffffu, here())) return true;
        const bool stop = ds_look(&sh.gave_up) != 0 || clock64() - begin > a.wait_limit;
        if (__any_sync(0xffffffffu, stop)) {
            if (ds_look(&sh.gave_up) == 0) atomicMin(a.status, kDsTimeout);
            *static_cast<volatile int*>(&sh.gave_up) = 1;
            return false;
        }
    }
}

// Sends this warp's v as its cell (`mine`) of the buffer at `cell` to every block.
__device__ __forceinline__ void ds_send(const uint64_t* cell, int mine, int cluster, uint32_t tag, float v) {
    const int lane = threadIdx.x & 31;
    __threadfence_block();  // the row's reference before the sum that its readers wait for
    if (lane < cluster) {
        const uint32_t to = ds_remote(ds_smem(cell + mine), static_cast<uint32_t>(lane));
        asm volatile("st.volatile.shared::cluster.u64 [%0], %1;" ::"r"(to),
                     "l"(static_cast<uint64_t>(tag) << 32 | __float_as_uint(v))
                     : "memory");
    }
    __syncwarp();
}
// The sum, or the largest, of a buffer's cells, the same bits for every warp;
// false where the wait ran out.
template <bool MAX>
__device__ __forceinline__ bool ds_receive(const DsArgs& a, DsShared& sh, const uint64_t* cell, int cells, uint32_t tag,
                                           float& v) {
    const int lane = threadIdx.x & 31;
    if (!ds_wait(a, sh, [&] {
            bool here = true;
            for (int e = lane; e < cells; e += 32) here = here && static_cast<uint32_t>(ds_look(cell + e) >> 32) == tag;
            return here;
        }))
        return false;
    v = MAX ? -INFINITY : 0.0f;
    for (int e = lane; e < cells; e += 32) {
        const float c = __uint_as_float(static_cast<uint32_t>(ds_look(cell + e)));
        v = MAX ? fmaxf(v, c) : v + c;
    }
    v = MAX ? ds_warp_max(v) : ds_warp_sum(v);
    return true;
}

// The teacher's entries of a row, in one warp's hands: ids to tc, exp((a -
// max) / T) to tp, its exponent to tl, and to tx the student's logits at the ids
// of this block's slice, for the loss (`all`) at every id.
struct DsTeacher {
    float *tp, *tl, *tx;
    int *tc, *table;
    float inv_psum, log_psum;
    bool bad, live, twice;  // twice: an id stands more than once
};

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
            if (all || (id >= c0 && id < c0 + n)) t.tx[i] = __bfloat162float(a.z[row * a.ld + id]);
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

// 2^(x k + c) of eight, added to acc two by two.
__device__ __forceinline__ void ds_add8(const DsArgs& a, const uint64_t (&x)[4], float c, uint64_t& acc) {
    const uint64_t kk = ds_pair(a.k), cc = ds_pair(c);
    uint64_t e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        f2_unpack(f2_fma(x[i], kk, cc), lo, hi);
        e[i] = f2_packf(ds_ex2(lo), ds_ex2(hi));
    }
    acc = f2_add(acc, f2_add(f2_add(e[0], e[1]), f2_add(e[2], e[3])));
}

// The gradient of a vector, the teacher's part left out: g / s 2^(x k - |k| m)
// dt/dz, with the row's sum s.  Where g is positive and c = log2(g / s) - |k| m
// is below kDsFast, g / s goes into the exponent: c's rounding (2^-25 of it, at
// most 2^-17) and that of the logarithms put the result off by 10^-5 of its
// value, a four-hundredth of its rounding to bf16.
constexpr float kDsFast = 256.0f;
template <int CAP>
__device__ __forceinline__ uint64_t ds_slope2(uint64_t x, uint64_t e) {
    return CAP == kDsCap ? f2_mul(e, f2_mul(x, x)) : e;
}
template <int CAP>
__device__ __forceinline__ uint4 ds_grad8(const DsArgs& a, const uint4& v, float c) {
    uint64_t x[4], e[4];
    ds_args8<CAP>(a, v, x, e);
    const uint64_t kk = ds_pair(a.k), cc = ds_pair(c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        f2_unpack(f2_fma(x[i], kk, cc), lo, hi);
        uint64_t y = f2_packf(ds_ex2(lo), ds_ex2(hi));
        if (CAP) y = f2_mul(y, ds_slope2<CAP>(x[i], e[i]));
        x[i] = y;
    }
    return ds_round8<CAP>(x);
}
// The same for any g and m: exponents as the row's sum has them, then l =
// log2(|g| / s) is added, so that probabilities far below the row's largest are
// not lost between the reference and the sum; g's sign last.  4096 rows of
// 128256 take 518 us so, with logits around 400, against 455; where the
// difference from m is formed they are summed three times, 870 us.
struct DsForm {
    float m0, c;  // an exponent is (x + m0) k + c: m0 = -0 or c = 0 drop out (see ds_power)
};
template <int CAP>
__device__ __forceinline__ DsForm ds_form(const DsArgs& a, float m) {
    return ds_far(a, m) ? DsForm{-ds_origin<CAP>(a, m), 0.0f} : DsForm{-0.0f, -ds_exponent(a, m)};
}
__device__ __forceinline__ uint64_t ds_powers(const DsArgs& a, uint64_t x, const DsForm& f) {
    return f2_fma(f2_add(x, ds_pair(f.m0)), ds_pair(a.k), ds_pair(f.c));
}
template <int CAP>
__device__ __forceinline__ uint4 ds_grad8_any(const DsArgs& a, const uint4& v, const DsForm& f, float l, uint32_t sign) {
    uint64_t x[4], e[4];
    ds_args8<CAP>(a, v, x, e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        f2_unpack(f2_add(ds_powers(a, x[i], f), ds_pair(l)), lo, hi);
        uint64_t y = f2_packf(ds_ex2(lo), ds_ex2(hi));
        if (CAP) y = f2_mul(y, ds_slope2<CAP>(x[i], e[i]));
        x[i] = y;
    }
    const uint4 o = ds_round8<CAP>(x);
    return make_uint4(o.x ^ sign, o.y ^ sign, o.z ^ sign, o.w ^ sign);
}

// This thread's largest sign * z (-r, t) of a slice in global memory, and its
// sum relative to m: for rows whose sum came out too large or too small.
template <int CAP>
__device__ __forceinline__ float ds_reference(const DsArgs& a, float z) {
    return CAP == kDsWideCap ? ds_arg<CAP>(a, z) : a.sign * z;  // (tanhf need not grow with its argument)
}
template <int CAP, int T>
__device__ __noinline__ float ds_slice_max(const DsArgs& a, const __nv_bfloat16* z, int n) {
    float m = kDsLowest;
    const uint4* v = reinterpret_cast<const uint4*>(z);
#pragma unroll 4
    for (int j = threadIdx.x; j < n >> 3; j += T) {
        float f[8];
        widen8(v[j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, ds_reference<CAP>(a, f[i]));
    }
    const int j = (n & ~7) + threadIdx.x;
    if (j < n) m = fmaxf(m, ds_reference<CAP>(a, __bfloat162float(z[j])));
    return CAP == kDsCap ? ds_arg<CAP>(a, a.sign * m) : m;
}
template <int CAP, int T>
__device__ __noinline__ float ds_slice_sum(const DsArgs& a, const __nv_bfloat16* z, int n, float m) {
    uint64_t s = 0u;
    const DsForm form = ds_form<CAP>(a, m);
    const uint4* v = reinterpret_cast<const uint4*>(z);
#pragma unroll 4
    for (int j = threadIdx.x; j < n >> 3; j += T) {
        uint64_t x[4], e[4];
        ds_args8<CAP>(a, v[j], x, e);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lo, hi;
            f2_unpack(ds_powers(a, x[i], form), lo, hi);
            s = f2_add(s, f2_packf(ds_ex2(lo), ds_ex2(hi)));
        }
    }
    float lo, hi;
    f2_unpack(s, lo, hi);
    const int j = (n & ~7) + threadIdx.x;
    return lo + hi + (j < n ? ds_rel<CAP>(a, ds_arg<CAP>(a, __bfloat162float(z[j])), m) : 0.0f);
}
// Whether a row's sum has to be taken again: outside of this range fp32 may
// have lost terms that count (2^-78 at least of a sum's 2^20) or the sum itself.
__device__ __forceinline__ bool ds_lost(float s) { return !(s > 0x1p-60f && s < 0x1p100f); }

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

// T threads work on the slice (and kDsTeachers warps for the teacher), a chunk
// is at most B vectors for each of them.
template <bool GRAD, int CAP, int T, int B>
__global__ void __launch_bounds__(T + 32 * kDsTeachers, T >= 512 ? 1 : T >= 256 ? 2 : 6) distill_kernel(const DsArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    __shared__ DsShared sh;
    let_next();
    constexpr int W = T / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool teaches = tid >= T;
    const int rank = static_cast<int>(ds_rank()), cluster = 1 << a.log_cluster;
    const long long first = blockIdx.x >> a.log_cluster;
    const int stride = static_cast<int>(gridDim.x >> a.log_cluster);
    const int rows = static_cast<int>((a.N - 1 - first) / stride + 1);  // of this cluster: not more clusters than rows
    const long long c0 = static_cast<long long>(rank) * a.slice;
    const int n = static_cast<int>(max(0LL, min(static_cast<long long>(a.slice), a.V - c0)));  // this block's logits
    const int nfull = n >> 3, ntail = n & 7;
    // every chunk has `chunk` vectors but the slice's last, also in the cluster's
    // last slice: it is shorter by 64 logits at most, and chunks are longer where
    // there are several
    const int chunk = a.chunk, end = a.chunks - 1, rest = nfull - end * chunk;
    uint4* ring = reinterpret_cast<uint4*>(raw);
    float* entries = reinterpret_cast<float*>(ring + a.slots * a.chunk);
    const int teacher_floats = (a.K + 3) / 4 * 16 + (1 << a.log_table);
    const int cells = cluster * W;
    uint64_t* const sums = reinterpret_cast<uint64_t*>(entries + kDsTeachers * teacher_floats);  // [kDsDepth][cells]
    uint64_t* const sums_again = sums + kDsDepth * cells;                                       // [2][cells]
    const bool wants_loss = rank == 0 && a.loss != nullptr;
    const auto ignored = [&](long long row) { return a.labels != nullptr && row < a.N && a.labels[row] == a.ignore; };

    for (int e = tid; e < (kDsDepth + 2) * cells; e += blockDim.x) sums[e] = 0u;
    if (tid < kDsDepth) sh.ready[tid] = sh.read[tid] = sh.told_row[tid] = 0;
    if (tid == 0) {
        for (int i = 0; i < kDsTeachers; ++i) mbar_init(ds_smem(&sh.done[i]), W);
        fence_mbar_init();
        sh.gave_up = 0;
    }
    __syncthreads();
    ds_cluster_arrive();
    const auto upstream = [&](long long row) {
        float g = a.T * a.scale;
        if (a.dloss != nullptr) g *= a.dloss[row * a.dloss_stride];
        if (a.factor != nullptr) g *= a.factor[1];
        return g;
    };
    const auto element = [&](float z, float p, float m, float log_s, float g) {
        const float q = ds_ex2(ds_power<CAP>(a, ds_arg_one<CAP>(a, z), m) - log_s);
        return __float2bfloat16((q - p) * g * ds_slope_one<CAP>(a, z));
    };
    if (!teaches) {
        // Three places in the stream: where chunks are asked for, summed, and
        // turned into gradient; each a chunk of its row and a place in the ring.
        const uint4* const ring_end = ring + a.slots * a.chunk;
        uint4* ask_at = ring + tid;
        const uint4 *sum_at = ring + tid, *out_at = ring + tid;
        int ask_c = 0, sum_c = 0, out_c = 0, ask_i = 0, sum_i = 0, out_i = 0;
        const long long row_step = static_cast<long long>(stride) * a.ld;
        const uint4* ask_z = reinterpret_cast<const uint4*>(a.z + first * a.ld + c0) + tid;
        const long long ask_step = row_step / 8 - static_cast<long long>(a.chunks) * chunk;  // from a row's end to the next
        const __nv_bfloat16* sum_z = a.z + first * a.ld + c0;
        uint4* out_z = nullptr;
        long long out_row = first;
        // whether a row is ignored: bit b of `skips` for row ask_i - b
        uint32_t skips = ignored(first) ? 1u : 0u;
        bool skip_next = ignored(first + stride);
        const auto step = [&](auto& at) {
            at += chunk;
            if (at >= ring_end) at -= a.slots * a.chunk;
        };
        const auto ask = [&]() {
            if (ask_i < rows) {
                const int len = (skips & 1u) ? 0 : ask_c == end ? rest : chunk;
                const uint32_t to = ds_smem(ask_at);
#pragma unroll
                for (int b = 0; b < B; ++b)
                    if (tid + b * T < len)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 16u * b * T), "l"(ask_z + b * T)
                                     : "memory");
                step(ask_at);
                ask_z += chunk;
                if (ask_c++ == end) {
                    ask_c = 0;
                    ++ask_i;
                    ask_z += ask_step;
                    skips = skips << 1 | (skip_next ? 1u : 0u);
                    skip_next = ignored(first + static_cast<long long>(ask_i + 1) * stride);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int k = 0; k < kDsAhead; ++k) ask();
        ds_cluster_wait();  // every block's shared memory can be stored to
        float m = CAP == kDsCap ? -0.5f : 0.0f;  // the reference of sums
        uint32_t again = 0u;           // exchanges for rows summed again
        float c = 0.0f;                // - the exponent of the one that the row being summed has
        uint64_t acc = 0u;
        float om = 0.0f, os = 0.0f, olog = 0.0f, og = 0.0f, oc = 0.0f;  // of the row being turned into gradient
        bool live = false, fast = false, skip = false;
        float up = 0.0f, dloss = a.dloss != nullptr ? a.dloss[first * a.dloss_stride] : 1.0f;  // factors of the upstream gradient
        const int steps = rows * a.chunks;
#pragma unroll 1
        for (int k = 0; k < steps + a.lag; ++k) {
            if (k < steps) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kDsAhead - 1) : "memory");
                if (sum_c == 0) {
                    c = -ds_exponent(a, m);
                    acc = 0u;
                    skip = skips >> (ask_i - sum_i) & 1u;
                    if (tid == 0) *static_cast<volatile float*>(&sh.reference[sum_i % kDsDepth]) = m;
                }
                const int len = skip ? 0 : sum_c == end ? rest : chunk;
#pragma unroll
                for (int b = 0; b < B; ++b)
                    if (tid + b * T < len) {
                        uint64_t z[4], e[4];
                        ds_args8<CAP>(a, sum_at[b * T], z, e);
                        ds_add8(a, z, c, acc);
                    }
                step(sum_at);
                if (sum_c++ == end) {
                    float lo, hi;
                    f2_unpack(acc, lo, hi);
                    lo += hi;
                    // V need not be a multiple of 8, nor the row padded: the
                    // logits behind the last whole vector go to one thread each
                    if (!skip && tid < ntail)
                        lo += ds_ex2(fmaf(ds_arg<CAP>(a, __bfloat162float(sum_z[8 * nfull + tid])), a.k, c));
                    // (an ignored row's is 1, so that nobody sums it again)
                    ds_send(sums + (sum_i % kDsDepth) * cells, rank * W + warp, cluster,
                            static_cast<uint32_t>(sum_i) + 1u, skip ? 1.0f : ds_warp_sum(lo));
                    sum_c = 0;
                    ++sum_i;
                    sum_z += row_step;
                }
            }
            if (k >= a.lag) {
                if (out_c == 0) {
                    const int i = out_i;
                    const int buf = i % kDsDepth;
                    // The teacher's part is prepared, and block 0's teacher
                    // reads this row's logits no more: a gradient may be
                    // written over them.
                    if (!ds_wait(a, sh, [&] {
                            return ds_look(&sh.ready[buf]) >> 1 == i + 1 &&
                                   (rank == 0 || ds_look(&sh.read[buf]) == i + 1);
                        }))
                        break;
                    live = (ds_look(&sh.ready[buf]) & 1) != 0;
                    if (!ds_receive<false>(a, sh, sums + buf * cells, cells, static_cast<uint32_t>(i) + 1u, os)) break;
                    om = ds_look(&sh.reference[buf]);
                    if (ds_lost(os)) {
                        const __nv_bfloat16* z = a.z + out_row * a.ld + c0;
                        uint64_t* cell = sums_again + (again++ & 1u) * cells;
                        ds_send(cell, rank * W + warp, cluster, again, ds_warp_max(ds_slice_max<CAP, T>(a, z, n)));
                        if (!ds_receive<true>(a, sh, cell, cells, again, om)) break;
                        cell = sums_again + (again++ & 1u) * cells;
                        ds_send(cell, rank * W + warp, cluster, again, ds_warp_sum(ds_slice_sum<CAP, T>(a, z, n, om)));
                        if (!ds_receive<false>(a, sh, cell, cells, again, os)) break;
                        if (!ds_far(a, om)) m = om;  // the first pass forms no differences
                    }
                    if (tid == 0) {
                        *static_cast<volatile float*>(&sh.told[buf][0]) = om;
                        *static_cast<volatile float*>(&sh.told[buf][1]) = os;
                        __threadfence_block();
                        *static_cast<volatile int*>(&sh.told_row[buf]) = i + 1;
                    }
                    if (GRAD) {
                        if (i == 0) {
                            wait_prior();  // the factor may come from the kernel before
                            up = a.factor != nullptr ? a.T * a.scale * a.factor[1] : a.T * a.scale;
                        }
                        og = up * dloss;
                        // asked for now, used at the next row
                        dloss = a.dloss != nullptr && i + 1 < rows ? a.dloss[(out_row + stride) * a.dloss_stride] : 1.0f;
                        olog = log2f(os);
                        oc = log2f(og) - olog + (CAP == kDsCap ? 2.0f : 0.0f) - ds_exponent(a, om);
                        fast = live && og > 0.0f && fabsf(oc) < kDsFast && !ds_far(a, om);
                        out_z = reinterpret_cast<uint4*>(a.dz + out_row * a.ld + c0) + tid;
                    }
                }
                if (GRAD) {
                    const int len = out_c == end ? rest : chunk;
                    if (fast) {
#pragma unroll
                        for (int b = 0; b < B; ++b)
                            if (tid + b * T < len) __stcs(out_z + b * T, ds_grad8<CAP>(a, out_at[b * T], oc));
                    } else if (live) {
                        const DsForm form = ds_form<CAP>(a, om);
                        const uint32_t sign = og < 0.0f ? 0x80008000u : 0u;
                        const float l = log2f(fabsf(og)) - olog + (CAP == kDsCap ? 2.0f : 0.0f);
#pragma unroll 1
                        for (int b = 0; tid + b * T < len; ++b)
                            __stcs(out_z + b * T, ds_grad8_any<CAP>(a, out_at[b * T], form, l, sign));
                    } else {
#pragma unroll 1
                        for (int b = 0; tid + b * T < len; ++b) __stcs(out_z + b * T, make_uint4(0u, 0u, 0u, 0u));
                    }
                    out_z += chunk;
                    step(out_at);
                }
                if (out_c++ == end) {
                    if (GRAD) {
                        if (tid < ntail) {
                            const long long at = out_row * a.ld + c0 + 8 * nfull + tid;
                            a.dz[at] = live ? element(__bfloat162float(a.z[at]), 0.0f, om, olog, og)
                                            : __float2bfloat16(0.0f);
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(ds_smem(&sh.done[out_i % kDsTeachers]));
                    }
                    out_c = 0;
                    ++out_i;
                    out_row += stride;
                }
            }
            ask();
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else {
        DsTeacher t{};
        t.tp = entries + (warp - W) * teacher_floats;
        t.tl = t.tp + a.K;
        t.tx = t.tl + a.K;
        t.tc = reinterpret_cast<int*>(t.tx + a.K);
        t.table = reinterpret_cast<int*>(t.tp + (a.K + 3) / 4 * 16);
        ds_cluster_wait();
        for (int i = warp - W; i < rows; i += kDsTeachers) {
            const long long row = first + static_cast<long long>(i) * stride;
            const int buf = i % kDsDepth;
            t.live = t.bad = false;
            if (!ignored(row)) ds_teacher(a, t, row, c0, n, wants_loss);
            __threadfence_block();  // what was read of the logits has arrived: it is in tx
            __syncwarp();
            if (lane == 0) *static_cast<volatile int*>(&sh.ready[buf]) = (i + 1) * 2 + t.live;
            if (rank == 0 && lane < cluster)
                asm volatile("st.volatile.shared::cluster.u32 [%0], %1;" ::"r"(
                                 ds_remote(ds_smem(&sh.read[buf]), static_cast<uint32_t>(lane))),
                             "r"(i + 1)
                             : "memory");
            __syncwarp();
            if (!ds_wait(a, sh, [&] { return ds_look(&sh.told_row[buf]) == i + 1; })) break;
            __threadfence_block();
            const float m = ds_look(&sh.told[buf][0]), s = ds_look(&sh.told[buf][1]);
            wait_prior();
            if (wants_loss) {
                const float log_s = logf(s);
                constexpr float kLn2 = 0.6931471805599453f;
                float sum = 0.0f;
                for (int e = lane; t.live && e < a.K; e += 32) {
                    const float p = t.tp[e] * t.inv_psum;
                    if (p == 0.0f || t.tc[e] < 0) continue;
                    const float y = ds_power<CAP>(a, ds_arg_one<CAP>(a, t.tx[e]), m);
                    sum += p * ((t.tl[e] - t.log_psum) - (y * kLn2 - log_s));
                }
                sum = ds_warp_sum(sum);
                if (lane == 0) a.loss[row] = t.bad ? __int_as_float(0x7fc00000) : (t.live ? a.T * (a.T * sum) : 0.0f);
            }
            if (t.bad && rank == 0 && lane == 0) atomicMin(a.status, kStatusBad);
            if (GRAD) {
                const float g = upstream(row), log_s = log2f(s);
                const uint32_t done = ds_smem(&sh.done[warp - W]), parity = static_cast<uint32_t>(i / kDsTeachers) & 1u;
                if (!ds_wait(a, sh, [&] { return mbar_try_wait(done, parity); })) break;
                __nv_bfloat16* dz = a.dz + row * a.ld;
                for (int e = lane; t.live && e < a.K; e += 32) {
                    const int c = t.tc[e];
                    if (c < c0 || c >= c0 + n) continue;
                    float p = t.tp[e];
                    if (t.twice) {  // the first entry of an id writes for all of them
                        bool before = false;
                        p = 0.0f;
                        for (int o = 0; o < a.K; ++o) {
                            if (t.tc[o] != c) continue;
                            before = before || o < e;
                            p += t.tp[o];
                        }
                        if (before) continue;
                    }
                    dz[c] = element(t.tx[e], p * t.inv_psum, m, log_s, g);
                }
                __syncwarp();
            }
        }
    }
    wait_prior();  // in every thread, whatever it did
    __syncthreads();
    ds_cluster_arrive();
    ds_cluster_wait();  // no block leaves while another may still store to it
    if (a.out == nullptr || rank != 0 || sh.gave_up) return;
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
