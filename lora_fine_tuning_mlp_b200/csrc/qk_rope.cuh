// Norms of queries and keys for each head with the position rotation in the
// same pass, forward and backward (include/lora_qk_rope.h).
//
//   y = R(p) (x rstd(x) gain);   dn = R(p)^T dy,  dgain = sum dn xh,
//   dx = rstd (dn gain - xh mean(dn gain xh)),  xh = x rstd
//
// Bound by HBM: 4 bytes an element forward, 6 backward (4 without the norm),
// and a head's arithmetic stays in registers.  A thread holds two 16-byte
// vectors of a head, chosen so that both partners of every pair it turns are
// its own: vectors j and j + rot/16 for pairs (i, i + rot/2), vectors 2j and
// 2j + 1 for neighbouring pairs; behind `rot`, neighbouring vectors.  D/16
// threads (rounded up to a power of two, `group`) make up a head, and a warp
// works on 32/group heads at a time, several times over, so that a token's
// angles and the gains are read once for all of them and every load of a thread
// is in flight before the first is used.
//
// On a B200, 4096 tokens of 32 + 8 heads of 128: forward 21 us, backward 35 and
// 7 for the gains' sums, 57 together, bound by waits for their loads (39 and 44 %
// of the warps' time, then 16 % of fixed latency) at the few warps that their
// registers allow; 32768 tokens of 32 + 4 heads of 64
// without the norm: 51 us a pass, 5.9 TB/s.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "f32x2.cuh"
#include "vec8.cuh"

namespace lmlp {
namespace step {

constexpr int kQkThreads = 128;
constexpr int kQkWarps = kQkThreads / 32;
// heads of a thread in the forward; without the norm fewer, in blocks of 64 registers a thread
constexpr int kQkUnroll = 4, kQkRopeUnroll = 2;
constexpr int kQkBwdBlocksPerSm = 3;  // of the backward through the norm, by its registers

struct QkView {
    uint4* p;
    long long sb, ss, sh;  // in 16-byte vectors
};

// Quotients of numbers below 2^31 by a divisor that is known at the launch, by
// a multiplication (Granlund and Montgomery, 1994): with 2^(l - 1) < d <= 2^l
// and m = floor(2^32 (2^l - d) / d) + 1, n / d = (mulhi(m, n) + n) >> l.
struct QkDivisor {
    uint32_t d, m;
    int l;
    __device__ __forceinline__ uint32_t quotient(uint32_t n) const { return (__umulhi(m, n) + n) >> l; }
};

struct QkArgs {
    QkView in[2], out[2];  // queries, keys (backward: the gradients of the forward's results, and of its inputs)
    QkView x[2];           // backward with the norm: the forward's inputs
    const uint4* gain[2];
    const float *cos, *sin;
    const long long* pos;
    long long pos_stride;
    long long T, P;
    QkDivisor seq;        // S
    QkDivisor by[2];      // a token's units of queries, of keys; flat: its heads
    QkDivisor per_token;  // its units
    int flat;
    int H[2];
    int D, nslot, nrot, half;  // nslot = D/16 threads of a head do work, nrot = rot/16 of them turn pairs
    int log_group;
    float eps, inv_d;
    float turn;       // +1, or -1 to turn back
    int* status;
    uint32_t units[2];  // of queries, of keys
    int blocks_q;     // backward: blocks [0, blocks_q) take queries, the others keys
    float* part;      // backward: [blocks][D] sums of dn xh, or null
};

// Vectors of the head that thread `slot` holds.
template <bool INTER>
__device__ __forceinline__ void qk_vectors(const QkArgs& a, int slot, int& v0, int& v1) {
    if (!INTER && slot < a.nrot) {
        v0 = slot;
        v1 = slot + a.nrot;
    } else {
        v0 = 2 * slot;
        v1 = 2 * slot + 1;
    }
}

// The values of two vectors as the two sides of the pairs that a thread turns,
// two pairs to a packed fp32 pair: sides of pair 2i and 2i + 1 in x[i] and y[i].
struct QkPairs {
    uint64_t x[4], y[4];
};

__device__ __forceinline__ uint32_t qk_low(uint32_t w) { return w << 16; }
__device__ __forceinline__ uint32_t qk_high(uint32_t w) { return w & 0xFFFF0000u; }

template <bool INTER>
__device__ __forceinline__ QkPairs qk_widen(const uint4& v0, const uint4& v1) {
    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    QkPairs r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (INTER) {
            r.x[i] = f2_pack(qk_low(w[2 * i]), qk_low(w[2 * i + 1]));
            r.y[i] = f2_pack(qk_high(w[2 * i]), qk_high(w[2 * i + 1]));
        } else {
            r.x[i] = f2_pack(qk_low(w[i]), qk_high(w[i]));
            r.y[i] = f2_pack(qk_low(w[4 + i]), qk_high(w[4 + i]));
        }
    }
    return r;
}

__device__ __forceinline__ uint32_t qk_bf16x2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool INTER>
__device__ __forceinline__ void qk_round(const QkPairs& r, uint4& v0, uint4& v1) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x0, x1, y0, y1;
        f2_unpack(r.x[i], x0, x1);
        f2_unpack(r.y[i], y0, y1);
        w[INTER ? 2 * i : i] = INTER ? qk_bf16x2(x0, y0) : qk_bf16x2(x0, x1);
        w[INTER ? 2 * i + 1 : 4 + i] = INTER ? qk_bf16x2(x1, y1) : qk_bf16x2(y0, y1);
    }
    v0 = make_uint4(w[0], w[1], w[2], w[3]);
    v1 = make_uint4(w[4], w[5], w[6], w[7]);
}

// The 8 angles of `slot` at position p: cosines in x and sines in y.
struct QkAngles {
    uint64_t c[4], s[4];
};
__device__ __forceinline__ QkAngles qk_angles(const QkArgs& a, long long p, int slot) {
    const float4* cp = reinterpret_cast<const float4*>(a.cos + p * a.half) + 2 * slot;
    const float4* sp = reinterpret_cast<const float4*>(a.sin + p * a.half) + 2 * slot;
    const uint64_t turn = f2_packf(a.turn, a.turn);
    QkAngles r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 c = __ldg(cp + i), s = __ldg(sp + i);
        r.c[2 * i] = f2_packf(c.x, c.y), r.c[2 * i + 1] = f2_packf(c.z, c.w);
        r.s[2 * i] = f2_mul(f2_packf(s.x, s.y), turn), r.s[2 * i + 1] = f2_mul(f2_packf(s.z, s.w), turn);
    }
    return r;
}

__device__ __forceinline__ void qk_rotate(QkPairs& f, const QkAngles& a) {
    const uint64_t minus = f2_packf(-1.0f, -1.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t x = f.x[i], y = f.y[i];
        f.x[i] = f2_fma(x, a.c[i], f2_mul(f2_mul(y, minus), a.s[i]));
        f.y[i] = f2_fma(y, a.c[i], f2_mul(x, a.s[i]));
    }
}

__device__ __forceinline__ float qk_lanes(uint64_t v) {
    float lo, hi;
    f2_unpack(v, lo, hi);
    return lo + hi;
}
// sum of p q over a thread's values
__device__ __forceinline__ float qk_dot(const QkPairs& p, const QkPairs& q) {
    uint64_t v = f2_mul(p.x[0], q.x[0]);
    uint64_t w = f2_mul(p.y[0], q.y[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        v = f2_fma(p.x[i], q.x[i], v);
        w = f2_fma(p.y[i], q.y[i], w);
    }
    return qk_lanes(f2_add(v, w));
}

// Sums over the lanes of a group, the same for each of them.
template <int N>
__device__ __forceinline__ void group_sums(float (&v)[N], int group) {
    for (int o = group >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

__device__ __forceinline__ uint4 qk_nan() { return make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u); }

// The token and the head that are row u of a unit for this lane; `in` if there
// is one.  A unit is U * (32 / group) heads of one token, or, where half of that
// and more would be empty (FLAT), of several tokens in a row: then each row has
// angles of its own to read.
template <bool FLAT>
struct QkPlace {
    uint32_t b, s;
    int h;
    bool in;
    __device__ __forceinline__ uint4* head(const QkView& v) const { return v.p + b * v.sb + s * v.ss + h * v.sh; }
    __device__ __forceinline__ long long position(const QkArgs& a) const {
        return a.pos == nullptr ? s : !FLAT || in ? a.pos[b * a.pos_stride + s] : 0;
    }
};
template <bool FLAT, int U>
__device__ __forceinline__ QkPlace<FLAT> qk_place(const QkArgs& a, const QkDivisor& by, int H, uint32_t unit, int u) {
    const uint32_t rows = 32u >> a.log_group, row = (threadIdx.x & 31) >> a.log_group;
    const uint32_t item = FLAT ? (unit * U + u) * rows + row : unit;  // `by`: a token's heads, or its units
    const uint32_t t = by.quotient(item), rest = item - t * by.d;
    QkPlace<FLAT> l;
    l.h = static_cast<int>(FLAT ? rest : (rest * U + u) * rows + row);
    l.in = FLAT ? t < a.T : l.h < H;
    l.b = a.seq.quotient(t);
    l.s = t - l.b * a.seq.d;
    return l;
}

// A warp takes a unit of queries or of keys.  IN_PLACE: results may lie over
// what is read (a thread reads all of a head that it will write, and no other).
template <bool NORM, bool INTER, bool FLAT, bool IN_PLACE>
__global__ void __launch_bounds__(kQkThreads, NORM ? 4 : 8) qk_rope_kernel(const QkArgs a) {
    constexpr int U = NORM ? kQkUnroll : kQkRopeUnroll;
    uint32_t unit = blockIdx.x * kQkWarps + (threadIdx.x >> 5);
    int kind;
    if (FLAT) {
        kind = unit >= a.units[0];
        if (kind) unit -= a.units[0];
        if (unit >= a.units[kind]) return;
    } else {  // a token's queries, then its keys
        const uint32_t t = a.per_token.quotient(unit);
        if (t >= a.T) return;
        unit -= t * a.per_token.d;
        kind = unit >= a.by[0].d;
        unit = kind ? t * a.by[1].d + unit - a.by[0].d : t * a.by[0].d + unit;
    }
    const int lane = threadIdx.x & 31, group = 1 << a.log_group, slot = lane & (group - 1);
    const QkView in = kind ? a.in[1] : a.in[0], out = kind ? a.out[1] : a.out[0];
    const QkDivisor by = kind ? a.by[1] : a.by[0];
    const int H = kind ? a.H[1] : a.H[0];
    const bool works = slot < a.nslot;
    int v0, v1;
    qk_vectors<INTER>(a, slot, v0, v1);
    const int rows = 32 >> a.log_group;
    const QkPlace<FLAT> l0 = qk_place<FLAT, U>(a, by, H, unit, 0);
    uint4 v[U][2];
    long long p[FLAT ? U : 1];
    const uint4* ip = l0.head(in);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        QkPlace<FLAT> l = l0;
        if (FLAT && u > 0) l = qk_place<FLAT, U>(a, by, H, unit, u), ip = l.head(in);
        v[u][0] = v[u][1] = make_uint4(0u, 0u, 0u, 0u);
        if (works && (FLAT ? l.in : l0.h + u * rows < H)) {
            v[u][0] = load_once<IN_PLACE>(ip + v0);
            v[u][1] = load_once<IN_PLACE>(ip + v1);
        }
        if (!FLAT) ip += rows * in.sh;
        if (FLAT || u == 0) p[FLAT ? u : 0] = l.position(a);
    }
    QkPairs g{};
    if (NORM && works) {
        const uint4* gp = kind ? a.gain[1] : a.gain[0];
        g = qk_widen<INTER>(__ldg(gp + v0), __ldg(gp + v1));
    }
    bool bad = false, turns = false;
    QkAngles ang{};
    const auto angles = [&](long long at) {
        bad = at < 0 || at >= a.P;
        if (bad && slot == 0) atomicMin(a.status, kStatusBad);
        turns = slot < a.nrot && !bad;
        if (turns) ang = qk_angles(a, at, slot);
    };
    angles(p[0]);
    float ss[U];
    if (NORM) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const QkPairs f = qk_widen<INTER>(v[u][0], v[u][1]);
            ss[u] = qk_dot(f, f);
        }
        group_sums(ss, group);
    }
    uint4* op = l0.head(out);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        QkPlace<FLAT> l = l0;
        if (FLAT && u > 0) {
            angles(p[u]);
            l = qk_place<FLAT, U>(a, by, H, unit, u);
            op = l.head(out);
        }
        QkPairs f = qk_widen<INTER>(v[u][0], v[u][1]);
        if (NORM) {
            const float r = rsqrtf(ss[u] * a.inv_d + a.eps);
            const uint64_t rr = f2_packf(r, r);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f.x[i] = f2_mul(f2_mul(f.x[i], rr), g.x[i]);
                f.y[i] = f2_mul(f2_mul(f.y[i], rr), g.y[i]);
            }
        }
        if (turns) qk_rotate(f, ang);
        if (works && (FLAT ? l.in : l0.h + u * rows < H)) {
            uint4 o0, o1;
            qk_round<INTER>(f, o0, o1);
            __stcs(op + v0, bad ? qk_nan() : o0);
            __stcs(op + v1, bad ? qk_nan() : o1);
        }
        if (!FLAT) op += rows * out.sh;
    }
}

// Backward through the norm.  With e = dn gain (dn = R(p)^T dy) and r the
// reciprocal root, dx = r e - x r^3 mean(e x): both sums of a head are taken
// over x itself and joined in one go.  A warp takes every gridDim-th unit of
// its kind, so that it can add up dn x r over all of them in registers; a
// block's sums go to `part`, which qk_gain_kernel adds up in block order.
constexpr int kQkBwdUnroll = 2;

template <bool INTER, bool FLAT, bool IN_PLACE>
__global__ void __launch_bounds__(kQkThreads, kQkBwdBlocksPerSm) qk_rope_bwd_kernel(const QkArgs a) {
    __shared__ float sums[kQkWarps][512];
    const int kind = static_cast<int>(blockIdx.x) >= a.blocks_q;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = 1 << a.log_group, slot = lane & (group - 1);
    const uint32_t nblocks = kind ? gridDim.x - a.blocks_q : a.blocks_q;
    const uint32_t first = (kind ? blockIdx.x - a.blocks_q : blockIdx.x) * kQkWarps + warp;
    const QkView dy = kind ? a.in[1] : a.in[0], dx = kind ? a.out[1] : a.out[0], x = kind ? a.x[1] : a.x[0];
    const int H = kind ? a.H[1] : a.H[0];
    const QkDivisor by = kind ? a.by[1] : a.by[0];
    constexpr int U = kQkBwdUnroll;
    const bool works = slot < a.nslot;
    int v0, v1;
    qk_vectors<INTER>(a, slot, v0, v1);
    QkPairs g{}, acc{};
    if (works) {
        const uint4* gp = kind ? a.gain[1] : a.gain[0];
        g = qk_widen<INTER>(__ldg(gp + v0), __ldg(gp + v1));
    }
    let_next();
    const uint32_t units = kind ? a.units[1] : a.units[0];
    for (uint32_t unit = first; unit < units; unit += nblocks * kQkWarps) {
        uint4 vy[U][2], vx[U][2];
        long long p[FLAT ? U : 1];
        QkPlace<FLAT> l[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            l[u] = qk_place<FLAT, U>(a, by, H, unit, u);
            vy[u][0] = vy[u][1] = vx[u][0] = vx[u][1] = make_uint4(0u, 0u, 0u, 0u);
            if (works && l[u].in) {
                const uint4 *yp = l[u].head(dy), *xp = l[u].head(x);
                vy[u][0] = load_once<IN_PLACE>(yp + v0);
                vy[u][1] = load_once<IN_PLACE>(yp + v1);
                vx[u][0] = load_once<IN_PLACE>(xp + v0);
                vx[u][1] = load_once<IN_PLACE>(xp + v1);
            }
            if (FLAT || u == 0) p[FLAT ? u : 0] = l[u].position(a);
        }
        bool bad[U];
        QkPairs d[U];
        float both[2 * U];
        {
            QkAngles ang{};
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (FLAT || u == 0) {
                    bad[u] = p[u] < 0 || p[u] >= a.P;
                    if (bad[u] && slot == 0) atomicMin(a.status, kStatusBad);
                    if (slot < a.nrot && !bad[u]) ang = qk_angles(a, p[u], slot);
                } else {
                    bad[u] = bad[0];
                }
                const QkPairs f = qk_widen<INTER>(vx[u][0], vx[u][1]);
                d[u] = qk_widen<INTER>(vy[u][0], vy[u][1]);
                if (slot < a.nrot && !bad[u]) qk_rotate(d[u], ang);
                both[2 * u] = qk_dot(f, f);
                QkPairs e;
#pragma unroll
                for (int i = 0; i < 4; ++i) e.x[i] = f2_mul(d[u].x[i], g.x[i]), e.y[i] = f2_mul(d[u].y[i], g.y[i]);
                both[2 * u + 1] = qk_dot(e, f);
            }
        }
        group_sums(both, group);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!works || !l[u].in) continue;
            const float r = rsqrtf(both[2 * u] * a.inv_d + a.eps);
            // of x r: its products stay in range where x^2 does
            const float m = -(both[2 * u + 1] * r * a.inv_d);
            const uint64_t rr = f2_packf(r, r), mm = f2_packf(m, m);
            const QkPairs f = qk_widen<INTER>(vx[u][0], vx[u][1]);
            QkPairs o;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint64_t hx = f2_mul(f.x[i], rr), hy = f2_mul(f.y[i], rr);
                if (!bad[u]) {
                    acc.x[i] = f2_fma(d[u].x[i], hx, acc.x[i]);
                    acc.y[i] = f2_fma(d[u].y[i], hy, acc.y[i]);
                }
                o.x[i] = f2_mul(rr, f2_fma(hx, mm, f2_mul(d[u].x[i], g.x[i])));
                o.y[i] = f2_mul(rr, f2_fma(hy, mm, f2_mul(d[u].y[i], g.y[i])));
            }
            uint4 o0, o1, *op = l[u].head(dx);
            qk_round<INTER>(o, o0, o1);
            __stcs(op + v0, bad[u] ? qk_nan() : o0);
            __stcs(op + v1, bad[u] ? qk_nan() : o1);
        }
    }
    if (a.part == nullptr) return;
    // a value's place among the 16 of its thread's two vectors
    float sum[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int x0 = INTER ? 4 * i : 2 * i, step = INTER ? 2 : 1, y0 = INTER ? 4 * i + 1 : 8 + 2 * i;
        f2_unpack(acc.x[i], sum[x0], sum[x0 + step]);
        f2_unpack(acc.y[i], sum[y0], sum[y0 + step]);
    }
    for (int o = group; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
    if (lane < a.nslot) {
#pragma unroll
        for (int i = 0; i < 16; ++i) sums[warp][8 * (i < 8 ? v0 : v1) + (i & 7)] = sum[i];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.D; e += kQkThreads) {
        float v = sums[0][e];
        for (int w = 1; w < kQkWarps; ++w) v += sums[w][e];
        a.part[static_cast<long long>(blockIdx.x) * a.D + e] = v;
    }
}

// dgain[e] = the blocks' sums in a fixed order: 32 columns a block, 32 threads
// each adding every 32nd block's, then those.  blockIdx.y: queries, keys.
__global__ void __launch_bounds__(1024) qk_gain_kernel(const float* part, int D, int blocks_q, int blocks,
                                                       float* dq_gain, float* dk_gain) {
    __shared__ float s[32][33];
    wait_prior();
    const int e = blockIdx.x * 32 + threadIdx.x;
    const int from = blockIdx.y ? blocks_q : 0, to = blockIdx.y ? blocks : blocks_q;
    float v = 0.0f;
    if (e < D)
        for (int b = from + threadIdx.y; b < to; b += 32) v += part[static_cast<long long>(b) * D + e];
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y == 0 && e < D) {
        for (int k = 1; k < 32; ++k) v += s[k][threadIdx.x];
        (blockIdx.y ? dk_gain : dq_gain)[e] = v;
    }
}

}  // namespace step
}  // namespace lmlp
