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
// works on 32/group heads of one token at a time, kQkUnroll times over, so
// that the token's angles and the gains are read once for all of them and
// every load of a thread is in flight before the first is used.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "vec8.cuh"

namespace lmlp {
namespace step {

constexpr int kQkThreads = 128;
constexpr int kQkWarps = kQkThreads / 32;
constexpr int kQkUnroll = 4;

struct QkView {
    uint4* p;
    long long sb, ss, sh;  // in 16-byte vectors
};

struct QkArgs {
    QkView in[2], out[2];  // queries, keys (backward: the gradients of the forward's results, and of its inputs)
    QkView x[2];           // backward with the norm: the forward's inputs
    const uint4* gain[2];
    const float *cos, *sin;
    const long long* pos;
    long long pos_stride;
    long long T, S, P;
    int H[2];
    int D, nslot, nrot, half;  // nslot = D/16 threads of a head do work, nrot = rot/16 of them turn pairs
    int log_group;
    float eps, inv_d;
    float turn;       // +1, or -1 to turn back
    int* status;
    int units[2];     // of a token: ceil(heads / heads of a unit)
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

// The 8 angles of `slot` at position p.
__device__ __forceinline__ void qk_angles(const QkArgs& a, long long p, int slot, float (&c)[8], float (&s)[8]) {
    if (slot < a.nrot) {
        const float4* cp = reinterpret_cast<const float4*>(a.cos + p * a.half) + 2 * slot;
        const float4* sp = reinterpret_cast<const float4*>(a.sin + p * a.half) + 2 * slot;
        const float4 c0 = __ldg(cp), c1 = __ldg(cp + 1), s0 = __ldg(sp), s1 = __ldg(sp + 1);
        c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w, c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
        s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w, s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] *= a.turn;
    }
}

template <bool INTER>
__device__ __forceinline__ void qk_rotate(float (&f)[2][8], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float& x = INTER ? f[i >> 2][2 * (i & 3)] : f[0][i];
        float& y = INTER ? f[i >> 2][2 * (i & 3) + 1] : f[1][i];
        const float a = x, b = y;
        x = a * c[i] - b * s[i];
        y = b * c[i] + a * s[i];
    }
}

// Sum over the lanes of a group, the same for each of them.
__device__ __forceinline__ float group_sum(float v, int group) {
    for (int o = group >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ uint4 qk_nan() { return make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u); }

// A warp's unit: one token and kQkUnroll * (32 / group) heads of its queries
// or of its keys.
template <bool NORM, bool INTER>
__global__ void __launch_bounds__(kQkThreads) qk_rope_kernel(const QkArgs a) {
    const long long unit = static_cast<long long>(blockIdx.x) * kQkWarps + (threadIdx.x >> 5);
    const int per_token = a.units[0] + a.units[1];
    const long long t = unit / per_token;
    if (t >= a.T) return;
    int chunk = static_cast<int>(unit - t * per_token);
    const int kind = chunk >= a.units[0];
    if (kind) chunk -= a.units[0];
    const int lane = threadIdx.x & 31, group = 1 << a.log_group, slot = lane & (group - 1);
    const long long b = t / a.S, s = t - b * a.S;
    const QkView in = kind ? a.in[1] : a.in[0], out = kind ? a.out[1] : a.out[0];
    const int H = kind ? a.H[1] : a.H[0];
    const int rows = 32 >> a.log_group;
    const int h0 = chunk * rows * kQkUnroll + (lane >> a.log_group);
    const bool works = slot < a.nslot;
    int v0, v1;
    qk_vectors<INTER>(a, slot, v0, v1);
    const uint4* ip = in.p + b * in.sb + s * in.ss;
    uint4 v[kQkUnroll][2];
#pragma unroll
    for (int u = 0; u < kQkUnroll; ++u) {
        const int h = h0 + u * rows;
        v[u][0] = v[u][1] = make_uint4(0u, 0u, 0u, 0u);
        if (works && h < H) {
            v[u][0] = load_once(ip + h * in.sh + v0);
            v[u][1] = load_once(ip + h * in.sh + v1);
        }
    }
    float g[2][8];
    if (NORM && works) {
        const uint4* gp = kind ? a.gain[1] : a.gain[0];
        widen8(__ldg(gp + v0), g[0]);
        widen8(__ldg(gp + v1), g[1]);
    }
    const long long p = a.pos != nullptr ? a.pos[b * a.pos_stride + s] : s;
    const bool bad = p < 0 || p >= a.P;
    if (bad && lane == 0) atomicExch(a.status, -1);
    float c[8], sn[8];
    if (works && !bad) qk_angles(a, p, slot, c, sn);
    uint4* op = out.p + b * out.sb + s * out.ss;
#pragma unroll
    for (int u = 0; u < kQkUnroll; ++u) {
        const int h = h0 + u * rows;
        float f[2][8];
        widen8(v[u][0], f[0]);
        widen8(v[u][1], f[1]);
        if (NORM) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(f[0][i], f[0][i], fmaf(f[1][i], f[1][i], ss));
            const float r = 1.0f / sqrtf(group_sum(ss, group) * a.inv_d + a.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[0][i] *= r * g[0][i];
                f[1][i] *= r * g[1][i];
            }
        }
        if (!works || h >= H) continue;
        if (slot < a.nrot) qk_rotate<INTER>(f, c, sn);
        op[h * out.sh + v0] = bad ? qk_nan() : round8(f[0]);
        op[h * out.sh + v1] = bad ? qk_nan() : round8(f[1]);
    }
}

// Backward through the norm.  A warp takes every gridDim-th unit of its kind,
// so that it can add up dn xh over all of them in registers; a block's sums go
// to `part`, which qk_gain_kernel adds up in block order.
constexpr int kQkBwdUnroll = 2;

template <bool INTER>
__global__ void __launch_bounds__(kQkThreads) qk_rope_bwd_kernel(const QkArgs a) {
    __shared__ float sums[kQkWarps][512];
    const int kind = static_cast<int>(blockIdx.x) >= a.blocks_q;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = 1 << a.log_group, slot = lane & (group - 1), rows = 32 >> a.log_group;
    const long long nblocks = kind ? gridDim.x - a.blocks_q : a.blocks_q;
    const long long first = (kind ? blockIdx.x - a.blocks_q : blockIdx.x) * static_cast<long long>(kQkWarps) + warp;
    const QkView dy = kind ? a.in[1] : a.in[0], dx = kind ? a.out[1] : a.out[0], x = kind ? a.x[1] : a.x[0];
    const int H = kind ? a.H[1] : a.H[0], per_token = kind ? a.units[1] : a.units[0];
    const bool works = slot < a.nslot;
    int v0, v1;
    qk_vectors<INTER>(a, slot, v0, v1);
    float g[2][8] = {}, acc[2][8] = {};
    if (works) {
        const uint4* gp = kind ? a.gain[1] : a.gain[0];
        widen8(__ldg(gp + v0), g[0]);
        widen8(__ldg(gp + v1), g[1]);
    }
    let_next();
    for (long long unit = first; unit < a.T * per_token; unit += nblocks * kQkWarps) {
        const long long t = unit / per_token;
        const int chunk = static_cast<int>(unit - t * per_token);
        const long long b = t / a.S, s = t - b * a.S;
        const int h0 = chunk * rows * kQkBwdUnroll + (lane >> a.log_group);
        const uint4 *yp = dy.p + b * dy.sb + s * dy.ss, *xp = x.p + b * x.sb + s * x.ss;
        uint4 vy[kQkBwdUnroll][2], vx[kQkBwdUnroll][2];
#pragma unroll
        for (int u = 0; u < kQkBwdUnroll; ++u) {
            const int h = h0 + u * rows;
            vy[u][0] = vy[u][1] = vx[u][0] = vx[u][1] = make_uint4(0u, 0u, 0u, 0u);
            if (works && h < H) {
                vy[u][0] = load_once(yp + h * dy.sh + v0);
                vy[u][1] = load_once(yp + h * dy.sh + v1);
                vx[u][0] = load_once(xp + h * x.sh + v0);
                vx[u][1] = load_once(xp + h * x.sh + v1);
            }
        }
        const long long p = a.pos != nullptr ? a.pos[b * a.pos_stride + s] : s;
        const bool bad = p < 0 || p >= a.P;
        if (bad && lane == 0) atomicExch(a.status, -1);
        float c[8], sn[8];
        if (works && !bad) qk_angles(a, p, slot, c, sn);
        uint4* op = dx.p + b * dx.sb + s * dx.ss;
#pragma unroll
        for (int u = 0; u < kQkBwdUnroll; ++u) {
            const int h = h0 + u * rows;
            float f[2][8], d[2][8];
            widen8(vx[u][0], f[0]);
            widen8(vx[u][1], f[1]);
            widen8(vy[u][0], d[0]);
            widen8(vy[u][1], d[1]);
            if (works && !bad && slot < a.nrot) qk_rotate<INTER>(d, c, sn);
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(f[0][i], f[0][i], fmaf(f[1][i], f[1][i], ss));
            const float r = 1.0f / sqrtf(group_sum(ss, group) * a.inv_d + a.eps);
            const bool store = works && h < H;
            float dot = 0.0f;
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    f[w][i] *= r;
                    if (store && !bad) acc[w][i] = fmaf(d[w][i], f[w][i], acc[w][i]);
                    d[w][i] *= g[w][i];
                    dot = fmaf(d[w][i], f[w][i], dot);
                }
            const float m = group_sum(dot, group) * a.inv_d;
            if (!store) continue;
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int i = 0; i < 8; ++i) d[w][i] = r * (d[w][i] - f[w][i] * m);
            op[h * dx.sh + v0] = bad ? qk_nan() : round8(d[0]);
            op[h * dx.sh + v1] = bad ? qk_nan() : round8(d[1]);
        }
    }
    if (a.part == nullptr) return;
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            for (int o = group; o < 32; o <<= 1) acc[w][i] += __shfl_xor_sync(0xffffffffu, acc[w][i], o);
    if (lane < a.nslot) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sums[warp][8 * v0 + i] = acc[0][i];
            sums[warp][8 * v1 + i] = acc[1][i];
        }
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
