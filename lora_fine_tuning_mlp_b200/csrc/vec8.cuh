// Eight bf16 values as one 16-byte vector, widened to fp32 and rounded back.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

namespace lmlp {
namespace step {

// Of the status word, which keeps the lowest: a wait that ran out
// (LORA_MLP_ERR_DEVICE_TIMEOUT, -7) is not hidden by an id out of its range.
constexpr int kStatusBad = -1;  // LORA_MLP_ERR_INVALID_ARG

__device__ __forceinline__ void widen8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 round8(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 bytes that this launch reads once and nobody writes meanwhile: not kept in
// L1, and written results (__stcs) leave L2 first.  32768 tokens of 32 + 4 heads
// turned both ways take 103 us so, 116 with a streaming load (ld.cs), 109 with
// plain stores.
__device__ __forceinline__ uint4 load_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// The same where the thread that reads may write these bytes afterwards: an
// ordinary load, with which the rotation above takes 7 % longer.
template <bool WRITTEN>
__device__ __forceinline__ uint4 load_once(const void* p) {
    if (!WRITTEN) return load_once(p);
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// The kernel before this one in the stream has ended and its writes are
// visible (programmatic dependent launch; nothing to wait for otherwise).
__device__ __forceinline__ void wait_prior() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel in the stream may start its blocks.
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;"); }

}  // namespace step
}  // namespace lmlp
