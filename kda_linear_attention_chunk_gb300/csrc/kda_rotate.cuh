// kda_rotate.cuh -- a lane's elements of a head as the pairs that a rotation turns together.
// Not installed.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace kda {

template <typename E> struct Pair;
template <> struct Pair<__nv_bfloat16> {
    static __device__ __forceinline__ float2 up(uint32_t w)
    {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t down(float lo, float hi)
    {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};
template <> struct Pair<__half> {
    static __device__ __forceinline__ float2 up(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }
    static __device__ __forceinline__ uint32_t down(float lo, float hi)
    {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};

// The lane's eight elements as pairs (a[i], b[i]) that turn together.  HALF: a are
// four consecutive elements and b those half the rotary width further on, so no
// lane needs another's; INTERLEAVED, and behind the rotary width: eight consecutive.
template <typename E, bool HALF>
__device__ __forceinline__ void unpack(const uint2 (&r)[2], float (&a)[4], float (&b)[4])
{
    const float2 w0 = Pair<E>::up(r[0].x), w1 = Pair<E>::up(r[0].y), w2 = Pair<E>::up(r[1].x), w3 = Pair<E>::up(r[1].y);
    if (HALF) {
        a[0] = w0.x; a[1] = w0.y; a[2] = w1.x; a[3] = w1.y;
        b[0] = w2.x; b[1] = w2.y; b[2] = w3.x; b[3] = w3.y;
    } else {
        a[0] = w0.x; b[0] = w0.y; a[1] = w1.x; b[1] = w1.y;
        a[2] = w2.x; b[2] = w2.y; a[3] = w3.x; b[3] = w3.y;
    }
}

template <typename E, bool HALF>
__device__ __forceinline__ void pack(const float (&a)[4], const float (&b)[4], uint2 (&r)[2])
{
    if (HALF) {
        r[0] = make_uint2(Pair<E>::down(a[0], a[1]), Pair<E>::down(a[2], a[3]));
        r[1] = make_uint2(Pair<E>::down(b[0], b[1]), Pair<E>::down(b[2], b[3]));
    } else {
        r[0] = make_uint2(Pair<E>::down(a[0], b[0]), Pair<E>::down(a[1], b[1]));
        r[1] = make_uint2(Pair<E>::down(a[2], b[2]), Pair<E>::down(a[3], b[3]));
    }
}

}  // namespace kda
