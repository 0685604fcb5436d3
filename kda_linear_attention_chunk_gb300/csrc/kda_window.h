// kda_window.h -- what the window-attention kernels share: the visible
// positions of a query and their rows in the ring cache.  Not installed.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "kda_common.cuh"
#include "kda_hybrid.h"

namespace kda {

constexpr float kLog2e = 1.4426950408889634f;

// 2^x on the special-function unit (2 ulp; results below 2^-126 are zero)
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// the pool entry of sequence n: -1 for a padded one; an id out of range is
// reported (by the caller that `reports`) and skipped
__device__ __forceinline__ int entry_of(const int32_t *slots, int n, int num_slots, int *err, bool reports)
{
    if (!slots) return n;
    const int s = slots[n];
    if (s >= 0 && s < num_slots) return s;
    if (s != -1 && reports) atomicOr(err, kErrBadSlot);
    return -1;
}

// row of position p in a ring cache of `rows` rows
__device__ __forceinline__ int ring_row(int p, int sinks, int rows)
{
    return p < sinks ? p : sinks + (p - sinks) % (rows - sinks);
}

template <typename E> struct Half2;
template <> struct Half2<__nv_bfloat16> {
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t w)
    {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
};
template <> struct Half2<__half> {
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }
};

}  // namespace kda
