// kda_tiles.cuh -- what the attention kernels on tcgen05 share: products of 128-row
// tiles, exponents, tensor maps.  Not installed.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "kda_sm100.cuh"

namespace kda {
namespace tiles {

using namespace sm100;

__host__ __device__ constexpr uint32_t idesc(int N, int b_mn, bool f16)
{
    return (1u << 4) | ((f16 ? 0u : 1u) << 7) | ((f16 ? 0u : 1u) << 10) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// Upper halves of the matrix descriptors (8-row groups 1024 bytes apart, version
// 1, 128-byte swizzle); a lower half is the address / 16 and the leading offset.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

__device__ __forceinline__ void mma_ss_lo(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc)
{
    asm volatile("{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %4, 0;\n mov.b64 x, {%1, %5};\n mov.b64 y, {%2, %5};\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}" ::"r"(d), "r"(a), "r"(b), "r"(id), "r"(acc),
                 "r"(kDescHi)
                 : "memory");
}
__device__ __forceinline__ void mma_ts_lo(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc)
{
    asm volatile("{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.b32 p, %4, 0;\n mov.b64 y, {%2, %5};\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}" ::"r"(d), "r"(a), "r"(b), "r"(id), "r"(acc),
                 "r"(kDescHi)
                 : "memory");
}

// One lane of the (converged) warp, the same every time.
__device__ __forceinline__ bool elect_one()
{
    uint32_t yes;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.b32 %0, 1, 0, p;\n}" : "=r"(yes));
    return yes != 0;
}

// S = Q K^T: both operands K-major, halves of 64 columns 16 KB apart
template <int D>
__device__ __forceinline__ void mma_scores(uint32_t s, uint32_t q, uint32_t k, uint32_t id)
{
    const uint32_t a = (q >> 4) | (1u << 16), b = (k >> 4) | (1u << 16);
#pragma unroll
    for (int i = 0; i < D / 16; i++) {
        const uint32_t at = (i / 4) * 1024 + (i % 4) * 2;
        mma_ss_lo(s, a + at, b + at, id, i > 0);
    }
}

// O += P V for the four 16-key steps from `from` on: P in TMEM, V MN-major, 16
// keys are 2048 bytes of it
template <int D>
__device__ __forceinline__ void mma_values(uint32_t o, uint32_t pt, uint32_t v, uint32_t id, int from, int steps, bool more)
{
    const uint32_t b = (v >> 4) | (1024u << 16);
    if (steps >= from + 4) {
#pragma unroll
        for (int i = 0; i < 4; i++) mma_ts_lo(o, pt + 8 * (from + i), b + 128 * (from + i), id, i > 0 ? 1 : more);
    } else {
#pragma unroll 1
        for (int i = from; i < steps; i++) mma_ts_lo(o, pt + 8 * i, b + 128 * i, id, i > from || more);
    }
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
        " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// A row's exponents are slope s - z, one paired instruction, with z = slope m rounded.  What
// z is off by cancels between P and their sum, provided that a change of m counts it
// (residue), and at most multiplies the P of the maximum.  Its size, 2^-24 of z, has to
// stay within P's range: up to 2^2 (fp16) or 2^5.  Beyond that, two scores that differ by
// the last bit of their 32 are 2^4 (fp16) or 2^32 apart in weight, and the slope becomes the
// power of two that brings m to 2^29: slope m is exact then, the largest score has the
// weight 1 and a lower one less than 2^-31.  (s - m) slope instead, two instructions a
// pair, costs 4 % of a long window: 413 us for 397 (8192 rows, W 4096).
template <typename E> __device__ __forceinline__ float slope(float m, float c)
{
    constexpr float kSteep = __is_same(E, __nv_bfloat16) ? 1 << 30 : 1 << 27;
    return fabsf(m * c) < kSteep ? c : __uint_as_float((283u << 23) - (__float_as_uint(m) & 0x7f800000u));
}
__device__ __forceinline__ float residue(float m, float slope) { return fmaf(m, slope, -(m * slope)); }

// The n lowest bits (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t below(int n) { return ~__funnelshift_lc(0u, ~0u, (uint32_t)max(n, 0)); }

// Waits for the TMEM loads, as seen by whatever uses these registers.
__device__ __forceinline__ void loaded(uint32_t (&a)[32], uint32_t (&b)[32], uint32_t (&c)[32], uint32_t (&d)[32])
{
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; i++) asm volatile("" : "+r"(a[i]), "+r"(b[i]), "+r"(c[i]), "+r"(d[i]));
}

// The driver's tensor-map encoder, looked up once.
inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess && q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
        return nullptr;
    }();
    return fn;
}

// a dense innermost axis of d elements, two more with the given extents and
// strides (elements); boxes of 64 x b1 x b2, 128-byte swizzled
inline bool make_map(CUtensorMap *m, const void *base, bool f16, int d, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int b1,
              int b2)
{
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)n1, (cuuint64_t)n2};
    const cuuint64_t strides[2] = {(cuuint64_t)s1 * 2, (cuuint64_t)s2 * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)b1, (cuuint32_t)b2}, es[3] = {1, 1, 1};
    return fn(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base),
              dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tiles
}  // namespace kda
