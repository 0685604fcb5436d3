// kda_norm_rope.cu -- RMS norm of each head of q and k and the rotation of its
// position, in one pass.
//
//     y = w x / sqrt(mean(x^2) + eps);  (a, b) <- (a c_i - b s_i, b c_i + a s_i)
//
// over the pairs (y[i], y[i + r/2]) or (y[2i], y[2i+1]), i < r/2, in fp32 with one
// rounding at the end.  The pass reads and writes each 16-bit element once, so
// HBM bounds it.  d/8 lanes hold one head (16 bytes each); a warp takes one token
// and kUnroll groups of heads, issues all their loads at once, and reads its 8
// cosines and sines of the table once for all of them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "kda_hybrid.h"

namespace kda {
namespace {

constexpr int kWarps = 8;
constexpr int kUnroll = 4;   // groups of 32 / (d/8) heads that a warp takes

struct NormRopeParams {
    const uint16_t *x[2];        // q, k
    uint16_t *y[2];
    int64_t stride[2];
    const float *weight[2];
    const float *table;
    const int32_t *positions;
    int heads[2], chunks[2];     // heads; warps per token
    int T, rotary, max_pos, norm;
    float eps;
    int *err;
};

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

template <typename E>
__device__ __forceinline__ void up8(const uint4 &r, float (&x)[8])
{
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 p = Pair<E>::up(w[i]);
        x[2 * i] = p.x;
        x[2 * i + 1] = p.y;
    }
}

__device__ __forceinline__ void load8(const float *p, float (&x)[8])
{
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

template <typename E, int D, bool HALF>
__global__ void __launch_bounds__(kWarps * 32)
norm_rope_kernel(const __grid_constant__ NormRopeParams p)
{
    constexpr int kLanes = D / 8, kPer = 32 / kLanes;   // lanes of a head, heads of a warp at a time
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int chunks = p.chunks[0] + p.chunks[1];
    int chunk = blockIdx.x % chunks;
    const int64_t t = (int64_t)(blockIdx.x / chunks) * kWarps + warp;
    if (t >= p.T) return;
    const int which = chunk >= p.chunks[0];
    if (which) chunk -= p.chunks[0];
    const int c = lane % kLanes, heads = p.heads[which];
    const int head0 = chunk * kPer * kUnroll + lane / kLanes;

    const uint16_t *x = p.x[which] + t * p.stride[which] + 8 * c;
    uint4 raw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; u++) {
        const int h = head0 + u * kPer;
        raw[u] = h < heads ? __ldcs(reinterpret_cast<const uint4 *>(x + (int64_t)h * D)) : make_uint4(0, 0, 0, 0);
    }
    float w[8], wp[8], cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; i++) w[i] = wp[i] = 1.f;
    const int half = p.rotary / 2;
    const bool turns = 8 * c < p.rotary, first = 8 * c < half;
    const int shift = turns ? (first ? half / 8 : -(half / 8)) : 0;   // the lane that holds the pairs' other elements
    if (p.weight[which]) {
        load8(p.weight[which] + 8 * c, w);
        if (HALF) load8(p.weight[which] + 8 * (c + shift), wp);
    }
    if (p.rotary) {
        int pos = __ldg(p.positions + t);
        if (pos < 0 || pos >= p.max_pos) {
            if (lane == 0) atomicOr(p.err, kErrBadPosition);
            pos = pos < 0 ? 0 : p.max_pos - 1;
        }
        if (turns) {
            const float *row = p.table + (int64_t)pos * p.rotary;
            if (HALF) {
                load8(row + 8 * c - (first ? 0 : half), cs);
                load8(row + 8 * c + (first ? half : 0), sn);
                if (first)
#pragma unroll
                    for (int i = 0; i < 8; i++) sn[i] = -sn[i];
            } else {
                const float4 a = __ldg(reinterpret_cast<const float4 *>(row + 4 * c));
                const float4 b = __ldg(reinterpret_cast<const float4 *>(row + half + 4 * c));
                cs[0] = a.x; cs[1] = a.y; cs[2] = a.z; cs[3] = a.w;
                sn[0] = b.x; sn[1] = b.y; sn[2] = b.z; sn[3] = b.w;
            }
        }
    }
    uint16_t *y = p.y[which] + (t * heads) * D + 8 * c;
#pragma unroll
    for (int u = 0; u < kUnroll; u++) {
        const int h = head0 + u * kPer;
        float v[8];
        up8<E>(raw[u], v);
        float rs = 1.f;
        if (p.norm) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; i++) ss = fmaf(v[i], v[i], ss);
#pragma unroll
            for (int o = kLanes / 2; o > 0; o /= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            rs = rsqrtf(ss * (1.f / D) + p.eps);
        }
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = v[i] * rs * w[i];
        if (HALF) {
            uint4 other;
            other.x = __shfl_sync(0xffffffffu, raw[u].x, lane + shift);
            other.y = __shfl_sync(0xffffffffu, raw[u].y, lane + shift);
            other.z = __shfl_sync(0xffffffffu, raw[u].z, lane + shift);
            other.w = __shfl_sync(0xffffffffu, raw[u].w, lane + shift);
            if (turns) {
                float o[8];
                up8<E>(other, o);
#pragma unroll
                for (int i = 0; i < 8; i++) v[i] = v[i] * cs[i] + (o[i] * rs * wp[i]) * sn[i];
            }
        } else if (turns) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float a = v[2 * i], b = v[2 * i + 1];
                v[2 * i] = a * cs[i] - b * sn[i];
                v[2 * i + 1] = b * cs[i] + a * sn[i];
            }
        }
        if (h < heads) {
            uint4 r;
            r.x = Pair<E>::down(v[0], v[1]);
            r.y = Pair<E>::down(v[2], v[3]);
            r.z = Pair<E>::down(v[4], v[5]);
            r.w = Pair<E>::down(v[6], v[7]);
            *reinterpret_cast<uint4 *>(y + (int64_t)h * D) = r;
        }
    }
}

template <typename E, int D>
cudaError_t launch(const NormRopeArgs &a, const NormRopeParams &p)
{
    const int64_t blocks = ((int64_t)a.T + kWarps - 1) / kWarps * (p.chunks[0] + p.chunks[1]);
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    if (a.layout == 0)
        norm_rope_kernel<E, D, true><<<(unsigned)blocks, kWarps * 32, 0, a.stream>>>(p);
    else
        norm_rope_kernel<E, D, false><<<(unsigned)blocks, kWarps * 32, 0, a.stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs &a)
{
    NormRopeParams p;
    p.x[0] = (const uint16_t *)a.q; p.x[1] = (const uint16_t *)a.k;
    p.y[0] = (uint16_t *)a.q_out; p.y[1] = (uint16_t *)a.k_out;
    p.stride[0] = a.q_stride; p.stride[1] = a.k_stride;
    p.weight[0] = a.q_weight; p.weight[1] = a.k_weight;
    p.table = a.table; p.positions = a.positions;
    const int per = 32 / (a.d / 8) * kUnroll;
    p.heads[0] = a.Hq; p.heads[1] = a.Hk;
    p.chunks[0] = (a.Hq + per - 1) / per; p.chunks[1] = (a.Hk + per - 1) / per;
    p.T = a.T; p.rotary = a.rotary; p.max_pos = a.max_pos; p.norm = a.norm; p.eps = a.eps;
    p.err = a.err_word;
    if (a.d == 128) return a.f16 ? launch<__half, 128>(a, p) : launch<__nv_bfloat16, 128>(a, p);
    return a.f16 ? launch<__half, 64>(a, p) : launch<__nv_bfloat16, 64>(a, p);
}

}  // namespace kda
