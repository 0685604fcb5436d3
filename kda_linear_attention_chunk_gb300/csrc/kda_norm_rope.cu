// kda_norm_rope.cu -- RMS norm of each head of q and k and the rotation of its
// position, in one pass.
//
//     y = w x / sqrt(mean(x^2) + eps);  (a, b) <- (a c_i - b s_i, b c_i + a s_i)
//
// over the pairs (y[i], y[i + r/2]) or (y[2i], y[2i+1]), i < r/2, in fp32 with one
// rounding at the end.  The pass reads and writes each 16-bit element once, so
// HBM bounds it.  d/8 lanes hold one head (16 bytes each); a warp takes one token
// and kUnroll groups of heads, issues all their loads at once, and reads its four
// cosines and sines of the table once for all of them.  8192 rows of 32 + 8 heads of
// 128 take 28.8 us on a GB300, 6.0 TB/s (with the pairs' other elements fetched from
// other lanes 38 us).
#include <stdint.h>

#include "kda_hybrid.h"
#include "kda_rotate.cuh"

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

// FULL: every element turns (rotary = D)
template <typename E, int D, bool HALF, bool FULL>
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
    const int half = FULL ? D / 2 : p.rotary / 2;
    const bool turns = FULL || 4 * c < half;             // this lane's pairs
    // elements ea .. ea + 3 and eb .. eb + 3 of a head
    const int ea = HALF && turns ? 4 * c : 8 * c, eb = HALF && turns ? 4 * c + half : 8 * c + 4;

    const uint16_t *x = p.x[which] + t * p.stride[which];
    uint2 raw[kUnroll][2];
#pragma unroll
    for (int u = 0; u < kUnroll; u++) {
        const int h = head0 + u * kPer;
        const uint16_t *at = x + (int64_t)h * D;
        if (h < heads) {
            if (HALF) {
                raw[u][0] = __ldcs(reinterpret_cast<const uint2 *>(at + ea));
                raw[u][1] = __ldcs(reinterpret_cast<const uint2 *>(at + eb));
            } else {
                const uint4 r = __ldcs(reinterpret_cast<const uint4 *>(at + ea));
                raw[u][0] = make_uint2(r.x, r.y);
                raw[u][1] = make_uint2(r.z, r.w);
            }
        } else {
            raw[u][0] = raw[u][1] = make_uint2(0, 0);
        }
    }
    // a' = rs (a ac - b bs),  b' = rs (b bc + a as): weights and angles are folded once
    // for the warp's heads
    float ac[4], as[4], bc[4], bs[4];
    {
        float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
        if (turns && half) {
            int pos = __ldg(p.positions + t);
            if (pos < 0 || pos >= p.max_pos) {
                if (lane == 0) atomicOr(p.err, kErrBadPosition);
                pos = pos < 0 ? 0 : p.max_pos - 1;
            }
            const float *row = p.table + (int64_t)pos * 2 * half + 4 * c;
            cs = __ldg(reinterpret_cast<const float4 *>(row));
            sn = __ldg(reinterpret_cast<const float4 *>(row + half));
        }
        float wa[4] = {1.f, 1.f, 1.f, 1.f}, wb[4] = {1.f, 1.f, 1.f, 1.f};
        if (p.weight[which]) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(p.weight[which] + ea));
            const float4 w = __ldg(reinterpret_cast<const float4 *>(p.weight[which] + eb));
            if (HALF) {
                wa[0] = v.x; wa[1] = v.y; wa[2] = v.z; wa[3] = v.w;
                wb[0] = w.x; wb[1] = w.y; wb[2] = w.z; wb[3] = w.w;
            } else {
                wa[0] = v.x; wb[0] = v.y; wa[1] = v.z; wb[1] = v.w;
                wa[2] = w.x; wb[2] = w.y; wa[3] = w.z; wb[3] = w.w;
            }
        }
        const float cv[4] = {cs.x, cs.y, cs.z, cs.w}, sv[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            ac[i] = wa[i] * cv[i];
            as[i] = wa[i] * sv[i];
            bc[i] = wb[i] * cv[i];
            bs[i] = wb[i] * sv[i];
        }
    }
    uint16_t *y = p.y[which] + t * heads * D;
#pragma unroll
    for (int u = 0; u < kUnroll; u++) {
        const int h = head0 + u * kPer;
        float a[4], b[4];
        unpack<E, HALF>(raw[u], a, b);
        if (p.norm) {
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                s0 = fmaf(a[i], a[i], s0);
                s1 = fmaf(b[i], b[i], s1);
            }
            float ss = s0 + s1;
#pragma unroll
            for (int k = kLanes / 2; k > 0; k /= 2) ss += __shfl_xor_sync(0xffffffffu, ss, k);
            const float rs = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                a[i] *= rs;
                b[i] *= rs;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float v = a[i], w = b[i];
            a[i] = v * ac[i];
            b[i] = w * bc[i];
            if (turns) {                                 // 0 times an infinity would not be 0
                a[i] = fmaf(-w, bs[i], a[i]);
                b[i] = fmaf(v, as[i], b[i]);
            }
        }
        if (h < heads) {
            uint2 r[2];
            pack<E, HALF>(a, b, r);
            uint16_t *at = y + (int64_t)h * D;
            if (HALF) {
                __stcs(reinterpret_cast<uint2 *>(at + ea), r[0]);
                __stcs(reinterpret_cast<uint2 *>(at + eb), r[1]);
            } else {
                __stcs(reinterpret_cast<uint4 *>(at + ea), make_uint4(r[0].x, r[0].y, r[1].x, r[1].y));
            }
        }
    }
}

template <typename E, int D>
cudaError_t launch(const NormRopeArgs &a, const NormRopeParams &p)
{
    const int64_t blocks = ((int64_t)a.T + kWarps - 1) / kWarps * (p.chunks[0] + p.chunks[1]);
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const bool full = a.rotary == D;
    auto *kernel = a.layout == 0 ? (full ? norm_rope_kernel<E, D, true, true> : norm_rope_kernel<E, D, true, false>)
                                 : (full ? norm_rope_kernel<E, D, false, true> : norm_rope_kernel<E, D, false, false>);
    kernel<<<(unsigned)blocks, kWarps * 32, 0, a.stream>>>(p);
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
