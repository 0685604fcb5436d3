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
    Turn<E, D, HALF, FULL> turn(c, p.rotary);

    const uint16_t *x = p.x[which] + t * p.stride[which];
    uint2 raw[kUnroll][2];
#pragma unroll
    for (int u = 0; u < kUnroll; u++) {
        const int h = head0 + u * kPer;
        if (h < heads) turn.load(x + (int64_t)h * D, raw[u]);
        else raw[u][0] = raw[u][1] = make_uint2(0, 0);
    }
    const float *row = nullptr;
    if (turn.turns && turn.half) {
        int pos = __ldg(p.positions + t);
        if (pos < 0 || pos >= p.max_pos) {
            if (lane == 0) atomicOr(p.err, kErrBadPosition);
            pos = pos < 0 ? 0 : p.max_pos - 1;
        }
        row = p.table + (int64_t)pos * 2 * turn.half + 4 * c;
    }
    turn.fold(row, p.weight[which]);
    uint16_t *y = p.y[which] + t * heads * D;
#pragma unroll
    for (int u = 0; u < kUnroll; u++) {
        const int h = head0 + u * kPer;
        turn.apply(raw[u], p.norm, p.eps);
        if (h < heads) turn.store(y + (int64_t)h * D, raw[u]);
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
