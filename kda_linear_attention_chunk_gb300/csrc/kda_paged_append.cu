// kda_paged_append.cu -- per-head RMS norm and rotation of q and k, with k and v on
// their way into a paged cache, in one pass.
//
// The arithmetic is kda_rotate.cuh's; each element is read and written once, so HBM
// bounds it.  A warp takes one token and kUnroll groups of heads of q, k or v, and
// has all its loads on their way before it looks for the token's sequence, position
// and page.
#include <stdint.h>

#include "kda_common.cuh"
#include "kda_paged.cuh"
#include "kda_rotate.cuh"

namespace kda {
namespace {

constexpr int kWarps = 8;
constexpr int kUnroll = 4;   // groups of 32 / (d/8) heads that a warp takes

struct AppendParams {
    const uint16_t *x[3];        // q, k, v
    int64_t stride[3];
    const float *weight[2], *angles;
    const int32_t *cu, *starts, *slots;
    PagedCache cache;
    uint16_t *q_out;
    int heads[3], chunks[3];     // heads; warps per token
    int N, T, rotary, max_pos, norm;
    float eps;
    int *err;
};

// FULL: every element turns (rotary = D)
template <typename E, int D, bool HALF, bool FULL>
__global__ void __launch_bounds__(kWarps * 32)
paged_append_kernel(const __grid_constant__ AppendParams p)
{
    constexpr int kLanes = D / 8, kPer = 32 / kLanes;   // lanes of a head, heads of a warp at a time
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int chunks = p.chunks[0] + p.chunks[1] + p.chunks[2];
    int chunk = blockIdx.x % chunks, which = 0;
    const int64_t t = (int64_t)(blockIdx.x / chunks) * kWarps + warp;
    if (t >= p.T) return;
    while (chunk >= p.chunks[which]) chunk -= p.chunks[which++];
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
    const bool reports = lane == 0 && which == 1 && chunk == 0;
    const int n = p.cu ? sequence_with(p.cu, p.N, (int)t, lane) : (int)t;
    if (n < 0) return;                                   // a row of no sequence
    const int entry = entry_of(p.slots, n, p.cache.num_slots, p.err, reports);
    if (entry < 0) return;
    const RowsAt r = rows_at(p.cu, p.starts, p.cache, n, p.T, 0, reports ? p.err : nullptr);
    const int pos = r.start + ((int)t - r.bos);
    uint16_t *to;                                        // head 0's row, and the distance of heads
    int64_t apart = D;
    if (which == 0) {
        to = p.q_out + t * heads * D;
    } else {
        const int id = page_at(p.cache, entry, pos);
        if (id < 0) {
            if (reports && pos < capacity(p.cache)) atomicOr(p.err, kErrBadPage);
            return;
        }
        apart = (int64_t)D << p.cache.page_log2;
        to = p.cache.pages + ((int64_t)id * 2 + (which - 1)) * heads * apart +
                (int64_t)(pos & ((1 << p.cache.page_log2) - 1)) * D;
    }
    if (which < 2) {
        const float *row = nullptr;
        if (turn.half) {
            if (pos >= p.max_pos && reports) atomicOr(p.err, kErrBadPosition);
            row = p.angles + (int64_t)min(pos, p.max_pos - 1) * 2 * turn.half + 4 * c;
        }
        turn.fold(row, p.weight[which]);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; u++) {
        const int h = head0 + u * kPer;
        if (which < 2) turn.apply(raw[u], p.norm, p.eps);
        if (h < heads) turn.store(to + h * apart, raw[u]);
    }
}

template <typename E, int D>
cudaError_t launch(const PagedAppendArgs &a, const AppendParams &p)
{
    const int64_t blocks = ((int64_t)a.T + kWarps - 1) / kWarps * (p.chunks[0] + p.chunks[1] + p.chunks[2]);
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const bool full = a.rotary == D;
    auto *kernel = a.layout == 0 ? (full ? paged_append_kernel<E, D, true, true> : paged_append_kernel<E, D, true, false>)
                                 : (full ? paged_append_kernel<E, D, false, true> : paged_append_kernel<E, D, false, false>);
    kernel<<<(unsigned)blocks, kWarps * 32, 0, a.stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs &a)
{
    AppendParams p;
    p.x[0] = (const uint16_t *)a.q; p.x[1] = (const uint16_t *)a.k; p.x[2] = (const uint16_t *)a.v;
    p.stride[0] = a.q_stride; p.stride[1] = a.k_stride; p.stride[2] = a.v_stride;
    p.weight[0] = a.q_weight; p.weight[1] = a.k_weight; p.angles = a.angles;
    p.cu = a.cu_seqlens; p.starts = a.starts; p.slots = a.slots;
    p.cache = a.cache; p.q_out = (uint16_t *)a.q_out;
    const int per = 32 / (a.d / 8) * kUnroll;
    for (int i = 0; i < 3; i++) {
        p.heads[i] = i ? a.Hk : a.Hq;
        p.chunks[i] = (p.heads[i] + per - 1) / per;
    }
    p.N = a.N; p.T = a.T; p.rotary = a.rotary; p.max_pos = a.max_pos; p.norm = a.norm; p.eps = a.eps;
    p.err = a.err_word;
    if (a.d == 128) return a.f16 ? launch<__half, 128>(a, p) : launch<__nv_bfloat16, 128>(a, p);
    return a.f16 ? launch<__half, 64>(a, p) : launch<__nv_bfloat16, 64>(a, p);
}

}  // namespace kda
