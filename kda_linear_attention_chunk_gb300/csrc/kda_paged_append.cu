// kda_paged_append.cu -- per-head RMS norm and rotation of q and k, with k and v on
// their way into a paged cache, in one pass.
//
// The arithmetic is kda_norm_rope.cu's; each element is read and written once, so HBM
// bounds it.  A warp takes one token and kUnroll groups of heads of q, k or v, and
// has all its loads on their way before it looks for the token's sequence, position
// and page.  8192 rows of 32 + 8 + 8 heads of 128 take 36.7 us on a GB300, 5.6 TB/s: issue
// slots are 70 % busy beside HBM's 83 %.
#include <stdint.h>

#include "kda_common.cuh"
#include "kda_paged.cuh"
#include "kda_rotate.cuh"

namespace kda {
namespace {

constexpr int kWarps = 8;
constexpr int kCtas = 5;     // CTAs an SM: 48 registers (4 and 64: 37.7 us for 36.7)
constexpr int kUnroll = 4;   // groups of 32 / (d/8) heads that a warp takes (2: 43, 8: 39 us)

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
__global__ void __launch_bounds__(kWarps * 32, kCtas)
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
    // the token's sequence; its facts are on their way together
    const bool reports = lane == 0 && which == 1 && chunk == 0;
    int *err = reports ? p.err : nullptr;
    const int n = p.cu ? last_at_or_below(p.cu, p.N, (int)t, lane) : (int)t;
    const int cu0 = p.cu ? __ldg(p.cu + n) : n, cu1 = p.cu ? __ldg(p.cu + n + 1) : n + 1;
    const int start = p.starts ? __ldg(p.starts + n) : 0, slot = p.slots ? __ldg(p.slots + n) : n;
    if (t < cu0 || t >= cu1) return;                     // a row of no sequence
    if (slot < 0 || slot >= p.cache.num_slots) {
        if (slot != -1 && reports) atomicOr(p.err, kErrBadSlot);
        return;
    }
    const RowsAt r = rows_at(cu0, cu1, start, p.cache, p.T, 0, err);
    const int pos = r.start + ((int)t - r.bos);
    uint16_t *to;                                        // head 0's row, and the distance of heads
    int64_t apart = D;
    if (which == 0) {
        to = p.q_out + t * heads * D;
    } else {
        const int id = page_at(p.cache, slot, pos);
        if (id < 0) {
            if (reports && pos < capacity(p.cache)) atomicOr(p.err, kErrBadPage);
            return;
        }
        apart = (int64_t)D << p.cache.page_log2;
        to = p.cache.pages + ((int64_t)id * 2 + (which - 1)) * heads * apart +
                (int64_t)(pos & ((1 << p.cache.page_log2) - 1)) * D;
    }
    // a' = rs (a ac - b bs),  b' = rs (b bc + a as): weights and angles are folded once
    // for the warp's heads
    float ac[4], as[4], bc[4], bs[4];
    if (which < 2) {
        float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
        if (turns && half) {
            if (pos >= p.max_pos && reports) atomicOr(p.err, kErrBadPosition);
            const float *row = p.angles + (int64_t)min(pos, p.max_pos - 1) * 2 * half + 4 * c;
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
#pragma unroll
    for (int u = 0; u < kUnroll; u++) {
        const int h = head0 + u * kPer;
        if (which < 2) {                                 // (values go as they are)
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
                if (turns) {                             // 0 times an infinity would not be 0
                    a[i] = fmaf(-w, bs[i], a[i]);
                    b[i] = fmaf(v, as[i], b[i]);
                }
            }
            pack<E, HALF>(a, b, raw[u]);
        }
        if (h < heads) {
            uint16_t *at = to + h * apart;
            if (HALF) {
                __stcs(reinterpret_cast<uint2 *>(at + ea), raw[u][0]);
                __stcs(reinterpret_cast<uint2 *>(at + eb), raw[u][1]);
            } else {
                __stcs(reinterpret_cast<uint4 *>(at + ea), make_uint4(raw[u][0].x, raw[u][0].y, raw[u][1].x, raw[u][1].y));
            }
        }
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
