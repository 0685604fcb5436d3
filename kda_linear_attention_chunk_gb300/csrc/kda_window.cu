// kda_window.cu -- window attention of packed new tokens over the ring cache and
// themselves (prefill, and the verification of drafts).
//
// For the query at position p:  o = sum_j softmax_j(scale q . k_j) v_j  over the
// positions j <= p with j > p - window or j < sinks.  One warp takes one (token,
// query head) and walks the visible keys with a running maximum and sum; keys of
// positions before the call's come from the cache, the others from the call's
// rows.  A second kernel then writes the rows that the cache keeps.
#include <stdint.h>

#include "kda_window.h"

namespace kda {
namespace {

struct PrefillParams {
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const int32_t *cu, *starts, *slots;
    uint16_t *pool, *out;
    int N, T, Hq, Hk, num_slots, pool_rows, window, sinks;
    float scale_log2;
    int *err;
};

// the last sequence that starts at or before row t (the one that holds it, if any does)
__device__ __forceinline__ int sequence_of(const int32_t *cu, int N, int t)
{
    int a = 0, b = N - 1;
    while (a < b) {
        const int c = (a + b + 1) / 2;
        if (cu[c] <= t) a = c; else b = c - 1;
    }
    return a;
}

// positions before the first row of sequence n, which has L rows
__device__ __forceinline__ int start_of(const PrefillParams &p, int n, int L, bool reports)
{
    if (!p.starts) return 0;
    const int s = p.starts[n], most = 0x7fffffff - L;
    if (s < 0 || s > most) {
        if (reports) atomicOr(p.err, kErrBadPosition);
        return s < 0 ? 0 : most;
    }
    return s;
}

template <typename E, int D>
__global__ void __launch_bounds__(256) window_prefill_kernel(const __grid_constant__ PrefillParams p)
{
    constexpr int kPer = D / 32;     // elements of a lane
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int t = (int)(w / p.Hq), h = (int)(w % p.Hq);
    if (t >= p.T) return;
    const int n = sequence_of(p.cu, p.N, t);
    const int bos = clamp_row(p.cu[n], p.T, p.err), eos = clamp_row(p.cu[n + 1], p.T, p.err);
    if (t < bos || t >= eos) return;
    const bool reports = t == bos && h == 0 && lane == 0;
    const int entry = entry_of(p.slots, n, p.num_slots, p.err, reports);
    if (entry < 0) return;
    const int start = start_of(p, n, eos - bos, reports), pos = start + t - bos;
    const int hk = h / (p.Hq / p.Hk);
    const uint16_t *kc = nullptr, *vc = nullptr;
    if (p.pool) {
        kc = p.pool + ((int64_t)entry * 2 * p.Hk + hk) * p.pool_rows * D;
        vc = kc + (int64_t)p.Hk * p.pool_rows * D;
    }
    float q[kPer], o[kPer], m = -INFINITY, l = 0.f;
    auto load = [&](const uint16_t *src, float (&x)[kPer]) {
        const uint32_t *s = reinterpret_cast<const uint32_t *>(src) + lane * (kPer / 2);
#pragma unroll
        for (int i = 0; i < kPer / 2; i++) {
            const float2 f = Half2<E>::unpack(s[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    };
    load(p.q + t * p.q_stride + (int64_t)h * D, q);
#pragma unroll
    for (int i = 0; i < kPer; i++) o[i] = 0.f;
    const int lo = pos - p.window + 1 < 0 ? 0 : pos - p.window + 1, ns = min(p.sinks, lo);
    for (int64_t i = 0; i < (int64_t)ns + (pos - lo) + 1; i++) {
        const int j = i < ns ? (int)i : lo + (int)(i - ns);
        const uint16_t *kr, *vr;
        if (j >= start) {
            kr = p.k + (bos + j - start) * p.k_stride + hk * D;
            vr = p.v + (bos + j - start) * p.v_stride + hk * D;
        } else {
            const int64_t r = (int64_t)ring_row(j, p.sinks, p.pool_rows) * D;
            kr = kc + r;
            vr = vc + r;
        }
        float x[kPer], s = 0.f;
        load(kr, x);
#pragma unroll
        for (int e = 0; e < kPer; e++) s = fmaf(q[e], x[e], s);
#pragma unroll
        for (int b = 16; b; b /= 2) s += __shfl_xor_sync(0xffffffffu, s, b);
        s *= p.scale_log2;
        const float mn = fmaxf(m, s), f = mn == -INFINITY ? 1.f : ex2(m - mn), e = mn == -INFINITY ? 0.f : ex2(s - mn);
        m = mn;
        l = l * f + e;
        load(vr, x);
#pragma unroll
        for (int k = 0; k < kPer; k++) o[k] = o[k] * f + e * x[k];
    }
    uint32_t *to = reinterpret_cast<uint32_t *>(p.out + ((int64_t)t * p.Hq + h) * D) + lane * (kPer / 2);
#pragma unroll
    for (int i = 0; i < kPer / 2; i++) to[i] = Half2<E>::pack(o[2 * i] / l, o[2 * i + 1] / l);
}

// Writes the rows that the cache keeps: sinks, and the sequence's last pool_rows
// - sinks positions.  16 bytes a thread.
template <int D>
__global__ void __launch_bounds__(256) ring_commit_kernel(const __grid_constant__ PrefillParams p)
{
    const int per = p.Hk * (D / 8);
    const int64_t w = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int t = (int)(w / per), e = (int)(w % per);
    if (t >= p.T) return;
    const int n = sequence_of(p.cu, p.N, t);
    const int bos = clamp_row(p.cu[n], p.T, nullptr), eos = clamp_row(p.cu[n + 1], p.T, nullptr);
    if (t < bos || t >= eos) return;
    const int entry = entry_of(p.slots, n, p.num_slots, nullptr, false);
    if (entry < 0) return;
    const int start = start_of(p, n, eos - bos, false), pos = start + t - bos;
    if (pos >= p.sinks && eos - t > p.pool_rows - p.sinks) return;
    const int hk = e / (D / 8), at = (e % (D / 8)) * 8;
    uint16_t *to = p.pool + ((int64_t)entry * 2 * p.Hk + hk) * p.pool_rows * D +
                   (int64_t)ring_row(pos, p.sinks, p.pool_rows) * D + at;
    *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(p.k + t * p.k_stride + hk * D + at);
    to += (int64_t)p.Hk * p.pool_rows * D;
    *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(p.v + t * p.v_stride + hk * D + at);
}

template <typename E, int D>
cudaError_t launch(const WindowArgs &a, const PrefillParams &p)
{
    window_prefill_kernel<E, D><<<(unsigned)(((int64_t)p.T * p.Hq + 7) / 8), 256, 0, a.stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.pool) return e;
    ring_commit_kernel<D><<<(unsigned)(((int64_t)p.T * p.Hk * (D / 8) + 255) / 256), 256, 0, a.stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_prefill(const WindowArgs &a)
{
    PrefillParams p;
    p.q = (const uint16_t *)a.q; p.k = (const uint16_t *)a.k; p.v = (const uint16_t *)a.v;
    p.q_stride = a.q_stride; p.k_stride = a.k_stride; p.v_stride = a.v_stride;
    p.cu = a.cu_seqlens; p.starts = a.starts; p.slots = a.slots;
    p.pool = (uint16_t *)a.pool; p.out = (uint16_t *)a.out;
    p.N = a.N; p.T = a.T; p.Hq = a.Hq; p.Hk = a.Hk; p.num_slots = a.num_slots; p.pool_rows = a.pool_rows;
    p.window = a.window; p.sinks = a.sinks;
    p.scale_log2 = a.scale * kLog2e;
    p.err = a.err_word;
    if (a.d == 128) return a.f16 ? launch<__half, 128>(a, p) : launch<__nv_bfloat16, 128>(a, p);
    return a.f16 ? launch<__half, 64>(a, p) : launch<__nv_bfloat16, 64>(a, p);
}

}  // namespace kda
