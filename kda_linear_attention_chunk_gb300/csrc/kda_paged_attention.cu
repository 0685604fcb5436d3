// kda_paged_attention.cu -- causal softmax attention over a paged cache with shared
// prefixes, in its simplest form: a warp for each row and query head.
//
//     o = sum_j 2^(c s_j - c m) v_j / sum_j 2^(c s_j - c m),   s_j = q . k_j,  c = scale log2 e
#include <stdint.h>

#include "kda_paged.cuh"

namespace kda {
namespace {

constexpr int kWarps = 8;

struct AttendParams {
    const uint16_t *q;
    int64_t q_stride;
    const int32_t *cu, *starts, *slots, *groups, *prefix_lens, *prefix_slots;
    PagedCache cache;
    uint16_t *out;
    int N, T, P, Hq, Hk, G;
    float scale_log2;
    int *err;
};

// the group of sequence n, by a converged warp; -1: none
__device__ __forceinline__ int group_with(const AttendParams &p, int n, int lane)
{
    return p.P ? sequence_with(p.groups, p.P, n, lane) : -1;
}

template <typename E, int D>
__global__ void __launch_bounds__(kWarps * 32) attend_rows_kernel(const __grid_constant__ AttendParams p)
{
    constexpr int kEach = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (item >= (int64_t)p.T * p.Hq) return;
    if (item == 0)
        for (int g = lane; g < p.P + 1 && p.P; g += 32)
            if (p.groups[g] < 0 || p.groups[g] > p.N || (g && p.groups[g] < p.groups[g - 1])) atomicOr(p.err, kErrBadSeqlens);
    const int t = (int)(item / p.Hq), hq = (int)(item - (int64_t)t * p.Hq), hk = hq / p.G;
    int *err = lane == 0 && hq == 0 ? p.err : nullptr;
    const int n = p.cu ? sequence_with(p.cu, p.N, t, lane) : t;
    if (n < 0) return;
    const int entry = entry_of(p.slots, n, p.cache.num_slots, p.err, err);
    if (entry < 0) return;
    const int g = group_with(p, n, lane);
    int prefix = 0, shared = -1;
    if (g >= 0) {
        shared = entry_of(p.prefix_slots, g, p.cache.num_slots, p.err, err);
        const int was = p.prefix_lens[g];
        prefix = shared < 0 ? 0 : min(max(was, 0), capacity(p.cache));
        if (err && shared >= 0 && prefix != was) atomicOr(err, kErrBadPosition);
    }
    const RowsAt r = rows_at(p.cu, p.starts, p.cache, n, p.T, prefix, err);
    const int last = min(r.start + (t - r.bos), capacity(p.cache) - 1);
    const uint16_t *q = p.q + t * p.q_stride + (int64_t)hq * D;
    float x[kEach], o[kEach], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < kEach / 2; i++) {
        const float2 v = Half2<E>::unpack(reinterpret_cast<const uint32_t *>(q)[lane + 32 * i]);
        x[2 * i] = v.x;
        x[2 * i + 1] = v.y;
        o[2 * i] = o[2 * i + 1] = 0.f;
    }
    const int64_t head = (int64_t)D << p.cache.page_log2;
    int id = -1;
    for (int j = 0; j <= last; j++) {
        if (j == 0 || j == prefix || (j & ((1 << p.cache.page_log2) - 1)) == 0) {
            id = page_at(p.cache, j < prefix ? shared : entry, j);
            if (id < 0 && err) atomicOr(err, kErrBadPage);
        }
        const uint32_t *k = reinterpret_cast<const uint32_t *>(p.cache.pages + ((int64_t)max(id, 0) * 2 * p.Hk + hk) * head +
                                                               (int64_t)(j & ((1 << p.cache.page_log2) - 1)) * D);
        const uint32_t *v = k + p.Hk * head / 2;
        float s = 0.f;
        float2 kv[kEach / 2], vv[kEach / 2];
#pragma unroll
        for (int i = 0; i < kEach / 2; i++) {
            kv[i] = Half2<E>::unpack(id < 0 ? 0u : k[lane + 32 * i]);
            vv[i] = Half2<E>::unpack(id < 0 ? 0u : v[lane + 32 * i]);
            s = fmaf(x[2 * i], kv[i].x, fmaf(x[2 * i + 1], kv[i].y, s));
        }
#pragma unroll
        for (int b = 16; b > 0; b /= 2) s += __shfl_xor_sync(0xffffffffu, s, b);
        const float top = fmaxf(m, s);
        if (top == -INFINITY) continue;
        const float f = ex2((m - top) * p.scale_log2), w = ex2((s - top) * p.scale_log2);
        m = top;
        l = fmaf(l, f, w);
#pragma unroll
        for (int i = 0; i < kEach / 2; i++) {
            o[2 * i] = fmaf(w, vv[i].x, o[2 * i] * f);
            o[2 * i + 1] = fmaf(w, vv[i].y, o[2 * i + 1] * f);
        }
    }
    uint32_t *to = reinterpret_cast<uint32_t *>(p.out + item * D);
#pragma unroll
    for (int i = 0; i < kEach / 2; i++) to[lane + 32 * i] = Half2<E>::pack(o[2 * i] / l, o[2 * i + 1] / l);
}

}  // namespace

int64_t paged_attention_workspace(int, int, int, int, int, int) { return 0; }

cudaError_t launch_paged_attention(const PagedAttentionArgs &a)
{
    AttendParams p;
    p.q = (const uint16_t *)a.q; p.q_stride = a.q_stride;
    p.cu = a.cu_seqlens; p.starts = a.starts; p.slots = a.slots;
    p.groups = a.groups; p.prefix_lens = a.prefix_lens; p.prefix_slots = a.prefix_slots;
    p.cache = a.cache; p.out = (uint16_t *)a.out;
    p.N = a.N; p.T = a.T; p.P = a.P; p.Hq = a.Hq; p.Hk = a.Hk; p.G = a.Hq / a.Hk;
    p.scale_log2 = a.scale * kLog2e; p.err = a.err_word;
    const int64_t blocks = ((int64_t)a.T * a.Hq + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    auto *kernel = a.d == 128 ? (a.f16 ? attend_rows_kernel<__half, 128> : attend_rows_kernel<__nv_bfloat16, 128>)
                              : (a.f16 ? attend_rows_kernel<__half, 64> : attend_rows_kernel<__nv_bfloat16, 64>);
    kernel<<<(unsigned)blocks, kWarps * 32, 0, a.stream>>>(p);
    return cudaGetLastError();
}

}  // namespace kda
