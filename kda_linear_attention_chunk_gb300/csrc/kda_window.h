// kda_window.h -- what the window-attention kernels share: the visible
// positions of a query and their rows in the ring cache.  Not installed.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "kda_common.cuh"
#include "kda_hybrid.h"
#include "kda_pdl.cuh"

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

struct WindowParams {
    const uint16_t *q, *k, *v;       // the call's rows
    int64_t q_stride, k_stride, v_stride;
    const int32_t *cu, *starts, *slots;   // starts: context lengths (decode: the tokens' positions)
    uint16_t *pool, *out;
    int N, T, Hq, Hk, num_slots, pool_rows, window, sinks;
    int G, tile_tokens;              // query heads per key head; tokens of a query tile
    int inv_G;                       // ceil(2^16 / G): r / G = r inv_G >> 16 for r < 128
    int items;                       // numbers of items, at least as many as there are
    int longer;                      // > 0: the batch is divided (divided() below)
    int groups;                      // groups of up to 16 query heads per key head (warp-MMA kernel)
    float scale_log2;
    int *err;
};

// The spans of `span` rows of a packed batch are numbered so that sequence n has the
// numbers from cu[n] / span + n on: at least as many as it has spans, without a
// pass over the table.  A sequence's facts:
struct Sequence {
    int cu0, cu1, start, slot;       // its two table entries, context length and slot, as they are
    int part;                        // the number's place among the sequence's spans (may be past its rows)
};

// The last sequence whose numbers start at or before `number`, by a converged warp:
// 32 probes at a time, the last of which bring the facts along.
__device__ __forceinline__ Sequence sequence_of(const WindowParams &p, int span, int number, int lane)
{
    int a = 0, n = p.N;              // the answer is in [a, a + n)
    while (n > 32) {
        const int step = (n + 31) / 32, at = a + lane * step;
        const bool le = lane * step < n && p.cu[at] / span + at <= number;
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, le || lane == 0));
        n = min(step, n - last * step);
        a += last * step;
    }
    const int at = a + min(lane, n - 1);
    Sequence s;
    s.cu0 = p.cu[at];
    s.cu1 = p.cu[at + 1];
    s.start = p.starts ? p.starts[at] : 0;
    s.slot = p.slots ? p.slots[at] : at;
    s.part = number - (s.cu0 / span + at);
    const int who = 31 - __clz(__ballot_sync(0xffffffffu, (lane < n && s.part >= 0) || lane == 0));
    s.cu0 = __shfl_sync(0xffffffffu, s.cu0, who);
    s.cu1 = __shfl_sync(0xffffffffu, s.cu1, who);
    s.start = __shfl_sync(0xffffffffu, s.start, who);
    s.slot = __shfl_sync(0xffffffffu, s.slot, who);
    s.part = __shfl_sync(0xffffffffu, s.part, who);
    return s;
}

// A divided batch: the tiles take the sequences of more than `longer` query rows a key
// head, the warp-MMA kernel the others.
__device__ __forceinline__ bool is_long(const WindowParams &p, int len) { return p.longer && (int64_t)len * p.G > p.longer; }

// spans of sequence n, if it is a long one
__device__ __forceinline__ int long_spans(const WindowParams &p, int span, int n)
{
    const int len = clamp_row(p.cu[n + 1], p.T, nullptr) - clamp_row(p.cu[n], p.T, nullptr);
    return is_long(p, len) ? (len - 1) / span + 1 : 0;
}

// The spans of the long sequences are numbered by lanes: first those of the sequences 0, 32,
// 64 and so on.  A lane's own, and those before:
struct LongSpans {
    int mine = 0, before = 0;
};
__device__ __forceinline__ LongSpans count_long(const WindowParams &p, int span, int lane)
{
    LongSpans s;
#pragma unroll 4
    for (int n = lane; n < p.N; n += 32) s.mine += long_spans(p, span, n);
    int end = s.mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int x = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end += x;
    }
    s.before = end - s.mine;
    return s;
}

// the sequence of a number, by a converged warp; part -1: there are fewer spans
__device__ __forceinline__ Sequence sequence_of_long(const WindowParams &p, int span, int number, int lane, const LongSpans &l)
{
    Sequence s = {0, 0, 0, 0, -1};
    const uint32_t whose = __ballot_sync(0xffffffffu, number >= l.before && number < l.before + l.mine);
    if (!whose) return s;
    const int first = __ffs(whose) - 1;
    int left = number - __shfl_sync(0xffffffffu, l.before, first);
    for (int base = first; base < p.N; base += 32 * 32) {
        const int n = base + 32 * lane, mine = n < p.N ? long_spans(p, span, n) : 0;
        int end = mine;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int x = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end += x;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, end > left);
        if (past) {
            const int who = __ffs(past) - 1, at = base + 32 * who;
            s.part = left - __shfl_sync(0xffffffffu, end - mine, who);
            s.cu0 = p.cu[at];
            s.cu1 = p.cu[at + 1];
            s.start = p.starts ? p.starts[at] : 0;
            s.slot = p.slots ? p.slots[at] : at;
            return s;
        }
        left -= __shfl_sync(0xffffffffu, end, 31);
    }
    return s;
}

// The rows that a span stands for, all checked; `reports`: whether this warp tells of
// entries out of range.
struct Rows {
    int bos, len, start, entry;      // the sequence's first row, rows, context length, cache entry
    int from, n;                     // the span's first row within the sequence, and its rows (0: none)
};
__device__ __forceinline__ Rows rows_in(const WindowParams &p, const Sequence &s, int span, int lane, bool reports)
{
    reports = reports && lane == 0 && s.part == 0;
    Rows r;
    r.bos = clamp_row(s.cu0, p.T, reports ? p.err : nullptr);
    r.len = max(0, clamp_row(s.cu1, p.T, reports ? p.err : nullptr) - r.bos);
    const int most = 0x7fffffff - r.len;
    r.start = min(max(s.start, 0), most);
    if (r.start != s.start && reports) atomicOr(p.err, kErrBadPosition);
    r.entry = s.slot;
    if (p.slots && (s.slot < 0 || s.slot >= p.num_slots)) {
        if (s.slot != -1 && reports) atomicOr(p.err, kErrBadSlot);
        r.entry = -1;
    }
    const int64_t from = (int64_t)s.part * span;
    r.n = s.part < 0 || from >= r.len || r.entry < 0 ? 0 : (int)min((int64_t)span, r.len - from);
    r.from = r.n ? (int)from : 0;
    return r;
}
__device__ __forceinline__ Rows rows_of(const WindowParams &p, int span, int number, int lane, bool reports)
{
    return rows_in(p, sequence_of(p, span, number, lane), span, lane, reports);
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

inline WindowParams window_params(const WindowArgs &a)
{
    WindowParams p = {};
    p.q = (const uint16_t *)a.q; p.k = (const uint16_t *)a.k; p.v = (const uint16_t *)a.v;
    p.q_stride = a.q_stride; p.k_stride = a.k_stride; p.v_stride = a.v_stride;
    p.cu = a.cu_seqlens; p.starts = a.starts; p.slots = a.slots;
    p.pool = (uint16_t *)a.pool; p.out = (uint16_t *)a.out;
    p.N = a.N; p.T = a.T; p.Hq = a.Hq; p.Hk = a.Hk; p.num_slots = a.num_slots; p.pool_rows = a.pool_rows;
    p.window = a.window; p.sinks = a.sinks;
    p.G = a.Hq / a.Hk;
    p.scale_log2 = a.scale * kLog2e;
    p.err = a.err_word;
    return p;
}

// The warp-MMA kernel for few rows a sequence (kda_window_rows.cu), without the
// writing of the cache; longer > 0: for a divided batch, behind the tiles' launch.
cudaError_t launch_window_rows(const WindowArgs &a, int longer);

}  // namespace kda
