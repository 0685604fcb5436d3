// kda_beam.cu -- one selection step of beam search.
//
//     candidate (b, t) of a prompt:  scores[b] + x_bt - log sum_u exp(x_bu)
//
// The best B of a prompt's B V candidates, with one pass over the logits, which bound
// it by HBM.  Within a row the order of the candidates is that of the logits, so the
// first kernel needs no normaliser: a CTA takes a slice of one row, and writes the
// slice's best B and its maximum and sum of exponentials.  The second, one CTA a prompt,
// joins the sums, compares what is left of the candidates and gives the children their
// slots.  Candidates of different beams may lie close together: they are compared as
// unevaluated sums of two fp32 numbers (the card's fp64 rate, a 64th of fp32's, made this
// kernel take 23-37 us in fp64).
//
// The best B of many values: the values fall into at least B groups; the smallest of the
// groups' maxima has at least B values at or above it, and mostly few more (B groups of equal
// size: about B ln B).  In a slice threads make up the groups, and only those whose own
// maximum reaches it look at their values again and collect the ones that do, which are
// ranked by counting.  Where equal or unevenly spread values make them too many, B rounds of
// a maximum below the one before find the same.  A prompt's candidates, where they are
// few, go the same way; where they are many, or too many of them are collected, the best of
// the slices' sorted lists is taken B times.  Ties go to the lowest index either way.
//
// On a GB300, captured: 16 prompts of 8 beams and 131,072 16-bit logits 21 us a call (of 28 MB, 4 us); one
// prompt of 4 beams and 32,000 logits 8.5 us, of 16, 32, 64 beams 24, 58, 119: latencies, one
// after the other.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "kda.h"
#include "kda_paged.h"
#include "kda_pdl.cuh"
#include "kda_tiles.cuh"

namespace kda {
namespace {

using tiles::add2;
using tiles::fma2;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kAtOnce = 4;                   // 16-byte loads of a thread on their way
constexpr int kLeast = 2048, kLongest = 32768;   // logits of a slice
// Candidates that are ranked by counting, of a slice and of a prompt.  Of 64 beams the bound leaves 266 on
// average and more than 520 in 2 % of the cases (a slice's rounds are long, and a call has many slices); a slice that
// leaves one of 64 groups without a value has 63 vectors of 8 logits and 7 single ones at most.
constexpr int kMost = 1024, kMostChosen = 520;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct BeamParams {
    const void *logits;
    int64_t row_stride;
    const float *scores;
    const int32_t *ended, *slots;
    int end_token;
    float *scores_out;
    int32_t *parents, *tokens, *ended_out, *new_slots, *src, *dst;
    uint64_t *best;                  // [G * B][slices][B]: keys, best first, 0 behind the last
    float2 *sums;                    // [G * B][slices]: maximum, sum of exponentials relative to it
    int G, B, V, slices, slice;      // slice: logits of one, a multiple of kLeast
    int groups;                      // of threads, whose maxima bound the best: at least B
};

// A number that grows with the value, and back.
__device__ __forceinline__ uint32_t rank_of(float x)
{
    const uint32_t b = __float_as_uint(x + 0.f);         // -0 and 0 are equal
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_at(uint32_t rank)
{
    return __uint_as_float(rank & 0x80000000u ? rank & 0x7fffffffu : ~rank);
}

// A logit and its token as a number that is larger for a better candidate; 0 for none.
__device__ __forceinline__ uint64_t key_of(float x, int token)
{
    return x > -INFINITY ? (uint64_t)rank_of(x) << 32 | (uint32_t)~token : 0;
}
__device__ __forceinline__ float value_of(uint64_t key) { return value_at((uint32_t)(key >> 32)); }
__device__ __forceinline__ int token_of(uint64_t key) { return (int)~(uint32_t)key; }

// a + b = s + e exactly
__device__ __forceinline__ float two_sum(float a, float b, float &e)
{
    const float s = __fadd_rn(a, b), t = __fadd_rn(s, -a);
    e = __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -t)), __fadd_rn(b, -t));
    return s;
}

// log l of l > 0 as a sum of two numbers, off by some 2^-25: l = 2^k f with f in [2^-1/2, 2^1/2],
// and what fp32 leaves of f by the logarithm's slope
__device__ __forceinline__ float2 log_of(double l)
{
    const float top = (float)l;
    int k;
    float f = frexpf(top, &k);                           // in [1/2, 1)
    if (f < 0.70710678f) f *= 2.f, k--;
    const double y = (double)k * 0.6931471805599453 + ((double)logf(f) + (l - (double)top) / (double)top);
    const float hi = (float)y;
    return make_float2(hi, (float)(y - (double)hi));
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two values of 16 bytes of logits at a time (of 32 bits: one): unpacked, and the larger ones of
// two words (without NaN).
template <typename E> struct Vec;
template <> struct Vec<float> {
    static constexpr int kN = 4;
    static constexpr uint32_t kLowest = 0xff800000u;     // -inf
    static __device__ __forceinline__ void up(const uint4 &v, float *x)
    {
        x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b)
    {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }
    static __device__ __forceinline__ float largest(uint32_t w) { return __uint_as_float(w); }
    static __device__ __forceinline__ float one(float x) { return x; }
};
template <typename E2> __device__ __forceinline__ uint32_t larger2(uint32_t a, uint32_t b)
{
    const E2 m = __hmax2(*reinterpret_cast<const E2 *>(&a), *reinterpret_cast<const E2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&m);
}
template <> struct Vec<__nv_bfloat16> {
    static constexpr int kN = 8;
    static constexpr uint32_t kLowest = 0xff80ff80u;
    static __device__ __forceinline__ void up(const uint4 &v, float *x)
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return larger2<__nv_bfloat162>(a, b); }
    static __device__ __forceinline__ float largest(uint32_t w)
    {
        return fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ float one(__nv_bfloat16 x) { return __bfloat162float(x); }
};
template <> struct Vec<__half> {
    static constexpr int kN = 8;
    static constexpr uint32_t kLowest = 0xfc00fc00u;
    static __device__ __forceinline__ void up(const uint4 &v, float *x)
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return larger2<__half2>(a, b); }
    static __device__ __forceinline__ float largest(uint32_t w)
    {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        return fmaxf(f.x, f.y);
    }
    static __device__ __forceinline__ float one(__half x) { return __half2float(x); }
};

// whether beam (of all) has candidates from its logits
__device__ __forceinline__ bool extends(const BeamParams &p, int beam)
{
    return p.scores[beam] > -INFINITY && !(p.ended && p.ended[beam]);
}

// A row of logits in vectors of 16 bytes from its first one on, wherever in memory it begins: which
// logits a thread has, and so the order of the row's sum, are the same for equal rows, whose
// candidates have to be equal.  kShifted: it may begin inside 16 bytes (20 registers more).
template <typename E, bool kShifted> struct Row {
    static constexpr int kN = Vec<E>::kN;
    const E *row;
    const uint4 *body;               // the 16 bytes in which the row begins,
    int shift;                       // at this byte of them
    int last;                        // the last vector whose bytes lie in two pieces of 16 that are all the row's
    __device__ Row(const BeamParams &p, int beam)
    {
        row = (const E *)p.logits + (int64_t)beam * p.row_stride;
        shift = (int)((uintptr_t)row & 15);
        body = reinterpret_cast<const uint4 *>((uintptr_t)row - shift);
        last = (int)(((int64_t)p.V * (int)sizeof(E) + shift) / 16) - 2;
    }
    // vectors v, v + kThreads, ...: those below end
    __device__ __forceinline__ void load(int v, int end, uint4 (&r)[kAtOnce]) const
    {
        const uint32_t none = Vec<E>::kLowest;
        if (!kShifted || shift == 0) {
#pragma unroll
            for (int i = 0; i < kAtOnce; i++)
                r[i] = v + i * kThreads < end ? __ldg(body + v + i * kThreads) : make_uint4(none, none, none, none);
        } else if (shift < 4) {
            load_shifted<0>(v, end, r);
        } else if (shift < 8) {
            load_shifted<1>(v, end, r);
        } else if (shift < 12) {
            load_shifted<2>(v, end, r);
        } else {
            load_shifted<3>(v, end, r);
        }
    }
    // kWords: 32-bit words of a piece before the row begins
    template <int kWords> __device__ __forceinline__ void load_shifted(int v, int end, uint4 (&r)[kAtOnce]) const
    {
        if (v >= 1 && v + (kAtOnce - 1) * kThreads < min(end, last + 1)) {
            uint4 next[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; i++) {
                r[i] = __ldg(body + v + i * kThreads);
                next[i] = first_words<kWords + 1>(body + v + i * kThreads + 1);
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; i++) r[i] = joined<kWords>(r[i], next[i]);
            return;
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; i++) {
            const int at = v + i * kThreads;
            const uint32_t none = Vec<E>::kLowest;
            if (at >= end) r[i] = make_uint4(none, none, none, none);
            else if (at >= 1 && at <= last) r[i] = joined<kWords>(__ldg(body + at), first_words<kWords + 1>(body + at + 1));
            else r[i] = single(at);
        }
    }
    template <int n> static __device__ __forceinline__ uint4 first_words(const uint4 *x)
    {
        if (n == 1) return make_uint4(__ldg(reinterpret_cast<const uint32_t *>(x)), 0, 0, 0);
        if (n == 2) {
            const uint2 y = __ldg(reinterpret_cast<const uint2 *>(x));
            return make_uint4(y.x, y.y, 0, 0);
        }
        return __ldg(x);
    }
    // the 16 bytes of a, then b, from `shift` on
    template <int kWords> __device__ __forceinline__ uint4 joined(const uint4 &a, const uint4 &b) const
    {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        const int bits = (shift & 2) * 8;
        return make_uint4(__funnelshift_r(w[kWords], w[kWords + 1], bits), __funnelshift_r(w[kWords + 1], w[kWords + 2], bits),
                          __funnelshift_r(w[kWords + 2], w[kWords + 3], bits), __funnelshift_r(w[kWords + 3], w[kWords + 4], bits));
    }
    // a vector, logit by logit: one at an end of the row, which may be that of the memory
    __device__ __forceinline__ uint4 single(int v) const
    {
        if (sizeof(E) == 4) {
            const uint32_t *x = reinterpret_cast<const uint32_t *>(row) + v * kN;
            return make_uint4(__ldg(x), __ldg(x + 1), __ldg(x + 2), __ldg(x + 3));
        }
        const uint16_t *x = reinterpret_cast<const uint16_t *>(row) + v * kN;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) w[i] = __ldg(x + 2 * i) | (uint32_t)__ldg(x + 2 * i + 1) << 16;
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <typename E, bool kShifted>
__global__ void __launch_bounds__(kThreads) slice_kernel(const __grid_constant__ BeamParams p)
{
    constexpr int kN = Vec<E>::kN;
    __shared__ uint64_t found[kMost], best_w[kWarps];
    __shared__ float top_w[kWarps], sum_w[kWarps], wide_w[kWarps][32];
    __shared__ int count;
    grid_go_on();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int beam = blockIdx.x / p.slices, slice = blockIdx.x - beam * p.slices;
    if (!extends(p, beam)) return;
    if (tid == 0) count = 0;
    const Row<E, kShifted> row(p, beam);
    const int vecs = p.V / kN, behind = p.V - vecs * kN;
    const int first = slice * (p.slice / kN) + tid, end = min(vecs, (slice + 1) * (p.slice / kN));
    // the few logits behind the vectors are the first slice's, one to a thread
    const int odd = slice == 0 && tid < behind ? vecs * kN + tid : -1;
    const float single = odd >= 0 ? Vec<E>::one(row.row[odd]) : -INFINITY;

    // the thread's maximum (without NaN) and the sum of exponentials relative to it, or to
    // 0 where nothing is finite; a NaN among the logits makes the sum NaN, and with it the
    // row's normaliser
    float top = single, sum = ex2(single > -INFINITY ? 0.f : single), base = 0.f, base2 = 0.f;
    if (top > -INFINITY) base = top, base2 = base * kLog2e;
    for (int v = first; v < end; v += kAtOnce * kThreads) {
        uint4 r[kAtOnce];
        row.load(v, end, r);
        uint32_t most = Vec<E>::kLowest;
#pragma unroll
        for (int i = 0; i < kAtOnce; i++)
            most = Vec<E>::larger(Vec<E>::larger(Vec<E>::larger(r[i].x, r[i].y), Vec<E>::larger(r[i].z, r[i].w)), most);
        const float high = Vec<E>::largest(most);
        if (high > top) {
            if (top > -INFINITY) sum *= ex2((top - high) * kLog2e);
            base = top = high;
            base2 = base * kLog2e;
        }
        if (fabsf(base) < 1024.f) {                      // a paired instruction for two exponents
            float2 part = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kAtOnce; i++) {
                float x[kN];
                Vec<E>::up(r[i], x);
#pragma unroll
                for (int j = 0; j < kN; j += 2) {
                    float2 e = fma2(make_float2(x[j], x[j + 1]), make_float2(kLog2e, kLog2e), make_float2(-base2, -base2));
                    e.x = ex2(e.x);
                    e.y = ex2(e.y);
                    part = add2(part, e);
                }
            }
            // what base2 was rounded by, at most 2^-14, is in every exponent
            const float all = part.x + part.y;
            sum += fmaf(all, -kLn2 * fmaf(base, kLog2e, -base2), all);
        } else {
#pragma unroll
            for (int i = 0; i < kAtOnce; i++) {
                float x[kN];
                Vec<E>::up(r[i], x);
#pragma unroll
                for (int j = 0; j < kN; j++) sum += ex2((x[j] - base) * kLog2e);
            }
        }
    }

    // Thread i is in group i % groups, so that a short slice, whose values the first threads have, leaves no
    // group without one.  (With neighbouring lanes a group, short slices went through rounds: one prompt of 8 beams
    // and 1300 16-bit logits took 13.5 us for 9.4, 16 prompts of 8 beams and 32,000 22 for 12.4.)
    float wide = top;
    for (int o = p.groups; o < 32; o *= 2) wide = fmaxf(wide, __shfl_xor_sync(0xffffffffu, wide, o));
    wide_w[warp][lane] = wide;
    float high = wide;
#pragma unroll
    for (int o = 16; o > 0; o /= 2) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
    if (top > -INFINITY) sum *= ex2((top - high) * kLog2e);
#pragma unroll
    for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
        top_w[warp] = high;
        sum_w[warp] = sum;
    }
    __syncthreads();
    float even = wide_w[0][lane], uneven = wide_w[1][lane];          // groups lane and lane + 32, or both halves of one
#pragma unroll
    for (int w = 2; w < kWarps; w += 2) {
        even = fmaxf(even, wide_w[w][lane]);
        uneven = fmaxf(uneven, wide_w[w + 1][lane]);
    }
    float bound = p.groups > 32 ? fminf(even, uneven) : fmaxf(even, uneven);
#pragma unroll
    for (int o = 16; o > 0; o /= 2) bound = fminf(bound, __shfl_xor_sync(0xffffffffu, bound, o));
    const int64_t at = (int64_t)beam * p.slices + slice;
    if (tid == 0) {
        float m = top_w[0], l = 0.f;
#pragma unroll
        for (int w = 1; w < kWarps; w++) m = fmaxf(m, top_w[w]);
#pragma unroll
        for (int w = 0; w < kWarps; w++) l += top_w[w] > -INFINITY ? sum_w[w] * ex2((top_w[w] - m) * kLog2e) : sum_w[w];
        p.sums[at] = make_float2(m, l);
    }
    // every value of the thread's, once more, with its token
    auto each = [&](auto &&use) {
        if (odd >= 0) use(single, odd);
        for (int v = first; v < end; v += kAtOnce * kThreads) {
            uint4 r[kAtOnce];
            row.load(v, end, r);
#pragma unroll
            for (int i = 0; i < kAtOnce; i++) {
                if (v + i * kThreads >= end) break;
                float x[kN];
                Vec<E>::up(r[i], x);
#pragma unroll
                for (int j = 0; j < kN; j++) use(x[j], (v + i * kThreads) * kN + j);
            }
        }
    };
    if (top >= bound && top > -INFINITY)
        each([&](float x, int token) {
            if (x >= bound && x > -INFINITY) {
                const int k = atomicAdd(&count, 1);
                if (k < kMost) found[k] = key_of(x, token);
            }
        });
    __syncthreads();
    uint64_t *to = p.best + at * p.B;
    const int n = count;
    if (n <= kMost) {
        for (int i = tid; i < max(n, p.B); i += kThreads) {
            if (i >= n) {
                to[i] = 0;
                continue;
            }
            const uint64_t mine = found[i];
            int rank = 0;
            for (int j = 0; j < n; j++) rank += found[j] > mine;
            if (rank < p.B) to[rank] = mine;
        }
        return;
    }
    uint64_t last = ~(uint64_t)0;
    for (int k = 0; k < p.B; k++) {
        uint64_t mine = 0;
        each([&](float x, int token) {
            const uint64_t key = key_of(x, token);
            if (key < last && key > mine) mine = key;
        });
#pragma unroll
        for (int o = 16; o > 0; o /= 2) {
            const uint64_t other = __shfl_xor_sync(0xffffffffu, mine, o);
            mine = other > mine ? other : mine;
        }
        __syncthreads();
        if (lane == 0) best_w[warp] = mine;
        __syncthreads();
        last = best_w[0];
#pragma unroll
        for (int w = 1; w < kWarps; w++) last = best_w[w] > last ? best_w[w] : last;
        if (tid == 0) to[k] = last;
    }
}

// A candidate of a prompt.  Those of a beam are in the order of their keys, which also tells
// logits apart that are equal beside the normaliser.
struct Candidate {
    uint64_t score;                  // ranks of the score's two parts, 0 for none
    uint64_t key;
    int beam;
};
__device__ __forceinline__ bool better(const Candidate &a, const Candidate &b)
{
    if (a.score != b.score) return a.score > b.score;
    return a.beam != b.beam ? a.beam < b.beam : a.key > b.key;
}

// The best of a converged warp's, in every lane.
__device__ __forceinline__ Candidate best_of(const Candidate &c)
{
    const uint32_t all = 0xffffffffu, high = (uint32_t)(c.score >> 32), top = __reduce_max_sync(all, high);
    bool in = high == top;
    const uint32_t low = __reduce_max_sync(all, in ? (uint32_t)c.score : 0);
    in = in && (uint32_t)c.score == low;
    const int beam = __reduce_min_sync(all, in ? c.beam : 0x7fffffff);
    in = in && c.beam == beam;
    const uint32_t value = __reduce_max_sync(all, in ? (uint32_t)(c.key >> 32) : 0);
    in = in && (uint32_t)(c.key >> 32) == value;
    const uint32_t token = __reduce_max_sync(all, in ? (uint32_t)c.key : 0);
    return {(uint64_t)top << 32 | low, (uint64_t)value << 32 | token, beam};
}

constexpr int kMaxBeams = 64;
// Candidates of a beam up to which a prompt's are looked at all, twice: some 1.2 us for each 256 of the prompt,
// as much as one of B rounds over the lists' first ones takes.  One prompt of 16 beams: 128 of a beam 18.8 us a call
// and 22.7 in rounds, 256 29.4 and 23.9; of 64 beams, 256 122 and 84, 1024 227 and 119.
constexpr int kFew = 128;

__global__ void __launch_bounds__(kThreads) select_kernel(const __grid_constant__ BeamParams p)
{
    extern __shared__ uint8_t taken[];                   // of each list: candidates that are among the best already
    __shared__ Candidate found[kMostChosen], best_w[2][kWarps], best[kMaxBeams];
    __shared__ float2 lse[kMaxBeams];
    __shared__ float score[kMaxBeams];
    __shared__ uint32_t low_w[kWarps];
    __shared__ int count;
    __shared__ int kind[kMaxBeams];                      // 0 no hypothesis, 1 extends, 2 ended
    __shared__ int parent[kMaxBeams], slot[kMaxBeams];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = p.B, first = blockIdx.x * B;
    const int lists = B * p.slices;                      // of a beam's slices, one beam after the other
    if (tid == 0) count = 0;
    if (tid < B) {
        const float s = p.scores[first + tid];
        kind[tid] = s > -INFINITY ? (p.ended && p.ended[first + tid] ? 2 : 1) : 0;
        score[tid] = s;
        slot[tid] = p.slots ? p.slots[first + tid] : -1;
    }
    grid_wait();
    __syncthreads();
    for (int b = warp; b < B; b += kWarps) {
        if (kind[b] != 1) continue;
        const float2 *sums = p.sums + (int64_t)(first + b) * p.slices;
        float m = -INFINITY;
        for (int s = lane; s < p.slices; s += 32) m = fmaxf(m, __ldcg(&sums[s].x));
#pragma unroll
        for (int o = 16; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        double l = 0.0;
        for (int s = lane; s < p.slices; s += 32) {
            const float2 v = __ldcg(&sums[s]);
            l += v.x > -INFINITY ? v.y * expf(v.x - m) : v.y;
        }
#pragma unroll
        for (int o = 16; o > 0; o /= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane == 0) {
            const float2 y = log_of(l);
            float e;
            const float s = two_sum(m, y.x, e);
            lse[b] = make_float2(s, e + y.y);            // not finite where m or l is not
        }
    }
    __syncthreads();
    // candidate n of list i, which is slice s of beam b
    auto candidate = [&](int i, int b, int s, int n) {
        Candidate c = {0, 0, b};
        float high = -INFINITY, low = 0.f;
        if (kind[b] == 2 && s == 0 && n == 0) {
            high = score[b];
            c.key = key_of(0.f, p.end_token);
        } else if (kind[b] == 1 && n < B) {
            c.key = __ldcg(p.best + ((int64_t)first * p.slices + i) * B + n);
            if (c.key) {
                float e1, e2;
                const float2 z = lse[b];
                const float sum = two_sum(two_sum(score[b], value_of(c.key), e1), -z.x, e2), rest = e1 + (e2 - z.y);
                high = sum + rest;                       // (NaN where the normaliser is)
                low = rest - (high - sum);
                if (isinf(sum)) high = sum, low = 0.f;
                if (z.x != z.x || isinf(z.x)) high = -INFINITY;
            }
        }
        if (high > -INFINITY) c.score = (uint64_t)rank_of(high) << 32 | rank_of(low);   // (not NaN)
        return c;
    };
    int n = kMostChosen + 1;
    if (B * p.slices <= kFew) {
        // The groups, whose maxima bound the best, shall get beams, slices and ranks alike.  Of one slice a beam, the
        // places of a rank move on by one beam with each rank; of several, place e holds the candidate of a scattered
        // number: odd factors and shifts are one to one below a power of two.  (33 logits of 64 beams, 48 us a
        // call, took 74 scattered; 32,000 of 16, 24 us, 177 in the other way.)
        const int all = lists * B, bits = 32 - __clz(all - 1), places = p.slices == 1 ? all : 1 << bits;
        auto placed = [&](int e) {
            const uint32_t mask = places - 1, h = (bits + 1) / 2;
            uint32_t x = (uint32_t)e * 0x9e3779b1u & mask;
            x = (x ^ x >> h) * 0x85ebca6bu & mask;
            x ^= x >> h;
            if (e >= places || (p.slices > 1 && x >= all)) return Candidate{0, 0, 0};
            if (p.slices == 1) {
                const int n = e / B, b = e % B + n;
                return candidate(b - (b < B ? 0 : B), b - (b < B ? 0 : B), 0, n);
            }
            const int i = x / B, b = i / p.slices;
            return candidate(i, b, i - b * p.slices, x - i * B);
        };
        const int place0 = lane * kWarps + warp;         // (few places: some for every warp)
        uint32_t top = 0;
        constexpr int kKept = 4;
        Candidate kept[kKept];                           // the thread's first ones
#pragma unroll
        for (int i = 0; i < kKept; i++) {
            kept[i] = i * kThreads < places ? placed(place0 + i * kThreads) : Candidate{0, 0, 0};
            top = max(top, (uint32_t)(kept[i].score >> 32));
        }
        for (int e = place0 + kKept * kThreads; e < places; e += kThreads) top = max(top, (uint32_t)(placed(e).score >> 32));
        for (int o = 1; o < kThreads / p.groups; o *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = __reduce_min_sync(0xffffffffu, top);
        if (lane == 0) low_w[warp] = top;
        __syncthreads();
        uint32_t bound = low_w[0];
#pragma unroll
        for (int w = 1; w < kWarps; w++) bound = min(bound, low_w[w]);
        auto collect = [&](const Candidate &c) {
            if (c.score && (uint32_t)(c.score >> 32) >= bound) {
                const int k = atomicAdd(&count, 1);
                if (k < kMostChosen) found[k] = c;
            }
        };
#pragma unroll
        for (int i = 0; i < kKept; i++) collect(kept[i]);
        for (int e = place0 + kKept * kThreads; e < places; e += kThreads) collect(placed(e));
        __syncthreads();
        n = count;
    }
    if (n <= kMostChosen) {
        // eight lanes count for a candidate
        for (int i0 = tid / 8; i0 - tid / 8 < max(n, B); i0 += kThreads / 8) {
            const bool there = i0 < n;
            const Candidate mine = there ? found[i0] : Candidate{0, 0, 0};
            int rank = 0;
            if (there)
                for (int j = tid % 8; j < n; j += 8) {
                    const uint64_t other = found[j].score;
                    rank += other > mine.score || (other == mine.score && better(found[j], mine));
                }
#pragma unroll
            for (int o = 4; o > 0; o /= 2) rank += __shfl_xor_sync(0xffffffffu, rank, o);
            if (tid % 8 == 0) {
                if (there && rank < B) best[rank] = mine;
                if (!there && i0 < B) best[i0] = {0, 0, 0};
            }
        }
    } else {
        // B times the best of the lists' first candidates: a thread has every 256th list
        for (int i = tid; i < lists; i += kThreads) taken[i] = 0;
        const int b0 = tid / p.slices, s0 = tid - b0 * p.slices, db = kThreads / p.slices, ds = kThreads - db * p.slices;
        Candidate own, of_warp;                          // the best of the thread's lists, and of the warp's
        int list = 0;                                    // whose it is
        auto look = [&]() {
            own = {0, 0, B};
            for (int i = tid, b = b0, s = s0; i < lists; i += kThreads, b += db, s += ds) {
                if (s >= p.slices) s -= p.slices, b++;
                const Candidate c = candidate(i, b, s, taken[i]);
                if (c.score && better(c, own)) own = c, list = i;
            }
        };
        look();
        of_warp = best_of(own);
        for (int k = 0; k < B; k++) {
            if (lane == 0) best_w[k & 1][warp] = of_warp;
            __syncthreads();
            const Candidate next = best_of(best_w[k & 1][lane % kWarps]);
            if (tid == 0) best[k] = next;
            const bool is_own = next.score && own.score == next.score && own.beam == next.beam && own.key == next.key;
            if (is_own) {
                taken[list]++;
                look();
            }
            if (__any_sync(0xffffffffu, is_own)) of_warp = best_of(own);
        }
    }
    __syncthreads();
    if (tid >= kMaxBeams) return;                        // the first two warps stay
    const bool mine = tid < B, live = mine && best[tid].score;
    if (mine) {
        const Candidate c = best[tid];
        const int from = live ? c.beam : -1, token = live ? token_of(c.key) : -1;
        parent[tid] = from;
        p.scores_out[first + tid] = live ? value_at((uint32_t)(c.score >> 32)) : -INFINITY;
        p.parents[first + tid] = from;
        p.tokens[first + tid] = token;
        if (p.ended_out) p.ended_out[first + tid] = live && (kind[from] == 2 || token == p.end_token);
    }
    if (!p.slots) return;
    asm volatile("bar.sync 1, 64;" ::: "memory");
    // bit b: beam b has a child; bit k: child k moves
    uint64_t parents = 0;
    bool moving = mine && !live;
    for (int j = 0; j < B; j++) {
        const int from = parent[j];
        if (from >= 0) parents |= (uint64_t)1 << from;
        moving = moving || (mine && j < tid && from == parent[tid]);
    }
    __shared__ uint32_t moves[2];
    const uint32_t vote = __ballot_sync(0xffffffffu, moving);
    if (lane == 0) moves[warp] = vote;
    asm volatile("bar.sync 1, 64;" ::: "memory");
    if (!mine) return;
    const int from = live ? slot[parent[tid]] : -1;
    int to = from;
    if (moving) {                                        // the n-th of them: the n-th beam without a child
        const uint64_t before = (((uint64_t)moves[1] << 32 | moves[0])) & (((uint64_t)1 << tid) - 1);
        uint64_t free_beams = ~parents;
        for (int k = __popcll(before); k > 0; k--) free_beams &= free_beams - 1;
        to = slot[__ffsll(free_beams) - 1];
    }
    p.new_slots[first + tid] = to;
    p.src[first + tid] = from;
    p.dst[first + tid] = moving && live ? to : -1;
}

// Logits of a slice: enough slices to fill the card four times over where the rows are few,
// and no slice longer than kLongest.
int slice_of(int rows, int V)
{
    const int64_t want = ((int64_t)rows * V / 608 + kLeast - 1) / kLeast * kLeast;
    return (int)(want < kLeast ? kLeast : want > kLongest ? kLongest : want);
}
int slices_of(int rows, int V)
{
    const int slice = slice_of(rows, V);
    return V <= slice ? 1 : (V + slice - 1) / slice;
}

}  // namespace

int64_t beam_workspace(int G, int B, int V)
{
    if (G < 1 || B < 1 || B > kMaxBeams || V < 1 || V > (1 << 24) || (int64_t)G * B > (1 << 20)) return -1;
    const int64_t parts = (int64_t)G * B * slices_of(G * B, V);
    return parts > 0x7fffffff ? -1 : parts * (B + 1) * 8;
}

cudaError_t launch_beam_select(const BeamArgs &a)
{
    BeamParams p;
    p.logits = a.logits; p.row_stride = a.row_stride;
    p.scores = a.scores; p.ended = a.ended; p.slots = a.slots; p.end_token = a.end_token;
    p.scores_out = a.scores_out; p.parents = a.parents; p.tokens = a.tokens; p.ended_out = a.ended_out;
    p.new_slots = a.new_slots; p.src = a.src; p.dst = a.dst;
    p.G = a.G; p.B = a.B; p.V = a.V;
    p.slice = slice_of(a.G * a.B, a.V);
    p.slices = slices_of(a.G * a.B, a.V);
    p.groups = kWarps;
    while (p.groups < a.B) p.groups *= 2;
    const int64_t parts = (int64_t)a.G * a.B * p.slices;
    p.best = (uint64_t *)a.workspace;
    p.sums = (float2 *)(p.best + parts * a.B);
    const bool shifted = (((uintptr_t)a.logits | (uint64_t)a.row_stride * (a.dtype == KDA_F32 ? 4 : 2)) & 15) != 0;
    auto *kernel = a.dtype == KDA_F32 ? (shifted ? slice_kernel<float, true> : slice_kernel<float, false>)
                   : a.dtype == KDA_F16 ? (shifted ? slice_kernel<__half, true> : slice_kernel<__half, false>)
                                        : (shifted ? slice_kernel<__nv_bfloat16, true> : slice_kernel<__nv_bfloat16, false>);
    kernel<<<(unsigned)parts, kThreads, 0, a.stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.G);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)(a.B * p.slices);     // at most 64 x 512
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, select_kernel, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace kda
