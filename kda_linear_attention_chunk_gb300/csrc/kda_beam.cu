// kda_beam.cu -- one selection step of beam search.
//
//     candidate (b, t) of a prompt:  scores[b] + x_bt - log sum_u exp(x_bu)
//
// The best B of a prompt's B V candidates, with one pass over the logits, which bound
// it by HBM.  Within a row the order of the candidates is that of the logits, so the
// first kernel needs no normaliser: a CTA holds kSlice logits of one row in registers,
// and writes their best B and their maximum and sum of exponentials.  The second, one
// CTA a prompt, joins the sums (fp64), compares what is left of the candidates in fp64,
// where different beams' may lie close together, and gives the children their slots.
//
// The best B of many values: the values fall into at least B groups by threads; the
// smallest of the groups' maxima has at least B values at or above it, and mostly few
// more (B groups of equal size: about B ln B).  Those are collected and ranked by
// counting.  Where equal or unevenly spread values make them too many, B rounds of a
// maximum below the one before find the same.  Ties go to the lowest index either way.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "kda.h"
#include "kda_paged.h"
#include "kda_pdl.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kEach = 32;                    // logits of a thread
constexpr int kSlice = kThreads * kEach;
constexpr int kMost = 512;                   // candidates that are ranked by counting
constexpr float kLog2e = 1.4426950408889634f;

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
    int G, B, V, slices, spread;     // spread: lanes of a group
};

// A value and its token as a number that is larger for a better candidate; 0 for none.
__device__ __forceinline__ uint64_t key_of(float x, int token)
{
    if (!(x > -INFINITY)) return 0;
    const uint32_t b = __float_as_uint(x + 0.f);         // -0 and 0 are equal
    return (uint64_t)(b & 0x80000000u ? ~b : b | 0x80000000u) << 32 | (uint32_t)~token;
}
__device__ __forceinline__ float value_of(uint64_t key)
{
    const uint32_t b = (uint32_t)(key >> 32);
    return __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
}
__device__ __forceinline__ int token_of(uint64_t key) { return (int)~(uint32_t)key; }

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename E> struct Vec;    // 16 bytes of logits
template <> struct Vec<float> {
    static constexpr int kN = 4;
    static __device__ __forceinline__ void up(const uint4 &v, float *x)
    {
        x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ float one(float x) { return x; }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int kN = 8;
    static __device__ __forceinline__ void up(const uint4 &v, float *x)
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ float one(__nv_bfloat16 x) { return __bfloat162float(x); }
};
template <> struct Vec<__half> {
    static constexpr int kN = 8;
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
    static __device__ __forceinline__ float one(__half x) { return __half2float(x); }
};

// whether beam (of all) has candidates from its logits
__device__ __forceinline__ bool extends(const BeamParams &p, int beam)
{
    return p.scores[beam] > -INFINITY && !(p.ended && p.ended[beam]);
}

template <typename E>
__global__ void __launch_bounds__(kThreads) slice_kernel(const __grid_constant__ BeamParams p)
{
    constexpr int kN = Vec<E>::kN, kVecs = kEach / kN;
    __shared__ uint64_t found[kMost];
    __shared__ float top_w[kWarps], sum_w[kWarps], low_w[kWarps];
    __shared__ uint64_t best_w[kWarps];
    __shared__ int count;
    grid_go_on();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int beam = blockIdx.x / p.slices, slice = blockIdx.x - beam * p.slices;
    if (!extends(p, beam)) return;
    if (tid == 0) count = 0;
    // the row: elements before the first 16-byte boundary, vectors, elements behind them
    const E *row = (const E *)p.logits + (int64_t)beam * p.row_stride;
    const int before = min(p.V, (int)((16 - ((uintptr_t)row & 15)) & 15) / (int)sizeof(E));
    const int vecs = (p.V - before) / kN, behind = p.V - before - vecs * kN;
    const uint4 *body = reinterpret_cast<const uint4 *>(row + before);
    const int v0 = slice * (kSlice / kN) + tid;
    float x[kEach + 1];
#pragma unroll
    for (int i = 0; i < kVecs; i++) {
        const int v = v0 + i * kThreads;
        if (v < vecs) {
            Vec<E>::up(__ldcs(body + v), x + i * kN);
        } else {
#pragma unroll
            for (int j = 0; j < kN; j++) x[i * kN + j] = -INFINITY;
        }
    }
    // the few others are the first slice's, one to a thread
    int odd = -1;
    if (slice == 0) odd = tid < before ? tid : tid >= 32 && tid - 32 < behind ? before + vecs * kN + tid - 32 : -1;
    x[kEach] = odd >= 0 ? Vec<E>::one(row[odd]) : -INFINITY;
    auto token = [&](int i) { return i < kEach ? before + (v0 + i / kN * kThreads) * kN + i % kN : odd; };

    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i <= kEach; i++) top = fmaxf(top, x[i]);       // (without NaN)
    // (a NaN among the logits makes the sum NaN, and with it the row's normaliser)
    const float base = top > -INFINITY ? top : 0.f;
#pragma unroll
    for (int i = 0; i <= kEach; i++) sum += ex2((x[i] - base) * kLog2e);
    float wide = top;
    for (int o = 1; o < p.spread; o *= 2) wide = fmaxf(wide, __shfl_xor_sync(0xffffffffu, wide, o));
    float low = wide, high = wide;                       // of the warp's groups
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
        high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
    }
    if (top > -INFINITY) sum *= ex2((top - high) * kLog2e);
#pragma unroll
    for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
        top_w[warp] = high;
        sum_w[warp] = sum;
        low_w[warp] = low;
    }
    __syncthreads();
    float bound = low_w[0];
#pragma unroll
    for (int w = 1; w < kWarps; w++) bound = fminf(bound, low_w[w]);
    const int64_t at = (int64_t)beam * p.slices + slice;
    if (tid == 0) {
        float m = top_w[0], l = 0.f;
#pragma unroll
        for (int w = 1; w < kWarps; w++) m = fmaxf(m, top_w[w]);
#pragma unroll
        for (int w = 0; w < kWarps; w++) l += top_w[w] > -INFINITY ? sum_w[w] * ex2((top_w[w] - m) * kLog2e) : sum_w[w];
        p.sums[at] = make_float2(m, l);
    }
    if (top >= bound && top > -INFINITY) {
#pragma unroll
        for (int i = 0; i <= kEach; i++)
            if (x[i] >= bound && x[i] > -INFINITY) {
                const int k = atomicAdd(&count, 1);
                if (k < kMost) found[k] = key_of(x[i], token(i));
            }
    }
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
#pragma unroll
        for (int i = 0; i <= kEach; i++) {
            const uint64_t key = key_of(x[i], token(i));
            if (key < last && key > mine) mine = key;
        }
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
    double score;
    uint64_t key;
    int beam;
};
__device__ __forceinline__ bool better(const Candidate &a, const Candidate &b)
{
    if (a.score != b.score) return a.score > b.score;
    return a.beam != b.beam ? a.beam < b.beam : a.key > b.key;
}

constexpr int kMaxBeams = 64;

__global__ void __launch_bounds__(kThreads) select_kernel(const __grid_constant__ BeamParams p)
{
    __shared__ double lse[kMaxBeams], score[kMaxBeams], low_w[kWarps];
    __shared__ Candidate found[kMost], best_w[kWarps], best[kMaxBeams];
    __shared__ int kind[kMaxBeams];                      // 0 no hypothesis, 1 extends, 2 ended
    __shared__ int parent[kMaxBeams], slot[kMaxBeams];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = p.B, first = blockIdx.x * B;
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
            l += v.x > -INFINITY ? (double)v.y * exp((double)v.x - (double)m) : (double)v.y;
        }
#pragma unroll
        for (int o = 16; o > 0; o /= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane == 0) lse[b] = (double)m + log(l);
    }
    __syncthreads();
    const int per = p.slices * B, all = B * per;         // places of a beam's candidates
    // the candidate at place e; score -inf: none
    auto candidate = [&](int e) {
        const int b = e / per, at = e - b * per;
        Candidate c = {-INFINITY, 0, b};
        if (kind[b] == 2 && at == 0) {
            c.score = score[b];
            c.key = key_of(0.f, p.end_token);
        } else if (kind[b] == 1) {
            c.key = __ldcg(p.best + (int64_t)(first + b) * per + at);
            const double v = c.key ? score[b] + ((double)value_of(c.key) - lse[b]) : -INFINITY;
            if (v > -INFINITY) c.score = v;              // (not NaN)
        }
        return c;
    };
    double top = -INFINITY;
    for (int e = tid; e < all; e += kThreads) top = fmax(top, candidate(e).score);
    for (int o = 1; o < p.spread; o *= 2) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
    for (int o = 16; o > 0; o /= 2) top = fmin(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) low_w[warp] = top;
    __syncthreads();
    double bound = low_w[0];
#pragma unroll
    for (int w = 1; w < kWarps; w++) bound = fmin(bound, low_w[w]);
    for (int e = tid; e < all; e += kThreads) {
        const Candidate c = candidate(e);
        if (c.score >= bound && c.score > -INFINITY) {
            const int k = atomicAdd(&count, 1);
            if (k < kMost) found[k] = c;
        }
    }
    __syncthreads();
    const int n = count;
    if (n <= kMost) {
        for (int i = tid; i < max(n, B); i += kThreads) {
            if (i >= n) {
                best[i] = {-INFINITY, 0, 0};
                continue;
            }
            const Candidate mine = found[i];
            int rank = 0;
            for (int j = 0; j < n; j++) rank += better(found[j], mine);
            if (rank < B) best[rank] = mine;
        }
    } else {
        Candidate last = {INFINITY, 0, -1};
        for (int k = 0; k < B; k++) {
            Candidate mine = {-INFINITY, 0, B};
            for (int e = tid; e < all; e += kThreads) {
                const Candidate c = candidate(e);
                if (c.score > -INFINITY && better(last, c) && better(c, mine)) mine = c;
            }
#pragma unroll
            for (int o = 16; o > 0; o /= 2) {
                const Candidate other = {__shfl_xor_sync(0xffffffffu, mine.score, o), __shfl_xor_sync(0xffffffffu, mine.key, o),
                                         __shfl_xor_sync(0xffffffffu, mine.beam, o)};
                if (better(other, mine)) mine = other;
            }
            __syncthreads();
            if (lane == 0) best_w[warp] = mine;
            __syncthreads();
            last = best_w[0];
#pragma unroll
            for (int w = 1; w < kWarps; w++)
                if (better(best_w[w], last)) last = best_w[w];
            if (tid == 0) best[k] = last;
        }
    }
    __syncthreads();
    const bool live = tid < B && best[tid < B ? tid : 0].score > -INFINITY;
    if (tid < B) {
        const Candidate c = best[tid];
        const int from = live ? c.beam : -1, token = live ? token_of(c.key) : -1;
        parent[tid] = from;
        p.scores_out[first + tid] = (float)c.score;
        p.parents[first + tid] = from;
        p.tokens[first + tid] = token;
        if (p.ended_out) p.ended_out[first + tid] = live && (kind[from] == 2 || token == p.end_token);
    }
    if (!p.slots) return;
    __syncthreads();
    if (tid >= B) return;
    // the n-th child that moves takes the slot of the n-th beam without a child
    auto moves = [&](int k) {
        if (parent[k] < 0) return true;
        for (int j = 0; j < k; j++)
            if (parent[j] == parent[k]) return true;
        return false;
    };
    int to = live ? slot[parent[tid]] : -1;
    const int from = to;
    const bool moving = moves(tid);
    if (moving) {
        int nth = 0, b = 0;
        for (int j = 0; j < tid; j++) nth += moves(j);
        for (;; b++) {
            bool childless = true;
            for (int j = 0; j < B; j++) childless = childless && parent[j] != b;
            if (childless && nth-- == 0) break;
        }
        to = slot[b];
    }
    p.new_slots[first + tid] = to;
    p.src[first + tid] = from;
    p.dst[first + tid] = moving && live ? to : -1;
}

int slices_of(int V) { return V <= kSlice ? 1 : (V + kSlice - 1) / kSlice; }

}  // namespace

int64_t beam_workspace(int G, int B, int V)
{
    if (G < 1 || B < 1 || B > kMaxBeams || V < 1 || V > (1 << 24) || (int64_t)G * B > (1 << 20)) return -1;
    const int64_t parts = (int64_t)G * B * slices_of(V);
    return parts > 0x7fffffff ? -1 : parts * (B + 1) * 8;
}

cudaError_t launch_beam_select(const BeamArgs &a)
{
    BeamParams p;
    p.logits = a.logits; p.row_stride = a.row_stride;
    p.scores = a.scores; p.ended = a.ended; p.slots = a.slots; p.end_token = a.end_token;
    p.scores_out = a.scores_out; p.parents = a.parents; p.tokens = a.tokens; p.ended_out = a.ended_out;
    p.new_slots = a.new_slots; p.src = a.src; p.dst = a.dst;
    p.G = a.G; p.B = a.B; p.V = a.V; p.slices = slices_of(a.V);
    int groups = kWarps;                                 // at least B
    while (groups < a.B) groups *= 2;
    p.spread = kThreads / groups;
    const int64_t parts = (int64_t)a.G * a.B * p.slices;
    p.best = (uint64_t *)a.workspace;
    p.sums = (float2 *)(p.best + parts * a.B);
    auto *kernel = a.dtype == KDA_F32 ? slice_kernel<float>
                   : a.dtype == KDA_F16 ? slice_kernel<__half> : slice_kernel<__nv_bfloat16>;
    kernel<<<(unsigned)parts, kThreads, 0, a.stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.G);
    cfg.blockDim = dim3(kThreads);
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
