// kda_paged_attention.cu -- attention over a paged cache with shared prefixes: the plan
// that cuts a call's work into parts, and the join of the pieces' results.
//
//     o = sum_j 2^(c s_j - c m) v_j / sum_j 2^(c s_j - c m),   s_j = q . k_j,  c = scale log2 e
//
// over pieces i of the keys with maxima m_i, sums l_i and outputs o_i:
//
//     m = max m_i,   o = sum_i 2^(c (m_i - m)) o_i / sum_i 2^(c (m_i - m)) l_i
//
// Four kernels: the plan (one CTA), the tiles and the rows kernel, and the join; each
// is launched early (programmatic dependent launch) and waits for what it needs.
#include <stdint.h>

#include "kda_paged_attend.cuh"

namespace kda {
namespace {

constexpr int kPlanThreads = 1024;

// the positions that group g shares, and whose pages they are in
struct Prefix {
    int len, entry;
};
__device__ __forceinline__ Prefix prefix_of(const AttendParams &p, int g, int *err)
{
    Prefix x;
    x.entry = entry_of(p.prefix_slots, g, p.cache.num_slots, p.err, err != nullptr);
    const int was = p.prefix_lens[g];
    x.len = x.entry < 0 ? 0 : min(max(was, 0), capacity(p.cache));
    if (err && x.entry >= 0 && x.len != was) atomicOr(err, kErrBadPosition);
    return x;
}
__device__ __forceinline__ int group_start(const AttendParams &p, int g) { return min(max(p.groups[g], 0), p.N); }

__device__ __forceinline__ Part make_part(const AttendParams &p, int i)
{
    Part x = {};
    x.prefix = -1;
    if (i < p.P) {
        const int a = group_start(p, i), b = group_start(p, i + 1);
        if (p.groups[i] != a || p.groups[i + 1] != b || a > b) atomicOr(p.err, kErrBadSeqlens);
        const Prefix y = prefix_of(p, i, p.err);
        x.t0 = p.cu ? clamp_row(p.cu[a], p.T, nullptr) : a;
        x.tokens = (p.cu ? clamp_row(p.cu[b], p.T, nullptr) : b) - x.t0;
        x.key1 = y.len;
        x.entry = y.entry;
    } else {
        const int n = i - p.P;
        int least = 0;
        x.entry = entry_of(p.slots, n, p.cache.num_slots, p.err, true);
        if (p.P) {
            int a = 0, b = p.P - 1;                      // the last group that starts at or before n
            while (a < b) {
                const int c = (a + b + 1) / 2;
                if (group_start(p, c) <= n) a = c; else b = c - 1;
            }
            if (group_start(p, a) <= n && n < group_start(p, a + 1)) {
                least = prefix_of(p, a, nullptr).len;
                if (least) x.prefix = a;
            }
        }
        if (x.entry >= 0) {
            const RowsAt r = rows_at(p.cu, p.starts, p.cache, n, p.T, least, p.err);
            x.t0 = r.bos;
            x.tokens = min(r.len, capacity(p.cache) - r.start);
            x.first = r.start;
            x.key0 = least;
            x.key1 = r.start + x.tokens;
        }
    }
    x.kind = x.tokens <= 0 || x.key1 <= x.key0 ? kNoWork : (int64_t)x.tokens * p.G <= kFewRows ? kRowsWork : kTilesWork;
    return x;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ AttendParams p)
{
    __shared__ int64_t sums[2][kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, all = p.P + p.N;
    grid_go_on();
    int64_t done[2] = {0, 0};                            // tiles and steps so far
    for (int base = 0; base < all; base += kPlanThreads) {
        const int i = base + tid;
        int64_t mine[2] = {0, 0};
        if (i < all) {
            const Part x = make_part(p, i);
            int4 *to = reinterpret_cast<int4 *>(p.parts + i);
            to[0] = make_int4(x.t0, x.tokens, x.first, x.key0);
            to[1] = make_int4(x.key1, x.entry, x.prefix, x.kind);
            if (x.kind == kTilesWork) mine[0] = part_tiles(x, i < p.P, 2 * p.tile_tokens);
            if (x.kind == kRowsWork) mine[1] = part_steps(x);
        }
        int64_t upto[2] = {mine[0], mine[1]};
#pragma unroll
        for (int k = 0; k < 2; k++) {
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int64_t y = __shfl_up_sync(0xffffffffu, upto[k], o);
                if (lane >= o) upto[k] += y;
            }
            if (lane == 31) sums[k][warp] = upto[k];
        }
        __syncthreads();
        if (warp < 2) {
            int64_t y = sums[warp][lane];
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int64_t z = __shfl_up_sync(0xffffffffu, y, o);
                if (lane >= o) y += z;
            }
            sums[warp][lane] = y;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; k++) {
            int64_t *to = k ? p.steps : p.tiles;
            if (i < all) to[i] = done[k] + upto[k] - mine[k] + (warp ? sums[k][warp - 1] : 0);
            done[k] += sums[k][kPlanThreads / 32 - 1];
        }
        __syncthreads();
    }
    if (tid == 0) {
        p.tiles[all] = done[0];
        p.steps[all] = done[1];
    }
}

// Joins the pieces of rows.  A CTA of eight warps takes one row of the batch and `heads`
// of its query heads; `team` warps share one head.
constexpr int kJoinWarps = 8;

// the pieces of one of a row's two parts
struct Pieces {
    const float *whole;              // if there is only one, with all keys
    const float2 *whole_ml;
    const float *cut;                // else the first worker's, and so on
    const float2 *cut_ml;
    int64_t apart, first;            // rows between two pieces; the first piece's row
    int64_t later;                   // and the second one's
    int n;                           // 0: there are none, or the row's answer is written
};

__device__ __forceinline__ Pieces pieces_of(const AttendParams &p, int part, const Part &x, int t, int hq, int which, bool alone)
{
    Pieces r = {};
    if (x.kind == kNoWork) return r;
    const bool shared = which == 1, tiles = x.kind == kTilesWork;
    const int hk = hq / p.G, g = hq - hk * p.G, i = t - x.t0, span = 2 * p.tile_tokens;
    const int64_t *before = tiles ? p.tiles : p.steps;
    const int64_t total = __ldcg(before + p.P + p.N);
    const int64_t share = tiles ? share_of(total, p.Hk, p.tile_workers, kLeastTiles)
                                : share_of(total, p.Hk, p.row_workers, kLeastSteps);
    int64_t begin = hk * total + __ldcg(before + part), end;
    int row;                                             // of the piece
    if (tiles) {
        const int j = i / span, u = i - j * span, q = u >= p.tile_tokens;
        begin += tiles_before(x, shared, span, j);
        end = begin + span_tiles(x, shared, span, j);
        row = q * kTileRows + (u - q * p.tile_tokens) * p.G + g;
    } else {
        end = begin + part_steps(x);
        row = i * p.G + g;
    }
    const int64_t w0 = begin / share, w1 = (end - 1) / share;
    if (w0 == w1) {
        if (alone) return r;
        r.whole = p.whole[which];
        r.whole_ml = p.whole_ml[which];
        r.first = (int64_t)t * p.Hq + hq;
        r.n = 1;
        return r;
    }
    const int rows = tiles ? kPieceRows : kFewRows;
    r.cut = tiles ? p.cut_tiles : p.cut_rows;
    r.cut_ml = tiles ? p.cut_tiles_ml : p.cut_rows_ml;
    r.first = cut_piece(w0, begin, w0 * share) * rows + row;
    r.later = 2 * (w0 + 1) * rows + row;
    r.apart = 2 * rows;
    r.n = (int)(w1 - w0 + 1);
    return r;
}

template <typename E, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ AttendParams p, int heads, int team)
{
    constexpr int kEach = D / 32;
    __shared__ float os[kJoinWarps][D], ms[kJoinWarps], ls[kJoinWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int chunks = (p.Hq + heads - 1) / heads, t = blockIdx.x / chunks, head0 = (blockIdx.x - t * chunks) * heads;
    const int n = p.cu ? sequence_with(p.cu, p.N, t, lane) : t;
    grid_wait();
    if (n < 0) return;
    const Part own = load_part(p.parts + p.P + n);
    if (own.kind == kNoWork || t - own.t0 >= own.tokens) return;
    Part prefix = {};
    if (own.prefix >= 0) prefix = load_part(p.parts + own.prefix);
    const int teams = kJoinWarps / team, place = warp % team;
    for (int h0 = head0; h0 < min(p.Hq, head0 + heads); h0 += teams) {
        const int hq = h0 + warp / team;
        const bool mine = hq < min(p.Hq, head0 + heads);
        Pieces ps[2] = {};
        if (mine) {
            ps[0] = pieces_of(p, p.P + n, own, t, hq, 0, own.prefix < 0);
            if (own.prefix >= 0) ps[1] = pieces_of(p, own.prefix, prefix, t, hq, 1, false);
        }
        const int all = ps[0].n + ps[1].n;               // the same in the whole team
        float m = -INFINITY, l = 0.f, acc[kEach];
#pragma unroll
        for (int e = 0; e < kEach; e++) acc[e] = 0.f;
        for (int i0 = 32 * place; i0 < all; i0 += 32 * team) {
            // a piece for each lane
            const int i = i0 + lane;
            const float *from = nullptr;
            float2 ml = make_float2(-INFINITY, 0.f);
            if (i < all) {
                const Pieces &x = i < ps[0].n ? ps[0] : ps[1];
                const int k = i < ps[0].n ? i : i - ps[0].n;
                const int64_t at = k == 0 ? x.first : x.later + (k - 1) * x.apart;
                from = (x.whole ? x.whole : x.cut) + at * D;
                ml = __ldcg((x.whole ? x.whole_ml : x.cut_ml) + at);
            }
            float top = fmaxf(m, ml.x);
#pragma unroll
            for (int o = 16; o > 0; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float was = m == -INFINITY ? 0.f : ex2((m - top) * p.scale_log2);
            const float f = ml.x == -INFINITY ? 0.f : ex2((ml.x - top) * p.scale_log2);
            float sum = ml.x == -INFINITY ? 0.f : f * ml.y;
#pragma unroll
            for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            l = l * was + sum;
            m = top;
#pragma unroll
            for (int e = 0; e < kEach; e++) acc[e] *= was;
            const int here = min(32, all - i0);
#pragma unroll 8
            for (int k = 0; k < here; k++) {
                const float fk = __shfl_sync(0xffffffffu, f, k);
                const float *at = reinterpret_cast<const float *>(__shfl_sync(0xffffffffu, (unsigned long long)from, k));
                if (fk == 0.f) continue;                 // nothing visible there: it may not even be written
                float o[kEach];
                if (kEach == 4) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(at) + lane);
                    o[0] = v.x; o[1] = v.y; o[2 % kEach] = v.z; o[3 % kEach] = v.w;
                } else {
                    const float2 v = __ldcg(reinterpret_cast<const float2 *>(at) + lane);
                    o[0] = v.x; o[1] = v.y;
                }
#pragma unroll
                for (int e = 0; e < kEach; e++) acc[e] = fmaf(fk, o[e], acc[e]);
            }
        }
        if (team > 1) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < kEach; e++) os[warp][kEach * lane + e] = acc[e];
            if (lane == 0) {
                ms[warp] = m;
                ls[warp] = l;
            }
            __syncthreads();
            if (place == 0) {
                float top = m;
                for (int w = 1; w < team; w++) top = fmaxf(top, ms[warp + w]);
                float sum = 0.f, o[kEach];
#pragma unroll
                for (int e = 0; e < kEach; e++) o[e] = 0.f;
                for (int w = 0; w < team; w++) {
                    if (ms[warp + w] == -INFINITY) continue;
                    const float f = ex2((ms[warp + w] - top) * p.scale_log2);
                    sum = fmaf(f, ls[warp + w], sum);
#pragma unroll
                    for (int e = 0; e < kEach; e++) o[e] = fmaf(f, os[warp + w][kEach * lane + e], o[e]);
                }
                l = sum;
#pragma unroll
                for (int e = 0; e < kEach; e++) acc[e] = o[e];
            }
        }
        if (all && place == 0) {
            const float inv = 1.f / l;
            uint16_t *to = p.out + ((int64_t)t * p.Hq + hq) * D + kEach * lane;
            if (kEach == 4)
                *reinterpret_cast<uint2 *>(to) = make_uint2(Half2<E>::pack(acc[0] * inv, acc[1] * inv),
                                                            Half2<E>::pack(acc[2 % kEach] * inv, acc[3 % kEach] * inv));
            else
                *reinterpret_cast<uint32_t *>(to) = Half2<E>::pack(acc[0] * inv, acc[1] * inv);
        }
    }
}

// the workspace's pieces, each from a multiple of 256 bytes on
struct Room {
    int64_t parts, tiles, steps, whole[2], whole_ml[2], cut_tiles, cut_tiles_ml, cut_rows, cut_rows_ml, size;
};
// no part has more rows than the call
bool can_have_tiles(int T, int G) { return (int64_t)T * G > kFewRows; }
Room room_of(int N, int T, int P, int Hq, int Hk, int d)
{
    Room r;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    const int64_t parts = (int64_t)P + N, heads = (int64_t)T * Hq;
    r.parts = take(parts * sizeof(Part));
    r.tiles = take((parts + 1) * 8);
    r.steps = take((parts + 1) * 8);
    for (int i = 0; i < 2; i++) {
        r.whole[i] = take(P ? heads * d * 4 : 0);
        r.whole_ml[i] = take(P ? heads * 8 : 0);
    }
    const int64_t tiles = 2 * kMaxSms * kPieceRows, rows = 2 * kMaxSms * kRowWorkersPerSm * kFewRows;
    const bool any_tiles = can_have_tiles(T, Hq / Hk), any_rows = Hq / Hk <= kFewRows;
    r.cut_tiles = take(any_tiles ? tiles * d * 4 : 0);
    r.cut_tiles_ml = take(any_tiles ? tiles * 8 : 0);
    r.cut_rows = take(any_rows ? rows * d * 4 : 0);
    r.cut_rows_ml = take(any_rows ? rows * 8 : 0);
    r.size = at;
    return r;
}

template <typename E, int D> cudaError_t launch_join(const PagedAttentionArgs &a, const AttendParams &p)
{
    // few rows: a CTA a head, whose warps share the pieces; many: all heads of a row
    int heads = a.Hq, team = 1;
    while (heads > 1 && (int64_t)a.T * ((a.Hq + heads - 1) / heads) < 4 * a.num_sms) heads = (heads + 1) / 2;
    while (team < kJoinWarps && heads * team < kJoinWarps) team *= 2;
    const int64_t blocks = (int64_t)a.T * ((a.Hq + heads - 1) / heads);
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, join_kernel<E, D>, p, heads, team);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

int64_t paged_attention_workspace(int N, int T, int P, int Hq, int Hk, int d) { return room_of(N, T, P, Hq, Hk, d).size; }

cudaError_t launch_paged_attention(const PagedAttentionArgs &a)
{
    AttendParams p = {};
    p.q = (const uint16_t *)a.q; p.q_stride = a.q_stride;
    p.cu = a.cu_seqlens; p.starts = a.starts; p.slots = a.slots;
    p.groups = a.groups; p.prefix_lens = a.prefix_lens; p.prefix_slots = a.prefix_slots;
    p.cache = a.cache; p.out = (uint16_t *)a.out;
    p.N = a.N; p.T = a.T; p.P = a.P; p.Hq = a.Hq; p.Hk = a.Hk; p.G = a.Hq / a.Hk;
    p.tile_tokens = kTileRows / p.G; p.inv_G = (65536 + p.G - 1) / p.G;
    p.scale_log2 = a.scale * kLog2e; p.err = a.err_word;
    const Room r = room_of(a.N, a.T, a.P, a.Hq, a.Hk, a.d);
    uint8_t *w = (uint8_t *)a.workspace;
    p.parts = (Part *)(w + r.parts);
    p.tiles = (int64_t *)(w + r.tiles);
    p.steps = (int64_t *)(w + r.steps);
    for (int i = 0; i < 2; i++) {
        p.whole[i] = (float *)(w + r.whole[i]);
        p.whole_ml[i] = (float2 *)(w + r.whole_ml[i]);
    }
    p.cut_tiles = (float *)(w + r.cut_tiles); p.cut_tiles_ml = (float2 *)(w + r.cut_tiles_ml);
    p.cut_rows = (float *)(w + r.cut_rows); p.cut_rows_ml = (float2 *)(w + r.cut_rows_ml);
    const int sms = a.num_sms < kMaxSms ? a.num_sms : kMaxSms;
    p.tile_workers = sms;
    p.row_workers = sms * kRowWorkersPerSm;
    // a call of single rows without prefixes has no part for the tiles kernel either, one of
    // many heads none for the rows kernel
    const bool tiles = can_have_tiles(a.T, p.G) && (a.cu_seqlens || a.P || p.G > kFewRows), rows = p.G <= kFewRows;
    p.after_tiles = tiles;
    plan_kernel<<<1, kPlanThreads, 0, a.stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && tiles) e = launch_paged_tiles(a, p);
    if (e == cudaSuccess && rows) e = launch_paged_rows(a, p);
    if (e != cudaSuccess) return e;
    if (a.d == 128) return a.f16 ? launch_join<__half, 128>(a, p) : launch_join<__nv_bfloat16, 128>(a, p);
    return a.f16 ? launch_join<__half, 64>(a, p) : launch_join<__nv_bfloat16, 64>(a, p);
}

}  // namespace kda
