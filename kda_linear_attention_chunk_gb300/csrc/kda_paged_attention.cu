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
// is launched early (programmatic dependent launch) and waits for what it needs.  The plan
// takes 4-6 us (a few loads that depend on one another), the join 7 (a row in 152 pieces) to 22
// (65,536 rows, most of them in two).
#include <stdint.h>

#include "kda_paged_attend.cuh"

namespace kda {
namespace {

constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ AttendParams p)
{
    __shared__ int64_t sums[2][kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, all = p.P + p.N;
    grid_go_on();
    int64_t done[2] = {0, 0};                            // tiles and steps so far
    for (int base = 0; base < all; base += kPlanThreads) {
        const int i = base + tid;
        int64_t mine[2] = {0, 0};
        Part x = {};
        if (i < all) {
            x = make_part(p, i);
            if (x.kind == kTilesWork) mine[0] = part_tiles(x, i < p.P, 2 * p.tile_tokens);
            if (x.kind == kRowsWork) mine[1] = steps_set_up(x) + part_steps(x);
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
        int64_t before[2];
#pragma unroll
        for (int k = 0; k < 2; k++) {
            before[k] = done[k] + upto[k] - mine[k] + (warp ? sums[k][warp - 1] : 0);
            done[k] += sums[k][kPlanThreads / 32 - 1];
        }
        if (i < all) {
            x.begin = before[x.kind == kRowsWork];
            store_part(p.parts + i, x);
            p.tiles[i] = before[0];
            p.steps[i] = before[1];
        }
        __syncthreads();
    }
    if (tid == 0) {
        p.lines->total[0] = done[0];
        p.lines->total[1] = done[1];
        p.lines->share[0] = share_of(done[0], p.Hk, p.tile_workers, kLeastTiles);
        p.lines->share[1] = share_of(done[1], p.Hk, p.row_workers, kLeastSteps);
    }
}

// Joins the pieces of rows.  A CTA takes one row of the batch and `heads` of its query heads;
// `team` groups of eight lanes share one head, every team-th piece each, and then every
// team-th pair of its columns.  What bounds it is the latency of a few loads that depend on
// one another, so a head has few lanes and each of them several loads on its way, and all
// heads of a CTA go at once.  Most of a row's facts are the same for all its heads; a head
// then costs two divisions, and nothing more where its answer is written already (a chunk of
// a prompt: all but the spans that two workers share).
constexpr int kJoinThreads = 256, kLanes = 8, kGroups = kJoinThreads / kLanes;

// a row's place in one of its two parts
struct Place {
    int64_t total, share;            // of the kernel's line
    int64_t begin, n;                // the steps of the row's span or part in the line of a key head
    int row, rows;                   // the row's first query head in a piece; rows of a piece
    bool tiles, any;
};
__device__ __forceinline__ Place place_of(const AttendParams &p, const Lines &lines, const Part &x, bool shared, int t)
{
    Place r = {};
    // (a row outside its prefix's part: cu_seqlens or groups broke their contract)
    r.any = x.kind != kNoWork && t >= x.t0 && t - x.t0 < x.tokens;
    if (!r.any) return r;
    r.tiles = x.kind == kTilesWork;
    r.total = lines.total[!r.tiles];
    r.share = lines.share[!r.tiles];
    r.begin = x.begin;
    const int i = t - x.t0, span = 2 * p.tile_tokens;
    if (r.tiles) {
        const int j = i / span, u = i - j * span, q = u >= p.tile_tokens;
        r.begin += span_begin(x, shared, span, j) + tiles_set_up(x);
        r.n = span_tiles(x, shared, span, j);
        r.row = q * kTileRows + (u - q * p.tile_tokens) * p.G;
        r.rows = kPieceRows;
    } else {
        r.begin += steps_set_up(x);
        r.n = part_steps(x);
        r.row = i * p.G;
        r.rows = kFewRows;
    }
    return r;
}

// the pieces of one of a row's parts, for one head
struct Pieces {
    const float *o;                  // the row in the first piece,
    const float2 *ml;
    int64_t second, apart;           // rows from there to the second one's, and between later ones'
    int n;                           // 0: there are none, or the row's answer is written
};
template <int D>
__device__ __forceinline__ Pieces pieces_of(const AttendParams &p, const Place &y, int t, int hq, bool shared, bool alone)
{
    Pieces r = {};
    if (!y.any) return r;
    const int hk = hq / p.G;
    const int64_t begin = hk * y.total + y.begin, w0 = quotient(begin, y.share), w1 = quotient(begin + y.n - 1, y.share);
    if (w0 == w1) {
        const int64_t row = (int64_t)t * p.Hq + hq;
        r.o = p.whole[shared] + row * D;
        r.ml = p.whole_ml[shared] + row;
        r.n = !alone;
    } else {
        const int64_t first = cut_piece(w0, begin, w0 * y.share) * y.rows + y.row + hq - hk * p.G;
        r.o = (y.tiles ? p.cut_tiles : p.cut_rows) + first * D;
        r.ml = (y.tiles ? p.cut_tiles_ml : p.cut_rows_ml) + first;
        r.second = y.rows;                               // (the first is its worker's second cut piece)
        r.apart = 2 * y.rows;
        r.n = (int)(w1 - w0 + 1);
    }
    return r;
}

// kBatch: pieces at a time, more of them where there are few rows
template <typename E, int D, int kBatch>
__global__ void __launch_bounds__(kJoinThreads, 6 / kBatch) join_kernel(const __grid_constant__ AttendParams p, int heads, int team)
{
    constexpr int kVecs = D / 4 / kLanes;                // 16-byte vectors of a lane in a row
    __shared__ float4 os[kGroups][D / 4];
    __shared__ float ms[kGroups], ls[kGroups];
    __shared__ Place at[2];
    const int group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
    const int chunks = (p.Hq + heads - 1) / heads, t = blockIdx.x / chunks, head0 = (blockIdx.x - t * chunks) * heads;
    const int n = p.cu ? sequence_with(p.cu, p.N, t, threadIdx.x & 31) : t;
    grid_wait();
    if (n < 0) return;
    const Part own = load_part(p.parts + p.P + n);
    const Lines lines = load_lines(p.lines);
    if (own.kind == kNoWork || t - own.t0 >= own.tokens) return;
    if (threadIdx.x == 0) at[0] = place_of(p, lines, own, false, t);
    if (threadIdx.x == 32) {                             // (another warp, at the same time)
        at[1].any = false;
        if (own.prefix >= 0) at[1] = place_of(p, lines, load_part(p.parts + own.prefix), true, t);
    }
    __syncthreads();
    const int place = group % team, end = min(p.Hq, head0 + heads);
    for (int h0 = head0; h0 < end; h0 += kGroups / team) {
        const int hq = h0 + group / team;
        float m = -INFINITY, l = 0.f;
        float4 acc[kVecs];
#pragma unroll
        for (int v = 0; v < kVecs; v++) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
        int all = 0;                                     // pieces: the same in the whole team
        if (hq < end) {
#pragma unroll 1
            for (int part = 0; part < 2; part++) {
                const Pieces x = pieces_of<D>(p, at[part], t, hq, part, own.prefix < 0);
                // piece i of both parts is that of group i % team
                for (int i0 = (place - all % team + team) % team; i0 < x.n; i0 += kBatch * team) {
                    float2 ml[kBatch];
                    float4 o[kBatch][kVecs];
#pragma unroll
                    for (int k = 0; k < kBatch; k++) {
                        const int i = i0 + k * team;
                        ml[k] = make_float2(-INFINITY, 0.f);
                        if (i < x.n) {
                            const int64_t row = i ? x.second + (i - 1) * x.apart : 0;
                            ml[k] = __ldcg(x.ml + row);
#pragma unroll
                            for (int v = 0; v < kVecs; v++)
                                o[k][v] = __ldcg(reinterpret_cast<const float4 *>(x.o + row * D) + v * kLanes + lane);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < kBatch; k++) {
                        if (ml[k].x == -INFINITY) {      // nothing visible there, and o may not even be written,
                            l += ml[k].y;                // or nothing but NaN, which maxima pass over: the sum has it
                            continue;
                        }
                        const float top = fmaxf(m, ml[k].x);
                        const float was = m == -INFINITY ? 0.f : ex2((m - top) * p.scale_log2);
                        const float f = ex2((ml[k].x - top) * p.scale_log2);
                        l = fmaf(f, ml[k].y, l * was);
                        m = top;
#pragma unroll
                        for (int v = 0; v < kVecs; v++) {
                            acc[v].x = fmaf(f, o[k][v].x, acc[v].x * was);
                            acc[v].y = fmaf(f, o[k][v].y, acc[v].y * was);
                            acc[v].z = fmaf(f, o[k][v].z, acc[v].z * was);
                            acc[v].w = fmaf(f, o[k][v].w, acc[v].w * was);
                        }
                    }
                }
                all += x.n;
            }
        }
        uint16_t *to = p.out + ((int64_t)t * p.Hq + hq) * D;
        if (team == 1) {
            if (!all) continue;
            const float inv = 1.f / l;
#pragma unroll
            for (int v = 0; v < kVecs; v++)
                reinterpret_cast<uint2 *>(to)[v * kLanes + lane] =
                    make_uint2(Half2<E>::pack(acc[v].x * inv, acc[v].y * inv), Half2<E>::pack(acc[v].z * inv, acc[v].w * inv));
            continue;
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < kVecs; v++) os[group][v * kLanes + lane] = acc[v];
        if (lane == 0) {
            ms[group] = m;
            ls[group] = l;
        }
        __syncthreads();
        if (!all) continue;
        const int first = group - place;                 // the team's first group
        float top = -INFINITY, sum = 0.f;
        for (int w = 0; w < team; w++) top = fmaxf(top, ms[first + w]);
        for (int w = 0; w < team; w++)
            sum = fmaf(ms[first + w] == -INFINITY ? 1.f : ex2((ms[first + w] - top) * p.scale_log2), ls[first + w], sum);
        const float inv = 1.f / sum;
        for (int c = threadIdx.x - first * kLanes; c < D / 2; c += team * kLanes) {
            float2 x = make_float2(0.f, 0.f);
            for (int w = 0; w < team; w++) {
                if (ms[first + w] == -INFINITY) continue;
                const float f = ex2((ms[first + w] - top) * p.scale_log2);
                const float2 o = reinterpret_cast<const float2 *>(os[first + w])[c];
                x.x = fmaf(f, o.x, x.x);
                x.y = fmaf(f, o.y, x.y);
            }
            reinterpret_cast<uint32_t *>(to)[c] = Half2<E>::pack(x.x * inv, x.y * inv);
        }
    }
}

// the workspace's pieces, each from a multiple of 256 bytes on
struct Room {
    int64_t parts, lines, tiles, steps, whole[2], whole_ml[2], cut_tiles, cut_tiles_ml, cut_rows, cut_rows_ml, size;
};
constexpr int kMostSequences = 1 << 24;
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
    r.lines = take(sizeof(Lines));
    r.tiles = take(parts * 8);
    r.steps = take(parts * 8);
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
    // few rows: a CTA a head, whose groups share the pieces; more: as many heads a CTA as let
    // all CTAs run at once, up to a group of lanes a head
    int heads = 1, team = kGroups;
    while (heads < a.Hq && team > 1 && (int64_t)a.T * ((a.Hq + heads - 1) / heads) > 3 * a.num_sms) {
        heads *= 2;
        team /= 2;
    }
    const int64_t blocks = (int64_t)a.T * ((a.Hq + heads - 1) / heads);
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, team < kGroups ? join_kernel<E, D, 2> : join_kernel<E, D, 4>, p, heads, team);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

int64_t paged_attention_workspace(int N, int T, int P, int Hq, int Hk, int d)
{
    if (N > kMostSequences || P > kMostSequences) return -1;
    return room_of(N, T, P, Hq, Hk, d).size;
}

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
    p.lines = (Lines *)(w + r.lines);
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
