// kda_paged_attend.cuh -- how the work of kda_paged_attention is cut up: what its
// kernels (kda_paged_attention.cu, kda_paged_tiles.cu, kda_paged_rows.cu) share.  Not
// installed.
//
// A part is a range of rows with a range of keys in one table row's pages: a group's rows
// with its prefix (parts 0 .. P-1), or a sequence's rows with its own keys (part P + n).
// Parts of at most kFewRows query rows a key head are the rows kernel's, with steps of 16
// keys, the others the tiles kernel's, in spans of two query tiles, with tiles of 128 keys.
// (Steps and tiles lie at multiples of their size, so each is within one page or is
// whole pages.)
//
// All steps of a kernel's parts, of one key head after the other, form a line, which
// its workers (a warp, or a CTA) share in equal pieces, whatever the lengths.  Each span or
// part takes some more of the line before its steps, for what its beginning costs a worker (a
// few loads, one after the other), so that short ones spread over more workers.  So a worker
// has the steps of some (part, span, head) to itself, but for its first and last ones,
// which it may share with its neighbours.  The row's maxima, sums and unnormalised outputs
// of every piece that is not a row's whole answer go to the workspace, where the join
// finds them by the same arithmetic.
#pragma once

#include <stdint.h>

#include "kda_paged.cuh"

namespace kda {

constexpr int kFewRows = 16;
constexpr int kStepKeys = 16, kTileKeys = 128, kTileRows = 128;
constexpr int kPieceRows = 2 * kTileRows;            // query rows of a tiles piece
constexpr int kMaxSms = 160;                         // the workspace has room for so many
constexpr int kRowWorkersPerSm = 8;

enum { kNoWork = 0, kRowsWork = 1, kTilesWork = 2 };

struct alignas(16) Part {
    int t0, tokens, first;           // first row, rows, position of the first one
    int key0, key1;                  // positions of its keys
    int entry;                       // whose pages they are in
    int prefix;                      // own keys: the part of the prefix, -1 if there is none
    int kind;
    int64_t begin, pad;              // its place in the line of a key head, with its set-up
};

// the lines of the tiles and of the rows kernel
struct alignas(16) Lines {
    int64_t total[2], share[2];      // steps of a key head, and a worker's share of all
};

struct AttendParams {
    const uint16_t *q;
    int64_t q_stride;
    const int32_t *cu, *starts, *slots, *groups, *prefix_lens, *prefix_slots;
    PagedCache cache;
    uint16_t *out;
    int N, T, P, Hq, Hk, G;
    int tile_tokens, inv_G;          // tokens of a query tile; ceil(2^16 / G): r / G = r inv_G >> 16 for r < 128
    float scale_log2;
    int *err;
    Part *parts;                     // [P + N]
    Lines *lines;
    int64_t *tiles, *steps;          // [P + N]: of one key head, before each part
    float *whole[2];                 // [T][Hq][d]: pieces with all of a part's keys, of own keys and of prefixes
    float2 *whole_ml[2];             // [T][Hq]: their maxima and sums
    float *cut_tiles, *cut_rows;     // [2 workers][kPieceRows | kFewRows][d]: pieces with some of them
    float2 *cut_tiles_ml, *cut_rows_ml;
    int tile_workers, row_workers;
    int after_tiles;                 // the rows kernel runs behind the tiles kernel
};

__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    return (a | b) >> 31 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);   // 32 bits, mostly: fewer instructions
}

// A worker's share of a line of `total` steps a head: at least `least`.
__device__ __forceinline__ int64_t share_of(int64_t total, int Hk, int workers, int least)
{
    const int64_t each = quotient(total * Hk + workers - 1, workers);
    return each < least ? least : each;
}
// What a beginning counts for, in tiles or steps.  With it 40 calls of random sizes, most of them
// small, took 0.76 of their time without (geometric mean; 224 sequences of 2 keys 13 us in place of
// 32, 19 drafts over four prefixes 66 in place of 83).  A long part's beginning is little beside its
// steps, and HBM bounds those: 64 sequences of up to 16k keys took 443 us with it, 437 without; the
// beams of 16 prompts of 8192 109.3 with it, 106.5 without.
constexpr int kTilesSetUp = 3, kStepsSetUp = 4, kShortTiles = 32, kShortSteps = 64;
// A worker's least: a beginning and one tile or step.
constexpr int kLeastTiles = kTilesSetUp + 1, kLeastSteps = kStepsSetUp + 1;

// Sum of floor((a i + b) / 128) over i < n, for a, b >= 0: the whole parts of a / 128 and b / 128
// sum up at once, and what is left counts the lattice points below a line, which turns into
// the same problem with the axes exchanged.
__device__ __forceinline__ int64_t sum_of_tiles(int64_t n, int a, int64_t b)
{
    int64_t sum = n * (n - 1) / 2 * (a / kTileKeys) + n * (b / kTileKeys);
    uint32_t m = kTileKeys, x = a % kTileKeys, y = (uint32_t)(b % kTileKeys);
    while (n > 0) {
        const int64_t top = x * n + y;
        if (top < m) break;
        n = quotient(top, m);
        y = (uint32_t)(top - n * m);
        const uint32_t was = x;
        x = m;
        m = was;
        sum += n * (n - 1) / 2 * (x / m) + n * (y / m);
        x %= m;
        y %= m;
    }
    return sum;
}

__device__ __forceinline__ int spans_of(const Part &x, int span) { return (x.tokens + span - 1) / span; }
// behind the last key that a span's rows see
__device__ __forceinline__ int span_end(const Part &x, bool shared, int span, int j)
{
    return shared ? x.key1 : (int)min((int64_t)x.key1, x.first + min(((int64_t)j + 1) * span, (int64_t)x.tokens));
}
__device__ __forceinline__ int first_tile(const Part &x) { return x.key0 / kTileKeys; }
__device__ __forceinline__ int span_tiles(const Part &x, bool shared, int span, int j)
{
    return (int)(((int64_t)span_end(x, shared, span, j) + kTileKeys - 1) / kTileKeys) - first_tile(x);
}
// tiles of the spans before span j
__device__ __forceinline__ int64_t tiles_before(const Part &x, bool shared, int span, int j)
{
    if (shared) return (int64_t)j * span_tiles(x, true, span, 0);
    return sum_of_tiles(j, span, (int64_t)x.first + span + kTileKeys - 1) - (int64_t)j * first_tile(x);
}
__device__ __forceinline__ int tiles_set_up(const Part &x)
{
    return x.key1 - x.key0 <= kShortTiles * kTileKeys ? kTilesSetUp : 0;
}
// the place of span j, with its set-up, in its part's line; that line's length
__device__ __forceinline__ int64_t span_begin(const Part &x, bool shared, int span, int j)
{
    return tiles_before(x, shared, span, j) + (int64_t)j * tiles_set_up(x);
}
__device__ __forceinline__ int64_t part_tiles(const Part &x, bool shared, int span)
{
    const int n = spans_of(x, span);
    return n ? span_begin(x, shared, span, n - 1) + tiles_set_up(x) + span_tiles(x, shared, span, n - 1) : 0;
}
__device__ __forceinline__ int part_steps(const Part &x)
{
    return (int)(((int64_t)x.key1 + kStepKeys - 1) / kStepKeys) - x.key0 / kStepKeys;
}
__device__ __forceinline__ int steps_set_up(const Part &x) { return part_steps(x) <= kShortSteps ? kStepsSetUp : 0; }

__device__ __forceinline__ Part load_part(const Part *p)
{
    Part x;
    const int4 *from = reinterpret_cast<const int4 *>(p);
    const int4 a = __ldcg(from), b = __ldcg(from + 1);
    const longlong2 c = __ldcg(reinterpret_cast<const longlong2 *>(from + 2));
    x.t0 = a.x; x.tokens = a.y; x.first = a.z; x.key0 = a.w;
    x.key1 = b.x; x.entry = b.y; x.prefix = b.z; x.kind = b.w;
    x.begin = c.x;
    return x;
}
__device__ __forceinline__ void store_part(Part *p, const Part &x)
{
    int4 *to = reinterpret_cast<int4 *>(p);
    to[0] = make_int4(x.t0, x.tokens, x.first, x.key0);
    to[1] = make_int4(x.key1, x.entry, x.prefix, x.kind);
    reinterpret_cast<longlong2 *>(to)[2] = make_longlong2(x.begin, 0);
}
__device__ __forceinline__ Lines load_lines(const Lines *p)
{
    const longlong2 a = __ldcg(reinterpret_cast<const longlong2 *>(p)), b = __ldcg(reinterpret_cast<const longlong2 *>(p) + 1);
    return {{a.x, a.y}, {b.x, b.y}};
}

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
            const RowsAt r = rows_at(p.cu ? p.cu[n] : n, p.cu ? p.cu[n + 1] : n + 1, p.starts ? p.starts[n] : 0, p.cache, p.T,
                                     least, p.err);
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

// The last i in [0, n) with before[i] <= x, where before[0] <= x, by a converged warp.
__device__ __forceinline__ int part_at(const int64_t *before, int n, int64_t x, int lane)
{
    int a = 0;
    while (n > 1) {
        const int step = (n + 31) / 32, i = lane * step;
        const bool le = i < n && __ldcg(before + a + i) <= x;
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, le || lane == 0));
        n = min(step, n - last * step);
        a += last * step;
    }
    return a;
}
// The last span that starts at or before place x of its part, by a converged warp.
__device__ __forceinline__ int span_at(const Part &part, bool shared, int span, int64_t x, int lane)
{
    int a = 0, n = spans_of(part, span);
    while (n > 1) {
        const int step = (n + 31) / 32, i = lane * step;
        const bool le = i < n && span_begin(part, shared, span, a + i) <= x;
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, le || lane == 0));
        n = min(step, n - last * step);
        a += last * step;
    }
    return a;
}

// Where a piece goes: to the output (it is all of its rows' keys), to the whole pieces of own
// keys or of prefixes, or to one of the worker's two cut pieces.
enum { kToOut = 0, kToOwn = 1, kToPrefix = 2, kToCut = 3 };
// begin, end: of the steps of the (part, span, head) in the line; from, to: the worker's share
__device__ __forceinline__ int goes_to(const Part &x, bool shared, int64_t begin, int64_t end, int64_t from, int64_t to)
{
    if (begin < from || end > to) return kToCut;
    return shared ? kToPrefix : x.prefix >= 0 ? kToOwn : kToOut;
}
// which of them: the one that others began, or the one that others end
__device__ __forceinline__ int64_t cut_piece(int64_t worker, int64_t begin, int64_t from) { return 2 * worker + (begin >= from); }

cudaError_t launch_paged_tiles(const PagedAttentionArgs &a, const AttendParams &p);
cudaError_t launch_paged_rows(const PagedAttentionArgs &a, const AttendParams &p);

}  // namespace kda
