// kda_window.cu -- window attention of packed new tokens over the ring cache and
// themselves (prefill), on the tensor cores.
//
// For the query at position p:  o = sum_j softmax_j(scale q . k_j) v_j  over the
// positions j <= p with j > p - window or j < sinks.  Keys of positions before
// the call's come from the cache, the others from the call's rows.
//
// An item of work is two tiles of up to 128 query rows of one key head: the G query
// heads that share it for floor(128 / G) consecutive tokens each, so that each key
// and value tile serves G heads and a tile spans few positions (little of the
// window's edges is computed and masked away).  The visible positions are a few
// runs of consecutive rows (sinks, the ring before and after its wrap, the call's
// rows); they fill tiles of 128 keys, each run from a multiple of 16 on.  Per key
// and query tile, with S, P and O in TMEM:
//
//     S = Q K^T            (tcgen05.mma, both operands in shared memory)
//     P = 2^(c S - c m)    one thread per query row: 128 scores in registers
//     O += P V             (P from TMEM in place of S, V MN-major as loaded)
//
// The two query tiles take turns on the tensor core: while one's scores are
// exponentiated, the other's products run.  The maximum m only follows the true
// one when it falls behind by more than 2^8 (all sums stay in fp32 and the final
// division makes the result independent of m), so O is rarely rescaled, and the
// threads that own the rows do it themselves.
//
// Roles: warps 0-3 and 4-7 the softmax of the two query tiles, warp 8 finds items and
// loads (a ring of four key and value tiles), warps 9 and 11 the MMAs of the two
// query tiles, warp 10 the zeros behind ragged runs of values.  A second kernel then
// writes the rows that the cache keeps.
//
// On a GB300, 32 query heads on 8 key heads of 128: 8192 rows in the middle of a
// context, window 4096, 0.40-0.43 ms (1.29-1.37 PFLOP/s); 32,768 rows at once
// 1.41-1.48 ms; 16 prompts in 8192 rows, window 1024, 84-86 us.  With long windows the
// chain of one query tile bounds it (scores, softmax, P V, the next scores: 2750 cycles
// a key tile, 2050 of them the tensor core's work for both query tiles); with short
// ones what an item costs beside its tiles.
#include <stdint.h>

#include "kda_sm100.cuh"
#include "kda_tiles.cuh"
#include "kda_window.h"

// Poll limit of the softmax's wait for scores.  A test build of the library sets it to
// zero: the wait then gives up at once although its MMAs complete, which takes every
// CTA through the wind-down.
#ifndef KDA_WAIT_LIMIT_SCORES
#define KDA_WAIT_LIMIT_SCORES (1u << 18)
#endif

namespace kda {
namespace {

using namespace sm100;
using namespace tiles;

constexpr int kThreads = 384;
constexpr int kKeys = 128;           // keys of a tile
constexpr int kBox = 16;             // rows of a TMA box: what a run is rounded up to
constexpr int kBigBox = 64;          // rows of one where a run has as many
constexpr int kStages = 4;           // tiles of the ring: keys in the even ones, values in the odd ones
// Runs of an item: sinks, the ring before and after its wrap, the call's rows.  The room
// for two more keeps the softmax warps' registers from a spill (4 bytes with room for
// four: 16 prompts 87.4 us instead of 86.6).
constexpr int kMaxRuns = 6;
constexpr int kBars = 3 * kStages + 23;
constexpr int kStage = 4096;         // bytes in which a softmax warp turns its rows of O around
// Registers: a softmax thread holds a row of 128 scores.  The block starts with
// kRegs for each thread and hands them out anew: 2 x 128 x 216 + 128 x 72 of its
// 384 x 168 (the launch checks that the kernel was built with that number).
constexpr int kRegs = 168, kRegsSoftmax = 216, kRegsOther = 72;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreads * kRegs, "more registers than the block has");
constexpr float kLag = 8.f;          // log2 of what the running maximum may lag behind

struct Run {
    int cached;                      // 1: rows of the ring cache, 0: rows of the call
    int row, pos, len;               // first row, its position, rows
};

// One item of work: two query tiles of one key head.
struct alignas(16) Item {
    Run runs[kMaxRuns];
    int nruns;
    int tokens;                      // rows of the item; 0: there are no more items
    int t0, first;                   // its first row and that row's position
    int hk, entry;                   // key head, cache entry
};

struct Ctl {
    Item items[2];
    uint4 claim;                     // the answer to a claim (16-byte aligned by what precedes it)
    int abort;
    uint32_t tmem;
    uint64_t bars[kBars];
};

// TMEM columns
constexpr int kTmS = 0, kTmO = 256;

// runs of consecutive rows that hold the positions [a, b) of the sequence
__device__ __forceinline__ void add_runs(Item &c, const WindowParams &p, int bos, int start, int a, int b)
{
    auto add = [&](int cached, int row, int pos, int len) {
        if (len > 0) c.runs[c.nruns++] = {cached, row, pos, len};
    };
    const int end = min(b, start);   // of the cached part
    if (a < end) {
        const int ring = p.pool_rows - p.sinks;
        if (end <= p.pool_rows) {
            add(1, a, a, end - a);   // nothing has wrapped: row = position
        } else {
            const int cut = min(end, max(a, p.sinks));
            add(1, a, a, cut - a);
            if (cut < end) {
                const int at = (cut - p.sinks) % ring, len = min(end - cut, ring - at);
                add(1, p.sinks + at, cut, len);
                add(1, p.sinks, cut + len, end - cut - len);
            }
        }
    }
    const int from = max(a, start);
    add(0, bos + (from - start), from, b - from);
}

// A piece of a key tile: `take` consecutive rows in its columns from `col` on.
struct Piece {
    int cached, row, pos, take, col;
};

// Walks the tiles of an item's runs.  A tile is filled with runs one after the other,
// each from a multiple of 16 columns on, up to 128 columns.
struct Tiles {
    const Item &c;
    int run = 0, off = 0;            // where the next tile starts
    int run0 = 0, off0 = 0;          // where this one does
    int keys;                        // columns, a multiple of 16
    int lo, hi, low;                 // lowest and highest position, lowest that is no sink
    bool complete;                   // no column without a key
    __device__ explicit Tiles(const Item &item) : c(item) {}
    // the piece that starts at (r, o), column `col`; moves on to the next
    __device__ Piece piece(int &r, int &o, int &col) const
    {
        const Run &x = c.runs[r];
        const Piece s = {x.cached, x.row + o, x.pos + o, min(kKeys - col, x.len - o), col};
        o += s.take;
        if (o >= x.len) {
            r++;
            o = 0;
        }
        col += (s.take + 15) & ~15;
        return s;
    }
    __device__ bool next(int sinks)
    {
        if (run >= c.nruns) return false;
        run0 = run;
        off0 = off;
        keys = 0;
        lo = low = 0x7fffffff;
        hi = -1;
        complete = true;
#pragma unroll 1
        do {
            const Piece s = piece(run, off, keys);
            const int end = s.pos + s.take - 1;
            lo = min(lo, s.pos);
            hi = max(hi, end);
            if (end >= sinks) low = min(low, max(s.pos, sinks));
            if (s.take & 15) complete = false;
        } while (keys < kKeys && run < c.nruns);
        return true;
    }
};

// whether any of the positions [first, last] sees any key of the tile (or may)
__device__ __forceinline__ bool sees(const Tiles &t, int first, int last, int window, int sinks)
{
    return first <= last && t.lo <= last && (t.hi > first - window || t.lo < sinks);
}

// positions of an item's query tile q
struct Span {
    int first, last, tokens;
    __device__ Span(const Item &item, int tile_tokens, int q)
    {
        tokens = q ? item.tokens - tile_tokens : min(item.tokens, tile_tokens);
        if (tokens <= 0) tokens = 0;
        first = tokens ? item.first + q * tile_tokens : 1;
        last = tokens ? first + tokens - 1 : 0;
    }
};

template <typename E, int D> struct Layout {
    static constexpr int kTile = 128 * D * 2;            // bytes of a query, key or value tile
    static constexpr int kHalf = 128 * 128;              // bytes of its 64 leftmost columns
    static constexpr int kOut = (2 + kStages) * kTile, kCtl = kOut + 8 * kStage;
    static constexpr int kSmem = 1024 + kCtl + sizeof(Ctl);
    static_assert(kSmem <= 227 * 1024, "more shared memory than a CTA has");
    static constexpr bool kF16 = !__is_same(E, __nv_bfloat16);
};

// The barriers; q is a query tile, s a stage of the key / value ring, i a place of
// the item ring.
struct Bars {
    uint32_t at;
    __device__ uint32_t full(int s) const { return at + 8 * s; }                    // tile loaded
    __device__ uint32_t empty(int s) const { return at + 8 * (kStages + s); }       // tile consumed by both products
    __device__ uint32_t values(int s) const { return at + 8 * (2 * kStages + s); }  // value tile without garbage
    __device__ uint32_t q_full(int q) const { return at + 8 * (3 * kStages + q); }
    __device__ uint32_t q_empty(int q) const { return at + 8 * (3 * kStages + 2 + q); }
    __device__ uint32_t s_full(int q) const { return at + 8 * (3 * kStages + 4 + q); }    // scores in TMEM
    __device__ uint32_t p_half(int q) const { return at + 8 * (3 * kStages + 6 + q); }    // probabilities of 64 keys
    __device__ uint32_t p_ready(int q) const { return at + 8 * (3 * kStages + 8 + q); }   // of all
    __device__ uint32_t o_done(int q) const { return at + 8 * (3 * kStages + 10 + q); }   // O complete
    __device__ uint32_t o_free(int q) const { return at + 8 * (3 * kStages + 12 + q); }   // O read
    __device__ uint32_t turn(int q) const { return at + 8 * (3 * kStages + 14 + q); }
    __device__ uint32_t drained(int q) const { return at + 8 * (3 * kStages + 16 + q); }
    __device__ uint32_t claimed() const { return at + 8 * (3 * kStages + 22); }     // a claim is answered
    __device__ uint32_t item_full(int i) const { return at + 8 * (3 * kStages + 18 + i); }
    __device__ uint32_t item_empty(int i) const { return at + 8 * (3 * kStages + 20 + i); }
};
constexpr int kItemReaders = 8 + 2 + 1;   // softmax warps, product warps, patch warp

// Tensor maps; k, v and pool: boxes of kBox rows, then of kBigBox.
struct Maps {
    CUtensorMap q, k[2], v[2], pool[2];
};

// What every role knows.
struct Ctx {
    const WindowParams &p;
    Ctl &c;
    Bars bars;
    uint8_t *smem;                   // 1024-byte aligned
    uint32_t base;                   // its shared-memory address
    uint32_t tmem;
    int lane;
    volatile int *abort;
    __device__ void give_up() const
    {
        atomicOr(p.err, kErrWaitTimeout);
        *abort = 1;
    }
    // A wait of the whole warp, the same answer in every lane: lanes poll and see the abort
    // flag one by one, and one that ran on without the others would meet no partner at
    // the next instruction of the whole warp.
    __device__ bool wait(uint32_t bar, int phase, uint32_t limit = 1u << 18) const
    {
        return __all_sync(0xffffffffu, mbar_wait(bar, phase & 1, abort, limit)) != 0;
    }
};

// The grid has a CTA for each number of an item.  A CTA on an SM, done with its own,
// takes over that of one that has not started yet (cluster launch control), so items
// of any length are dealt evenly without a counter in memory.  Late positions, which
// have most keys, come first.
__device__ __forceinline__ void claim_cta(uint32_t answer, uint32_t bar)
{
    mbar_arrive_expect_tx(bar, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer),
                 "r"(bar) : "memory");
}
// the number of the CTA that was taken over, -1 if none is left
__device__ __forceinline__ int claimed_cta(uint32_t answer)
{
    int cta;
    asm volatile("{\n .reg .pred p;\n .reg .b128 r;\n ld.shared.b128 r, [%1];\n"
                 " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n mov.b32 %0, -1;\n"
                 " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n}" : "=r"(cta) : "r"(answer) : "memory");
    return cta;
}

// Writes the CTA's next item to `item`; `claims`: how many were made (0: its own comes
// first).  The lanes of the converged warp agree on what is returned: 1 found, 0 none
// left, -1 a wait gave up.
template <bool LONG> __device__ __forceinline__ int find_item(const Ctx &x, int &claims, Item &item, const LongSpans &l)
{
    const WindowParams &p = x.p;
    const int span = 2 * p.tile_tokens, lane = x.lane;
    const uint32_t answer = smem_u32(&x.c.claim);
    for (bool own = claims == 0;; own = false) {
        int at = blockIdx.x;
        if (!own) {
            if (elect_one()) claim_cta(answer, x.bars.claimed());
            __syncwarp();
            if (!x.wait(x.bars.claimed(), claims - 1)) {
                mbar_wait_drain(x.bars.claimed(), (claims - 1) & 1);
                return -1;
            }
            at = __shfl_sync(0xffffffffu, claimed_cta(answer), 0);
            fence_proxy_async_smem();                    // the next answer is written behind this read
            __syncwarp();
        }
        claims++;
        if (at < 0) return 0;
        const int number = p.items - 1 - at, slot = number / p.Hk, hk = number - slot * p.Hk;
        // (the other kernel of a divided batch goes through all sequences, and reports)
        const Rows r = LONG ? rows_in(p, sequence_of_long(p, span, slot, lane, l), span, lane, false)
                            : rows_of(p, span, slot, lane, hk == 0);
        if (!r.n) continue;          // past the sequence's rows, or padded
        if (lane == 0) {
            item.nruns = 0;
            item.hk = hk;
            item.entry = r.entry;
            item.tokens = r.n;
            item.t0 = r.bos + r.from;
            item.first = r.start + r.from;
            const int last = item.first + item.tokens - 1, lo = max(0, item.first - p.window + 1);
            if (lo > p.sinks) {
                add_runs(item, p, r.bos, r.start, 0, p.sinks);
                add_runs(item, p, r.bos, r.start, lo, last + 1);
            } else {
                add_runs(item, p, r.bos, r.start, 0, last + 1);
            }
        }
        __syncwarp();
        return 1;
    }
}

// ---- items and loads ---------------------------------------------------------
template <typename E, int D, bool LONG>
__device__ __forceinline__ void load_role(const Ctx &x, const Maps &maps)
{
    using L = Layout<E, D>;
    const WindowParams &p = x.p;
    const uint32_t sq = x.base, skv = x.base + 2 * L::kTile;
    int it = 0, claims = 0, item = 0, qs[2] = {0, 0};    // tiles and query tiles loaded, items written
    bool ok = true, more = true;
    const LongSpans l = LONG ? count_long(p, 2 * p.tile_tokens, x.lane) : LongSpans();
    while (ok && more) {
        Item &now = x.c.items[item & 1];
        if (item >= 2) ok = x.wait(x.bars.item_empty(item & 1), item / 2 - 1);
        if (!ok) break;
        const int found = find_item<LONG>(x, claims, now, l);
        ok = found >= 0;
        more = found > 0;
        if (!ok) break;
        if (x.lane == 0) {
            if (!more) now.tokens = 0;
            mbar_arrive(x.bars.item_full(item & 1));
        }
        item++;
        if (!more) break;
        const int nq = __shfl_sync(0xffffffffu, now.tokens > p.tile_tokens ? 2 : 1, 0);
        const int t0 = __shfl_sync(0xffffffffu, now.t0, 0), hk = __shfl_sync(0xffffffffu, now.hk, 0);
        const int entry_head = __shfl_sync(0xffffffffu, now.entry, 0) * 2 * p.Hk + hk;
        bool queries = false;
        Tiles t(now);
        while (ok && __shfl_sync(0xffffffffu, t.next(p.sinks), 0)) {
            const int keys = __shfl_sync(0xffffffffu, t.keys, 0);
#pragma unroll 1
            for (int kv = 0; kv < 2; kv++) {
                const int s = it % kStages;
                if (ok && it >= kStages) ok = x.wait(x.bars.empty(s), it / kStages - 1);
                if (!ok) break;
                const uint32_t bar = x.bars.full(s), to = skv + s * L::kTile;
                if (elect_one()) mbar_arrive_expect_tx(bar, (uint32_t)(keys * 128 * (D / 64)));
                __syncwarp();
#pragma unroll 1
                for (int r = t.run0, o = t.off0, col = 0; col < keys;) {
                    const Piece piece = t.piece(r, o, col);
                    const int take = __shfl_sync(0xffffffffu, piece.take, 0), at = __shfl_sync(0xffffffffu, piece.col, 0);
                    const int row = __shfl_sync(0xffffffffu, piece.row, 0);
                    const bool cached = __shfl_sync(0xffffffffu, piece.cached, 0);
                    if (elect_one()) {
                        const CUtensorMap *const of = cached ? maps.pool : kv ? maps.v : maps.k;
                        const int c1 = cached ? row : hk, c2 = cached ? entry_head + kv * p.Hk : row;
                        int b = 0;
#pragma unroll 1
                        for (; b + kBigBox <= take; b += kBigBox)
#pragma unroll 1
                            for (int h = 0; h < D / 64; h++)
                                tma_load_3d(to + h * L::kHalf + (at + b) * 128, of + 1, 64 * h, c1 + (cached ? b : 0),
                                            c2 + (cached ? 0 : b), bar);
#pragma unroll 1
                        for (; b < take; b += kBox)
#pragma unroll 1
                            for (int h = 0; h < D / 64; h++)
                                tma_load_3d(to + h * L::kHalf + (at + b) * 128, of, 64 * h, c1 + (cached ? b : 0),
                                            c2 + (cached ? 0 : b), bar);
                    }
                    __syncwarp();
                }
                it++;
                if (queries) continue;
                queries = true;                          // after the first keys, which need not wait for their room
#pragma unroll 1
                for (int q = 0; q < nq && ok; q++) {
                    if (qs[q]) ok = x.wait(x.bars.q_empty(q), qs[q] - 1);
                    if (ok && elect_one()) {
                        // half a query tile is G tile_tokens rows of 128 bytes
                        mbar_arrive_expect_tx(x.bars.q_full(q), (uint32_t)(p.G * p.tile_tokens * 128 * (D / 64)));
#pragma unroll
                        for (int h = 0; h < D / 64; h++)
                            tma_load_3d(sq + q * L::kTile + h * L::kHalf, &maps.q, 64 * h, hk * p.G,
                                        t0 + q * p.tile_tokens, x.bars.q_full(q));
                    }
                    if (ok) qs[q]++;
                }
            }
        }
    }
    if (!ok && x.lane == 0) x.give_up();
    // nothing may still be on its way into shared memory when the CTA ends
#pragma unroll 1
    for (int q = 0; q < 2; q++)
        if (qs[q]) mbar_wait_drain(x.bars.q_full(q), (qs[q] - 1) & 1);
#pragma unroll 1
    for (int i = it < kStages ? 0 : it - kStages; i < it; i++) mbar_wait_drain(x.bars.full(i % kStages), (i / kStages) & 1);
}

// ---- products of one query tile ---------------------------------------------------
// The whole warp walks the loop and one elected lane issues: operands that are
// uniform over the warp stay in uniform registers, where the instruction takes them
// (85 cycles an MMA from a loop that one lane runs alone).  The two query tiles take
// turns, so that one's scores are exponentiated during the other's products: left
// alone they fall into step (4100 cycles a tile of keys instead of 2700).
template <typename E, int D>
__device__ __forceinline__ void product_role(const Ctx &x, int which)
{
    using L = Layout<E, D>;
    const WindowParams &p = x.p;
    const int q = __shfl_sync(0xffffffffu, which, 0);
    const uint32_t tm = __shfl_sync(0xffffffffu, x.tmem, 0);
    const uint32_t ts = tm + kTmS + 128 * q, to = tm + kTmO + 128 * q;
    const uint32_t qs = x.base + q * L::kTile, skv = x.base + 2 * L::kTile;
    int it = 0, parts = 0, turns = 0, mine = 0;          // tiles consumed; products P V issued; turns taken; items with rows
    bool ok = true;
    for (int item = 0; ok; item++) {
        const Item &now = x.c.items[item & 1];
        ok = x.wait(x.bars.item_full(item & 1), item / 2);
        const int tokens = __shfl_sync(0xffffffffu, now.tokens, 0);
        if (!ok || tokens == 0) break;
        const Span rows(now, p.tile_tokens, q);
        const bool both = tokens > p.tile_tokens, any = __shfl_sync(0xffffffffu, rows.tokens > 0, 0);
        int done = 0;                                    // products P V of this item
        Tiles t(now);
        bool have = __shfl_sync(0xffffffffu, t.next(p.sinks), 0);
        bool sees_now = __shfl_sync(0xffffffffu, sees(t, rows.first, rows.last, p.window, p.sinks), 0);
        int keys = __shfl_sync(0xffffffffu, t.keys, 0);
        ok = x.wait(x.bars.full(it % kStages), it / kStages) && (!any || x.wait(x.bars.q_full(q), mine));
        if (elect_one()) {
            if (ok && sees_now) {
                mma_scores<D>(ts, qs, skv + it % kStages * L::kTile, idesc(keys, 0, L::kF16));
                mma_commit(x.bars.s_full(q));
            }
            mma_commit(x.bars.empty(it % kStages));
        }
        it++;
        while (have && ok) {
            const int sv = it % kStages, steps = keys / 16;       // this tile's values
            const bool saw = sees_now;
            ok = x.wait(x.bars.values(sv), it / kStages);
            it++;
            const int sk = it % kStages;                 // the next tile's keys
            have = __shfl_sync(0xffffffffu, t.next(p.sinks), 0);
            if (have) {
                sees_now = __shfl_sync(0xffffffffu, sees(t, rows.first, rows.last, p.window, p.sinks), 0);
                keys = __shfl_sync(0xffffffffu, t.keys, 0);
                ok = ok && x.wait(x.bars.full(sk), it / kStages);
                it++;
            } else if (any && elect_one()) {
                mma_commit(x.bars.q_empty(q));           // every product with the query tile is issued
            }
            __syncwarp();
            if (both && ok && (q || turns)) ok = x.wait(x.bars.turn(q), q ? turns : turns - 1);
            if (ok && saw) {
                if (done == 0 && mine > 0) ok = x.wait(x.bars.o_free(q), mine - 1);
                ok = ok && x.wait(x.bars.p_half(q), parts);
                if (ok) {
                    tc_fence_after();
                    if (elect_one()) mma_values<D>(to, ts, skv + sv * L::kTile, idesc(D, 1, L::kF16), 0, steps, done > 0);
                    ok = x.wait(x.bars.p_ready(q), parts);
                }
                if (ok) {
                    tc_fence_after();
                    if (elect_one()) mma_values<D>(to, ts, skv + sv * L::kTile, idesc(D, 1, L::kF16), 4, steps, true);
                    done++;
                    parts++;
                }
            }
            if (elect_one()) {
                if (ok && have && sees_now) {
                    mma_scores<D>(ts, qs, skv + sk * L::kTile, idesc(keys, 0, L::kF16));
                    mma_commit(x.bars.s_full(q));
                }
                if (both) mbar_arrive(x.bars.turn(!q));
                mma_commit(x.bars.empty(sv));
                if (have) mma_commit(x.bars.empty(sk));
                else if (any) mma_commit(x.bars.o_done(q));
            }
            __syncwarp();
            if (both) turns++;
        }
        if (any) mine++;
        __syncwarp();
        if (x.lane == 0) mbar_arrive(x.bars.item_empty(item & 1));
    }
    if (!ok && x.lane == 0) x.give_up();
    // every product is finished before the TMEM and shared memory go
    if (elect_one()) mma_commit(x.bars.drained(q));
    mbar_wait_drain(x.bars.drained(q), 0);
}

// ---- zeros behind ragged runs ------------------------------------------------------
// Value rows past a run hold anything, and 0 x NaN is NaN: the rows that a run is
// rounded up to become zeros.  Every value tile passes through
// here.
template <typename E, int D>
__device__ __forceinline__ void patch_role(const Ctx &x)
{
    using L = Layout<E, D>;
    const WindowParams &p = x.p;
    bool ok = true;
    for (int item = 0, it = 1; ok; item++) {
        const Item &now = x.c.items[item & 1];
        ok = x.wait(x.bars.item_full(item & 1), item / 2);
        if (!ok || now.tokens == 0) break;
        Tiles t(now);
        for (; ok && t.next(p.sinks); it += 2) {
            const int s = it % kStages;
            ok = x.wait(x.bars.full(s), it / kStages);
            if (!ok) break;
            if (!t.complete) {
#pragma unroll 1
                for (int r = t.run0, o = t.off0, col = 0; col < t.keys;) {
                    const Piece piece = t.piece(r, o, col);
                    const int from = piece.col + piece.take;
#pragma unroll 1
                    for (int e = x.lane; e < (col - from) * (D / 8); e += 32) {
                        const int at = from + e / (D / 8), v = e % (D / 8);
                        *reinterpret_cast<uint4 *>(x.smem + (2 + s) * L::kTile + (v / 8) * L::kHalf + at * 128 + (v % 8) * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (x.lane == 0) mbar_arrive(x.bars.values(s));
        }
        __syncwarp();
        if (x.lane == 0) mbar_arrive(x.bars.item_empty(item & 1));
    }
    if (!ok && x.lane == 0) x.give_up();
}

// ---- softmax, one thread per query row, and the output -------------------------------
template <typename E, int D>
__device__ __forceinline__ void softmax_role(const Ctx &x, int warp)
{
    using L = Layout<E, D>;
    const WindowParams &p = x.p;
    const int q = warp >> 2, row = 32 * (warp & 3) + x.lane, lane = x.lane;
    const int token = row * p.inv_G >> 16;               // row / G
    const uint32_t lanes = x.tmem + ((uint32_t)(warp & 3) << 21);
    const uint32_t ts = lanes + kTmS + 128 * q, to = lanes + kTmO + 128 * q;
    const float c2 = p.scale_log2;
    uint8_t *stage = x.smem + L::kOut + warp * kStage;
    int it = 0, mine = 0;                                // score tiles, items with rows
    bool ok = true;
    for (int item = 0; ok; item++) {
        const Item &now = x.c.items[item & 1];
        ok = x.wait(x.bars.item_full(item & 1), item / 2);
        if (!ok || now.tokens == 0) break;
        const Span rows(now, p.tile_tokens, q);
        const int lo_row = rows.first + (32 * (warp & 3) * p.inv_G >> 16);
        const int hi_row = rows.first + min((32 * (warp & 3) + 31) * p.inv_G >> 16, rows.tokens - 1);   // (no sum beyond 2^31)
        const bool dead = 32 * (warp & 3) >= rows.tokens * p.G;      // no row of this warp is one: O may be anything
        const int pos = rows.first + token, t0 = now.t0 + q * p.tile_tokens, hk = now.hk;
        float m = -INFINITY, sum = 0.f;
        Tiles t(now);
        while (rows.tokens && t.next(p.sinks)) {
            if (!sees(t, rows.first, rows.last, p.window, p.sinks)) continue;
            // every key of the tile visible to every row of the warp: no test per key
            const bool whole = t.complete && t.keys == kKeys && t.hi <= lo_row && t.low > hi_row - p.window;
            // Lanes may give up one by one: the vote on the maxima below is also the one on that
            // (a vote here: 405 us for 399, 8192 rows, W 4096); a lane that gave up goes
            // on until then with what its row of TMEM holds.
            const bool got = mbar_wait(x.bars.s_full(q), it & 1, x.abort, KDA_WAIT_LIMIT_SCORES);
            it++;
            if (dead) {                                  // whatever is there will do as these rows' P
                ok = __all_sync(0xffffffffu, got);
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive(x.bars.p_half(q));
                    mbar_arrive(x.bars.p_ready(q));
                }
                continue;
            }
            __syncwarp();
            tc_fence_after();
            uint32_t s[4][32];
#pragma unroll
            for (int i = 0; i < 4; i++)
                if (32 * i < t.keys) tmem_ld32(ts + 32 * i, s[i]);
            loaded(s[0], s[1], s[2], s[3]);
            if (!whole) {
                uint32_t seen[4] = {0, 0, 0, 0};         // visible columns
#pragma unroll 1
                for (int r = t.run0, o = t.off0, col = 0; col < t.keys;) {
                    const Piece s = t.piece(r, o, col);
                    const int end = s.col + min(s.take, pos - s.pos + 1);            // columns at or before the row
                    const int old = s.col + (max(pos - p.window, -1) - s.pos) + 1;   // columns behind the window,
                    const int sink = s.col + p.sinks - s.pos;                        // but for the sinks
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        seen[i] |= below(end - 32 * i) & ~below(s.col - 32 * i) & ~(below(old - 32 * i) & ~below(sink - 32 * i));
                }
#pragma unroll
                for (int i = 0; i < 4; i++) {
#pragma unroll
                    for (int j = 0; j < 32; j++)
                        if (!(seen[i] & (1u << j))) s[i][j] = 0xff800000u;   // -inf
                }
            }
            float mx[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                mx[i] = __uint_as_float(s[i][0]);
#pragma unroll
                for (int j = 1; j < 32; j++) mx[i] = fmaxf(mx[i], __uint_as_float(s[i][j]));
            }
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            const float was = slope<E>(m, c2);
            const bool behind = m != -INFINITY && (top - m) * was > kLag;
            if (__any_sync(0xffffffffu, behind || !got)) {
                ok = __all_sync(0xffffffffu, got);
                if (!ok) break;
                // the products into O so far were complete before these scores were, and
                // the next one waits for this warp
                const float f = behind ? ex2(fmaf(m - top, c2, residue(top, slope<E>(top, c2)) - residue(m, was))) : 1.f;
                for (int i = 0; i < D / 32; i++) {
                    uint32_t o[32];
                    tmem_ld32(to + 32 * i, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; j++) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                    tmem_st32(to + 32 * i, o);
                }
                tmem_wait_st();
                sum *= f;
                if (behind) m = top;
            }
            if (m == -INFINITY) m = top;                 // the row's first visible keys: its O is still zero
            const float now_c = slope<E>(m, c2), z = m == -INFINITY ? 0.f : -m * now_c;
            float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                if (i == 2) {                            // the first 64 keys are in TMEM: their product can start
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(x.bars.p_half(q));
                }
                if (32 * i < t.keys) {
                    uint32_t w[16];
#pragma unroll
                    for (int j = 0; j < 16; j++) {
                        float2 e = fma2(make_float2(__uint_as_float(s[i][2 * j]), __uint_as_float(s[i][2 * j + 1])),
                                        make_float2(now_c, now_c), make_float2(z, z));
                        e.x = ex2(e.x);
                        e.y = ex2(e.y);
                        part[j & 1] = add2(part[j & 1], e);
                        w[j] = Half2<E>::pack(e.x, e.y);
                    }
                    tmem_st16(ts + 16 * i, w);
                }
            }
            sum += (part[0].x + part[0].y) + (part[1].x + part[1].y);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(x.bars.p_ready(q));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(x.bars.item_empty(item & 1));
        if (!ok || !rows.tokens) continue;
        ok = x.wait(x.bars.o_done(q), mine);
        if (!ok) break;
        tc_fence_after();
        mine++;
        // O / sum in 16 bits, 64 columns at a time through shared memory, so that a
        // store instruction writes four rows of 128 bytes
        const float inv = 1.f / sum;
        const int live = rows.tokens * p.G - 32 * (warp & 3);        // of this warp's rows
        uint16_t *out = p.out + ((int64_t)t0 * p.Hq + hk * p.G) * D + 8 * (lane & 7);
#pragma unroll 1
        for (int h = 0; h < D / 64; h++) {
            uint32_t o[2][32];
            tmem_ld32(to + 64 * h, o[0]);
            tmem_ld32(to + 64 * h + 32, o[1]);
            tmem_wait_ld();
            if (h == D / 64 - 1) {                       // O is free for the next item
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(x.bars.o_free(q));
            }
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const uint32_t *v = &o[j / 4][8 * (j & 3)];
                uint4 r;
                r.x = Half2<E>::pack(__uint_as_float(v[0]) * inv, __uint_as_float(v[1]) * inv);
                r.y = Half2<E>::pack(__uint_as_float(v[2]) * inv, __uint_as_float(v[3]) * inv);
                r.z = Half2<E>::pack(__uint_as_float(v[4]) * inv, __uint_as_float(v[5]) * inv);
                r.w = Half2<E>::pack(__uint_as_float(v[6]) * inv, __uint_as_float(v[7]) * inv);
                *reinterpret_cast<uint4 *>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) = r;
            }
            __syncwarp();
            uint4 v[8];
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const int r = 4 * j + (lane >> 3);
                v[j] = *reinterpret_cast<const uint4 *>(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
            }
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const int rr = 4 * j + (lane >> 3), r = 32 * (warp & 3) + rr, tok = r * p.inv_G >> 16;
                if (rr < live) *reinterpret_cast<uint4 *>(out + (tok * (p.Hq - p.G) + r) * D + 64 * h) = v[j];
            }
            __syncwarp();
        }
    }
    if (!ok) x.give_up();
}

// LONG: for a divided batch
template <typename E, int D, bool LONG>
__global__ void __launch_bounds__(kThreads, 1)
window_prefill_kernel(const __grid_constant__ Maps maps, const __grid_constant__ WindowParams p)
{
    using L = Layout<E, D>;
    extern __shared__ uint8_t smem_raw[];
    if (LONG) {                      // mostly there is nothing to do, and the other kernel wants the SMs
        grid_go_on();
        bool any = false;
        for (int n = threadIdx.x; n < p.N; n += kThreads) any |= long_spans(p, 1, n) > 0;
        if (!__syncthreads_or(any)) return;
    }
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - smem_u32(smem_raw));
    Ctl &c = *reinterpret_cast<Ctl *>(smem + L::kCtl);
    const Bars bars{smem_u32(c.bars)};
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp == 8 && lane == 0) {
        c.abort = 0;
        for (int s = 0; s < kStages; s++) {
            mbar_init(bars.full(s), 1);
            mbar_init(bars.empty(s), 2);
            mbar_init(bars.values(s), 1);
        }
        for (int q = 0; q < 2; q++) {
            mbar_init(bars.q_full(q), 1);
            mbar_init(bars.q_empty(q), 1);
            mbar_init(bars.s_full(q), 1);
            mbar_init(bars.p_half(q), 4);
            mbar_init(bars.p_ready(q), 4);
            mbar_init(bars.o_done(q), 1);
            mbar_init(bars.o_free(q), 4);
            mbar_init(bars.turn(q), 1);
            mbar_init(bars.drained(q), 1);
            mbar_init(bars.item_full(q), 1);
            mbar_init(bars.item_empty(q), kItemReaders);
        }
        mbar_init(bars.claimed(), 1);
        mbar_fence_init();
        tma_prefetch_desc(&maps.q);
        for (int i = 0; i < 2; i++) {
            tma_prefetch_desc(&maps.k[i]);
            tma_prefetch_desc(&maps.v[i]);
            tma_prefetch_desc(&maps.pool[i]);
        }
    }
    if (warp == 9) {
        tmem_alloc(smem_u32(&c.tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_go_on();
    const Ctx x{p, c, bars, smem, base, c.tmem, lane, &c.abort};
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == 8) load_role<E, D, LONG>(x, maps);
        else if (warp == 10) patch_role<E, D>(x);
        else product_role<E, D>(x, warp == 11);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        softmax_role<E, D>(x, warp);
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(x.tmem, 512);
}

// Writes the rows that the cache keeps: sinks, and each sequence's last pool_rows -
// sinks positions.  A CTA takes kCommitRows consecutive rows of a sequence, a warp
// one of them at a time.
constexpr int kCommitRows = 8;

template <int D>
__global__ void __launch_bounds__(256) ring_commit_kernel(const __grid_constant__ WindowParams p)
{
    const int lane = threadIdx.x & 31;
    const Rows r = rows_of(p, kCommitRows, blockIdx.x, lane, false);
    const int i = r.from + (threadIdx.x >> 5);           // this warp's row of the sequence
    // The attention kernel may still be running, and reads the cached rows of sequences
    // that have some; nobody leaves before it is done.
    if (r.start != 0 || i >= r.from + r.n) grid_wait();
    if (i >= r.from + r.n) return;
    const int pos = r.start + i, ring = p.pool_rows - p.sinks;
    if (pos >= p.sinks && r.len - i > ring) {            // a later row of the call takes its place
        grid_wait();
        return;
    }
    const uint16_t *k = p.k + (r.bos + i) * p.k_stride, *v = p.v + (r.bos + i) * p.v_stride;
    uint16_t *to = p.pool + (int64_t)r.entry * 2 * p.Hk * p.pool_rows * D + (int64_t)ring_row(pos, p.sinks, p.pool_rows) * D;
    const int64_t head = (int64_t)p.pool_rows * D;
    const int n = 2 * p.Hk * (D / 8);                    // vectors of 16 bytes: keys, then values
    for (int e0 = lane; e0 < n; e0 += 32 * 8) {
        uint4 x[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int e = e0 + 32 * j, h = e / (D / 8), at = e % (D / 8) * 8;
            if (e < n) x[j] = *reinterpret_cast<const uint4 *>((h < p.Hk ? k + h * D : v + (h - p.Hk) * D) + at);
        }
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int e = e0 + 32 * j, h = e / (D / 8), at = e % (D / 8) * 8;
            if (e < n) *reinterpret_cast<uint4 *>(to + h * head + at) = x[j];
        }
    }
    grid_wait();
}

// Whether the call has so few query rows a sequence and key head (on average) that
// the warp-MMA kernel, which takes 16 to 64 of them at a time, is faster than tiles
// of 128: up to 32, and up to 256 where so few items leave most SMs without a tile
// (the other kernel spreads each over eight CTAs).  Measured (us, warp-MMA / tiles;
// G = 4, d = 128): 64 sequences, window 1024: 16 rows 58 / 77, 32 rows 72 / 80, 64
// rows 121 / 81; one sequence, window 4096: 32 rows 21 / 56, 256 rows 48 / 63; 16
// fresh sequences: 64 rows 22 / 20, 256 rows 31 / 19.  Over G = 1 to 128 and d = 64 and 128 the
// quotient of the two is, for the 64 sequences, 0.62-0.83 at 16 rows, 0.75-1.15 at 32 and
// 1.2-1.8 at 64; for the one sequence 0.3-0.5 at 32 rows and 0.4-1.2 at 256.
bool few_rows(const WindowParams &p, int num_sms)
{
    const int64_t rows = (int64_t)p.T * p.G;
    return rows <= (int64_t)32 * p.N || (rows <= (int64_t)256 * p.N && p.items * 8 <= num_sms);
}

// The rule goes by the average, which says nothing of a long sequence among many short or
// empty ones.  So where few_rows holds, a batch of kDividedRows query rows a key head or
// more is divided (kda_window.h): the tiles take its sequences of more than kLongRows,
// and their CTAs leave at once where there are none.  Measured (us, undivided / divided; G = 4,
// d = 128): one sequence of 512 tokens among 63 empty ones, window 1024 74 / 34, window
// 4096 197 / 73; 2048 tokens among 255 empty ones 270 / 61 and 715 / 132; 64 sequences of
// eight tokens each, of which none is long, 74 / 77.  Below, division gains less (128
// tokens among 15 empty ones, 512 rows: 34 / 34 and 85 / 73).
constexpr int kLongRows = 256, kDividedRows = 1024;

template <typename E, int D, bool LONG>
cudaError_t launch_tiles(const WindowArgs &a, const WindowParams &p)
{
    Maps maps;
    bool ok = make_map(&maps.q, a.q, a.f16, D, a.Hq, D, a.T, a.q_stride, p.G, p.tile_tokens);
    for (int i = 0; i < 2 && ok; i++) {
        const int box = i ? kBigBox : kBox;
        ok = make_map(&maps.k[i], a.k, a.f16, D, a.Hk, D, a.T, a.k_stride, 1, box) &&
             make_map(&maps.v[i], a.v, a.f16, D, a.Hk, D, a.T, a.v_stride, 1, box);
        if (!a.pool) maps.pool[i] = maps.k[i];           // never used: no position is before the call's
        else ok = ok && make_map(&maps.pool[i], a.pool, a.f16, D, a.pool_rows, D, (int64_t)a.num_slots * 2 * a.Hk,
                                 (int64_t)a.pool_rows * D, box, 1);
    }
    if (!ok) return cudaErrorInvalidValue;
    const int smem = Layout<E, D>::kSmem;
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = once_per_device(ready, a.device, [&]() {
        cudaFuncAttributes built;
        cudaError_t r = cudaFuncGetAttributes(&built, window_prefill_kernel<E, D, LONG>);
        if (r == cudaSuccess && built.numRegs != kRegs) r = cudaErrorInvalidConfiguration;
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(window_prefill_kernel<E, D, LONG>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        return r;
    });
    if (e != cudaSuccess) return e;
    window_prefill_kernel<E, D, LONG><<<p.items, kThreads, smem, a.stream>>>(maps, p);
    return cudaGetLastError();
}

template <typename E, int D>
cudaError_t launch(const WindowArgs &a, const WindowParams &p)
{
    cudaError_t e;
    if (!few_rows(p, a.num_sms)) {
        e = launch_tiles<E, D, false>(a, p);
    } else if ((int64_t)p.T * p.G < kDividedRows) {
        e = launch_window_rows(a, 0);
    } else {
        WindowParams l = p;
        l.longer = kLongRows;
        const int64_t most = (int64_t)p.T * p.G / (kLongRows + 1);   // long sequences that there can be
        l.items = (int)((p.T / (2 * p.tile_tokens) + (most < p.N ? most : p.N)) * p.Hk);
        e = launch_tiles<E, D, true>(a, l);
        if (e == cudaSuccess) e = launch_window_rows(a, kLongRows);
    }
    if (e != cudaSuccess || !a.pool) return e;
    // its CTAs start where those of the attention kernel have ended
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.T / kCommitRows + p.N));
    cfg.blockDim = dim3(256);
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, ring_commit_kernel<D>, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t launch_window_prefill(const WindowArgs &a)
{
    WindowParams p = window_params(a);
    p.tile_tokens = 128 / p.G;
    p.inv_G = (65536 + p.G - 1) / p.G;
    const int64_t items = ((int64_t)a.T / (2 * p.tile_tokens) + a.N) * a.Hk;
    if (items > 0x7fffffff) return cudaErrorInvalidConfiguration;
    p.items = (int)items;
    if (a.d == 128) return a.f16 ? launch<__half, 128>(a, p) : launch<__nv_bfloat16, 128>(a, p);
    return a.f16 ? launch<__half, 64>(a, p) : launch<__nv_bfloat16, 64>(a, p);
}

}  // namespace kda
