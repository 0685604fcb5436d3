// kda_paged_tiles.cu -- attention over a paged cache for parts of many query rows (a
// group's prefix, chunks of prompts, drafts), on the tensor cores.
//
// A tile of 128 query rows is the G query heads that share a key head for floor(128 / G)
// consecutive rows of the part; a span is two of them.  Per key tile of 128 positions (whole
// pages, or half of one) and query tile, with S, P and O in TMEM:
//
//     S = Q K^T            (tcgen05.mma, both operands in shared memory)
//     P = 2^(c S - c m)    one thread per query row: 128 scores in registers
//     O += P V             (P from TMEM in place of S, V MN-major as loaded)
//
// The two query tiles take turns on the tensor core: while one's scores are exponentiated,
// the other's products run.  Where a span is only one query
// tile (a small group's prefix, drafts) and has several key tiles, these are dealt to the two
// pipelines instead, each with a maximum, sum and O of its own, and the first joins them: one
// pipeline's chain of products and exponentials, 1.9 us a tile, is longer than the tile's way
// from HBM, 1.5.  The maximum m only follows the true one when it falls behind by more than
// 2^8, so O is rarely rescaled, and the threads that own the rows do it.
//
// On a GB300, 32 query heads on 8 key heads of 128: 16 x 8 beams over prefixes of 8192 positions
// 80 us, 5.5 TB/s; 64 samples over 131,072 positions 109 us, 4.9 TB/s and 1.26 PFLOP/s (without
// its exponentials 96: loads and products); 2048 rows behind 32,768 735 us, 1.54 PFLOP/s.  An item's
// first scores come 4 us after its start: the plan's entry, the page table's, the first keys.
//
// One CTA an SM takes an equal share of the line of all tiles, so a long prefix is spread
// over the card and short parts share a CTA; what it computes of a span whose keys it
// does not have to itself goes to the workspace in fp32.  A page is one or several TMA boxes;
// pages without visible positions are boxes outside the tensor, which read as zeros
// without a trip to memory.
//
// Roles: warps 0-3 and 4-7 the softmax of the two query tiles, warp 8 the items and loads (room
// for two tiles of keys and three of values), warps 9 and 11 the MMAs of the two query tiles, warp 10
// the zeros in place of values that no row sees.
#include <stdint.h>

#include "kda_paged_attend.cuh"
#include "kda_sm100.cuh"
#include "kda_tiles.cuh"

// Poll limit of the softmax's wait for scores.  A test build of the library sets it to
// zero: the wait then gives up at once although its MMAs complete, which takes every
// CTA through the wind-down.
#ifndef KDA_WAIT_LIMIT_PAGED
#define KDA_WAIT_LIMIT_PAGED (1u << 18)
#endif

namespace kda {
namespace {

using namespace sm100;
using namespace tiles;

constexpr int kThreads = 384;
// Room for tiles of keys and of values, which stay longer: until the exponentials are done.  (With room
// for two of them it takes prefetches into L2 to be as fast, 160 us for 167 without, 64 samples.)
constexpr int kKeyRoom = 2, kValueRoom = 3, kRoom = kKeyRoom + kValueRoom;
constexpr int kBars = 3 * kRoom + 23;
constexpr int kStage = 4096;         // bytes of the query tile in which a softmax warp turns its rows of O around
// Registers: a softmax thread holds a row of 128 scores.  The block starts with
// kRegs for each thread and hands them out anew: 2 x 128 x 216 + 128 x 72 of its
// 384 x 168 (the launch checks that the kernel was built with that number).
constexpr int kRegs = 168, kRegsSoftmax = 216, kRegsOther = 72;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreads * kRegs, "more registers than the block has");
constexpr int kDealt = 8;            // key tiles from which one query tile's are dealt
constexpr float kLag = 8.f;          // log2 of what the running maximum may lag behind

// One item of work: a span's rows, one key head, some of the span's key tiles.
struct Item {
    int tokens;                      // rows of the span; 0: there are no more items
    int t0, first;                   // its first row and that row's position
    int hk, shared;
    int tile0, tiles;                // key tiles
    int key0, end;                   // visible positions: key0 .. end - 1, and up to the row's own (not shared)
    int where;                       // goes_to(), and the first row of a cut piece
    int64_t cut;
    // One query tile only: its key tiles are dealt to both pipelines, which are joined in the end.
    // Worth it from some tiles on (16 x 8 beams over 8192 positions 111.8 us without, 108.1 with;
    // three to five tiles of small heads 36.2 and 36.8).
    // Pipeline q takes the tiles whose keys have the q-th room, so that it sees every phase of its
    // barriers there, and need not see the other's.  (Of values it sees some, but always after the
    // one before: the patch warp takes them one after the other.)
    int turn;                        // the room of the item's first keys
    __device__ bool dealt(int tile_tokens) const { return tokens <= tile_tokens && tiles >= kDealt; }
};

struct Ctl {
    Item items[2];
    float2 other_ml[kTileRows];      // maxima and sums over the second pipeline's tiles of a dealt item
    int abort;
    uint32_t tmem;
    uint64_t bars[kBars];
};

// TMEM columns
constexpr int kTmS = 0, kTmO = 256;

template <typename E, int D> struct Layout {
    static constexpr int kTile = 128 * D * 2;            // bytes of a query, key or value tile
    static constexpr int kHalf = 128 * 128;              // bytes of its 64 leftmost columns
    static constexpr int kCtl = (2 + kRoom) * kTile;
    static_assert(4 * kStage <= kTile, "the rows of O are turned around in the query tile");
    static constexpr int kSmem = 1024 + kCtl + sizeof(Ctl);
    static_assert(kSmem <= 227 * 1024, "more shared memory than a CTA has");
    static constexpr bool kF16 = !__is_same(E, __nv_bfloat16);
};

// The place of the g-th tile of keys (kv 0) or of values (1), and which use of it that is.
__device__ __forceinline__ int place(int kv, int g) { return kv ? kKeyRoom + g % kValueRoom : g % kKeyRoom; }
__device__ __forceinline__ int use(int kv, int g) { return kv ? g / kValueRoom : g / kKeyRoom; }

// The barriers; q is a query tile, s a place of the key / value ring, i one of the item
// ring.
struct Bars {
    uint32_t at;
    __device__ uint32_t full(int s) const { return at + 8 * s; }                    // tile loaded
    __device__ uint32_t empty(int s) const { return at + 8 * (kRoom + s); }       // tile consumed by both products
    __device__ uint32_t values(int s) const { return at + 8 * (2 * kRoom + s); }  // value tile without garbage
    __device__ uint32_t q_full(int q) const { return at + 8 * (3 * kRoom + q); }
    __device__ uint32_t q_empty(int q) const { return at + 8 * (3 * kRoom + 2 + q); }
    __device__ uint32_t s_full(int q) const { return at + 8 * (3 * kRoom + 4 + q); }    // scores in TMEM
    __device__ uint32_t p_half(int q) const { return at + 8 * (3 * kRoom + 6 + q); }    // probabilities of 64 keys
    __device__ uint32_t p_ready(int q) const { return at + 8 * (3 * kRoom + 8 + q); }   // of all
    __device__ uint32_t o_done(int q) const { return at + 8 * (3 * kRoom + 10 + q); }   // O complete
    __device__ uint32_t o_free(int q) const { return at + 8 * (3 * kRoom + 12 + q); }   // O read
    __device__ uint32_t turn(int q) const { return at + 8 * (3 * kRoom + 14 + q); }
    __device__ uint32_t drained(int q) const { return at + 8 * (3 * kRoom + 16 + q); }
    __device__ uint32_t item_full(int i) const { return at + 8 * (3 * kRoom + 18 + i); }
    __device__ uint32_t item_empty(int i) const { return at + 8 * (3 * kRoom + 20 + i); }
    __device__ uint32_t other_done() const { return at + 8 * (3 * kRoom + 22); }    // a dealt item's second pipeline is
};
constexpr int kItemReaders = 8 + 2 + 1;   // softmax warps, product warps, patch warp

struct Maps {
    CUtensorMap q, pages;
};

// What every role knows.
struct Ctx {
    const AttendParams &p;
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

// columns of key tile i of an item that may hold visible keys, a multiple of 16
__device__ __forceinline__ int tile_keys(int end, int tile) { return min(kTileKeys, (end - tile * kTileKeys + 15) & ~15); }

// An item's query tile q: its rows of the batch, the last one's position, and how many of the
// item's key tiles any of them sees (the first ones).
struct Span {
    int first, tokens, last, seen;
    __device__ Span(const Item &item, int tile_tokens, int q)
    {
        tokens = max(0, q ? item.tokens - tile_tokens : min(item.tokens, tile_tokens));
        first = item.first + q * tile_tokens;
        last = first + tokens - 1;
        const int end = item.shared ? item.end : min(item.end, last + 1);
        seen = tokens ? min(item.tiles, max(0, (int)(((int64_t)end + kTileKeys - 1) / kTileKeys) - item.tile0)) : 0;
    }
};

// ---- items and loads ---------------------------------------------------------
template <typename E, int D>
__device__ __forceinline__ void load_role(const Ctx &x, const Maps &maps)
{
    using L = Layout<E, D>;
    const AttendParams &p = x.p;
    const PagedCache &cache = p.cache;
    const uint32_t sq = x.base, skv = x.base + 2 * L::kTile;
    const int parts = p.P + p.N, span = 2 * p.tile_tokens, page = 1 << cache.page_log2;
    const int box = min(page, kTileKeys), outside = cache.num_pages * 2 * p.Hk;
    const Lines lines = load_lines(p.lines);
    const int64_t total = lines.total[0], share = lines.share[0];
    const int64_t from = blockIdx.x * share, to = min(total * p.Hk, from + share);
    int64_t at = from;
    int g = 0, item = 0, qs[2] = {0, 0};                 // tiles (of keys and of values each) and query tiles loaded, items written
    int drain[2] = {0, 0};                               // tiles of keys, of values on their way at least once
    bool ok = true;
    for (;; item++) {
        Item &now = x.c.items[item & 1];
        if (item >= 2) ok = x.wait(x.bars.item_empty(item & 1), item / 2 - 1);
        if (!ok) break;
        // the part, span and key head of this place in the line
        int hk = 0, j = 0;
        bool shared = false;
        Part y = {};
        int64_t begin = 0, stop = 0;
        if (at < to) {
            hk = (int)quotient(at, total);
            const int part = part_at(p.tiles, parts, at - hk * total, x.lane);
            shared = part < p.P;
            y = load_part(p.parts + part);
            begin = hk * total + y.begin;
            j = span_at(y, shared, span, at - begin, x.lane);
            begin += span_begin(y, shared, span, j) + tiles_set_up(y);
            stop = begin + span_tiles(y, shared, span, j);
            at = max(at, begin);
        }
        if (at >= to) {
            if (x.lane == 0) {
                now.tokens = 0;
                mbar_arrive(x.bars.item_full(item & 1));
            }
            break;
        }
        const int tile0 = first_tile(y) + (int)(at - begin), n = (int)(min(stop, to) - at);
        const int t0 = y.t0 + j * span, end = span_end(y, shared, span, j);
        at += n;
        if (x.lane == 0) {
            now.tokens = min(span, y.tokens - j * span);
            now.t0 = t0;
            now.first = shared ? 0 : y.first + j * span;
            now.hk = hk;
            now.shared = shared;
            now.tile0 = tile0;
            now.tiles = n;
            now.key0 = y.key0;
            now.end = end;
            now.turn = g & 1;
            now.where = goes_to(y, shared, begin, stop, from, to);
            now.cut = cut_piece(blockIdx.x, begin, from) * kPieceRows;
        }
        __syncwarp();
        const bool now_dealt = now.dealt(p.tile_tokens);
        // The second pipeline waits for the first query tile's queries in dealt items alone: those before
        // these must have come when it does, or it would take their phase, still open, for the one it wants.
        if (now_dealt && qs[0]) ok = x.wait(x.bars.q_full(0), qs[0] - 1);
        if (!ok) break;
        if (x.lane == 0) mbar_arrive(x.bars.item_full(item & 1));
        __syncwarp();
        const int seen[2] = {Span(now, p.tile_tokens, 0).seen, Span(now, p.tile_tokens, 1).seen};
        const int32_t *table = cache.table + (int64_t)y.entry * cache.max_pages;
        // A lane has a box of its own: 64 columns of page rows box lb of a tile.  It loads the entry of
        // the page table one tile ahead.  (One lane for all, as the products have it, took 0.2 us a box,
        // 3 us a tile of small pages.)
        const int lb = x.lane / (D / 64), lh = x.lane % (D / 64);
        auto entry_at = [&](int tile) {
            const int j = (tile * kTileKeys + lb * box) >> cache.page_log2;
            return lb * box < kTileKeys && j < cache.max_pages ? __ldg(table + j) : -1;
        };
        auto load_queries = [&]() {
#pragma unroll 1
            for (int q = 0; q < 2 && ok; q++) {
                if (!seen[q]) continue;
                if (qs[q]) ok = x.wait(x.bars.q_empty(q), qs[q] - 1);
                if (ok && elect_one()) {
                    // half a query tile is G tile_tokens rows of 128 bytes
                    mbar_arrive_expect_tx(x.bars.q_full(q), (uint32_t)(p.G * p.tile_tokens * 128 * (D / 64)));
#pragma unroll
                    for (int h = 0; h < D / 64; h++)
                        tma_load_3d(sq + q * L::kTile + h * L::kHalf, &maps.q, 64 * h, hk * p.G, t0 + q * p.tile_tokens,
                                    x.bars.q_full(q));
                }
                __syncwarp();
                if (ok) qs[q]++;
            }
        };
        int id = entry_at(tile0);
#pragma unroll 1
        for (int i = 0; i < n && ok; i++, g++) {
            const int pos = (tile0 + i) * kTileKeys, at_b = pos + lb * box;
            const int boxes = (tile_keys(end, tile0 + i) + box - 1) / box;
            const bool mine = lb < boxes, needed = mine && at_b + box > y.key0, there = id >= 0 && id < cache.num_pages;
            if (needed && !there && lh == 0) atomicOr(p.err, kErrBadPage);
            const int c1 = at_b & (page - 1), c2 = needed && there ? id * 2 * p.Hk + hk : outside;
            if (i + 1 < n) id = entry_at(tile0 + i + 1);
#pragma unroll 1
            for (int kv = 0; kv < 2; kv++) {
                const int s = place(kv, g), k = use(kv, g);
                if (k) ok = x.wait(x.bars.empty(s), k - 1);
                if (!ok) break;
                const uint32_t bar = x.bars.full(s), dst = skv + s * L::kTile;
                if (elect_one()) mbar_arrive_expect_tx(bar, (uint32_t)(boxes * box * 128 * (D / 64)));
                __syncwarp();
                if (mine)
                    tma_load_3d(dst + lh * L::kHalf + lb * box * 128, &maps.pages, 64 * lh, c1,
                                c2 == outside ? outside : c2 + kv * p.Hk, bar);
                __syncwarp();
                drain[kv]++;
                // The first item's queries come behind the first keys; later ones' room is free only when
                // the output is written, and two tiles need not wait for that.
                if (kv == 0 && i == 0 && item == 0) load_queries();
            }
            if (ok && i == min(1, n - 1) && item) load_queries();
        }
        // The first keys of the next item may be for a pipeline that did not see the tile before them in
        // their room.
        if (now_dealt)
            for (int i = g - kKeyRoom; i < g && ok; i++) ok = x.wait(x.bars.full(place(0, i)), use(0, i));
        if (!ok) break;
    }
    if (!ok && x.lane == 0) x.give_up();
    // nothing may still be on its way into shared memory when the CTA ends
#pragma unroll 1
    for (int q = 0; q < 2; q++)
        if (qs[q]) mbar_wait_drain(x.bars.q_full(q), (qs[q] - 1) & 1);
#pragma unroll 1
    for (int kv = 0; kv < 2; kv++)
        for (int i = max(0, drain[kv] - (kv ? kValueRoom : kKeyRoom)); i < drain[kv]; i++)
            mbar_wait_drain(x.bars.full(place(kv, i)), use(kv, i) & 1);
}

// ---- products of one query tile ---------------------------------------------------
// The whole warp walks the loop and one elected lane issues: operands that are
// uniform over the warp stay in uniform registers, where the instruction takes them.
// The two query tiles take turns, so that one's scores are exponentiated during the
// other's products.
template <typename E, int D>
__device__ __forceinline__ void product_role(const Ctx &x, int which)
{
    using L = Layout<E, D>;
    const AttendParams &p = x.p;
    const int q = __shfl_sync(0xffffffffu, which, 0);
    const uint32_t tm = __shfl_sync(0xffffffffu, x.tmem, 0);
    const uint32_t ts = tm + kTmS + 128 * q, to = tm + kTmO + 128 * q;
    const uint32_t qs = x.base + q * L::kTile, skv = x.base + 2 * L::kTile;
    // tiles consumed; products P V issued; turns taken; items with rows; query tiles used
    int g = 0, parts = 0, turns = 0, mine = 0, queries[2] = {0, 0};
    bool ok = true;
    for (int item = 0; ok; item++) {
        const Item &now = x.c.items[item & 1];
        ok = x.wait(x.bars.item_full(item & 1), item / 2);
        const int tokens = __shfl_sync(0xffffffffu, now.tokens, 0);
        if (!ok || tokens == 0) break;
        const bool both = tokens > p.tile_tokens, dealt = __shfl_sync(0xffffffffu, now.dealt(p.tile_tokens), 0);
        const int seen = __shfl_sync(0xffffffffu, Span(now, p.tile_tokens, dealt ? 0 : q).seen, 0);
        const int seen0 = __shfl_sync(0xffffffffu, Span(now, p.tile_tokens, 0).seen, 0);
        const int n = __shfl_sync(0xffffffffu, now.tiles, 0), tile0 = __shfl_sync(0xffffffffu, now.tile0, 0);
        const int end = __shfl_sync(0xffffffffu, now.end, 0);
        const bool any = seen > 0;
        if (dealt) {
            ok = x.wait(x.bars.q_full(0), queries[0]);
#pragma unroll 1
            for (int i = (q + __shfl_sync(0xffffffffu, now.turn, 0)) & 1; i < n && ok; i += 2) {
                const int sk = place(0, g + i), sv = place(1, g + i);
                ok = x.wait(x.bars.full(sk), use(0, g + i));
                const int keys = tile_keys(end, tile0 + i);
                const bool last = i + 2 >= n;
                if (ok && elect_one()) {
                    mma_scores<D>(ts, x.base, skv + sk * L::kTile, idesc(keys, 0, L::kF16));
                    mma_commit(x.bars.s_full(q));
                    mma_commit(x.bars.empty(sk));        // for both pipelines
                    mma_commit(x.bars.empty(sk));
                }
                __syncwarp();
                ok = ok && x.wait(x.bars.values(sv), use(1, g + i));
                if (ok && i < 2 && mine > 0) ok = x.wait(x.bars.o_free(q), mine - 1);
                ok = ok && x.wait(x.bars.p_half(q), parts);
                if (ok) {
                    tc_fence_after();
                    if (elect_one()) mma_values<D>(to, ts, skv + sv * L::kTile, idesc(D, 1, L::kF16), 0, keys / 16, i > 1);
                    ok = x.wait(x.bars.p_ready(q), parts);
                }
                if (ok) {
                    tc_fence_after();
                    if (elect_one()) {
                        mma_values<D>(to, ts, skv + sv * L::kTile, idesc(D, 1, L::kF16), 4, keys / 16, true);
                        mma_commit(x.bars.empty(sv));
                        mma_commit(x.bars.empty(sv));
                        if (last) mma_commit(x.bars.o_done(q));
                    }
                    parts++;
                }
                __syncwarp();
            }
            g += n;
        } else {
            int keys = tile_keys(end, tile0);
            ok = x.wait(x.bars.full(place(0, g)), use(0, g)) && (!any || x.wait(x.bars.q_full(q), queries[q]));
            if (elect_one()) {
                if (ok && any) {
                    mma_scores<D>(ts, qs, skv + place(0, g) * L::kTile, idesc(keys, 0, L::kF16));
                    mma_commit(x.bars.s_full(q));
                }
                mma_commit(x.bars.empty(place(0, g)));
            }
            __syncwarp();
            for (int i = 0; i < n && ok; i++, g++) {
                const int sv = place(1, g), steps = keys / 16;    // this tile's values
                ok = x.wait(x.bars.values(sv), use(1, g));
                const int sk = place(0, g + 1);          // the next tile's keys
                const bool have = i + 1 < n;
                if (have) {
                    keys = tile_keys(end, tile0 + i + 1);
                    ok = ok && x.wait(x.bars.full(sk), use(0, g + 1));
                }
                __syncwarp();
                if (both && ok && (q || turns)) ok = x.wait(x.bars.turn(q), q ? turns : turns - 1);
                if (ok && i < seen) {
                    if (i == 0 && mine > 0) ok = x.wait(x.bars.o_free(q), mine - 1);
                    ok = ok && x.wait(x.bars.p_half(q), parts);
                    if (ok) {
                        tc_fence_after();
                        if (elect_one()) mma_values<D>(to, ts, skv + sv * L::kTile, idesc(D, 1, L::kF16), 0, steps, i > 0);
                        ok = x.wait(x.bars.p_ready(q), parts);
                    }
                    if (ok) {
                        tc_fence_after();
                        if (elect_one()) mma_values<D>(to, ts, skv + sv * L::kTile, idesc(D, 1, L::kF16), 4, steps, true);
                        parts++;
                    }
                }
                if (elect_one()) {
                    if (ok && have && i + 1 < seen) {
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
        }
        if (any) mine++;
        if (seen0) queries[0]++;
        if (q && any && !dealt) queries[1]++;
        __syncwarp();
        if (x.lane == 0) mbar_arrive(x.bars.item_empty(item & 1));
    }
    if (!ok && x.lane == 0) x.give_up();
    // every product is finished before the TMEM and shared memory go
    if (elect_one()) mma_commit(x.bars.drained(q));
    mbar_wait_drain(x.bars.drained(q), 0);
}

// ---- zeros in place of values that no row sees ----------------------------------------
// Value rows before the first key and behind the last hold anything, and 0 x NaN is NaN.
// Every value tile passes through here.
template <typename E, int D>
__device__ __forceinline__ void patch_role(const Ctx &x)
{
    using L = Layout<E, D>;
    bool ok = true;
    for (int item = 0, g = 0; ok; item++) {
        const Item &now = x.c.items[item & 1];
        ok = x.wait(x.bars.item_full(item & 1), item / 2);
        if (!ok || now.tokens == 0) break;
        const int n = now.tiles;
        for (int i = 0; i < n && ok; i++, g++) {
            const int s = place(1, g);
            ok = x.wait(x.bars.full(s), use(1, g));
            if (!ok) break;
            const int pos = (now.tile0 + i) * kTileKeys, keys = tile_keys(now.end, now.tile0 + i);
            if (pos < now.key0 || pos + keys > now.end) {
#pragma unroll 1
                for (int e = x.lane; e < keys * (D / 8); e += 32) {
                    const int r = e / (D / 8), v = e % (D / 8);
                    if (pos + r < now.key0 || pos + r >= now.end)
                        *reinterpret_cast<uint4 *>(x.smem + (2 + s) * L::kTile + (v / 8) * L::kHalf + r * 128 + (v % 8) * 16) =
                            make_uint4(0, 0, 0, 0);
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
    const AttendParams &p = x.p;
    const int q = warp >> 2, row = 32 * (warp & 3) + x.lane, lane = x.lane;
    const int token = row * p.inv_G >> 16;               // row / G
    const uint32_t lanes = x.tmem + ((uint32_t)(warp & 3) << 21);
    const uint32_t ts = lanes + kTmS + 128 * q, to = lanes + kTmO + 128 * q;
    const float c2 = p.scale_log2;
    uint8_t *stage = x.smem + q * L::kTile + (warp & 3) * kStage;   // (every product with the queries is done by then)
    int it = 0, mine = 0, joined = 0;                    // score tiles, items with rows, dealt ones
    bool ok = true;
    for (int item = 0; ok; item++) {
        const Item &now = x.c.items[item & 1];
        ok = x.wait(x.bars.item_full(item & 1), item / 2);
        if (!ok || now.tokens == 0) break;
        const bool dealt = now.dealt(p.tile_tokens);
        const int qt = dealt ? 0 : q, now_turn = now.turn;           // whose rows these are
        const Span rows(now, p.tile_tokens, qt);
        const bool dead = 32 * (warp & 3) >= rows.tokens * p.G;      // no row of this warp is one: O may be anything
        const int key0 = now.key0, tile0 = now.tile0, t0 = now.t0 + qt * p.tile_tokens, hk = now.hk, where = now.where;
        const int64_t cut = now.cut + qt * kTileRows;
        // behind the last key that this row sees, and that the warp's first row does
        const int see = now.shared ? now.end : min(now.end, rows.first + token + 1);
        const int least = now.shared ? now.end : min(now.end, rows.first + (32 * (warp & 3) * p.inv_G >> 16) + 1);
        float m = -INFINITY, sum = 0.f;
        const int end = now.end;
        for (int i = dealt ? (q + now_turn) & 1 : 0; i < rows.seen; i += dealt ? 2 : 1) {
            const int pos = (tile0 + i) * kTileKeys, keys = tile_keys(end, tile0 + i);
            // every key of the tile visible to every row of the warp: no test per key
            const bool whole = pos >= key0 && pos + kTileKeys <= least;
            // Lanes may give up one by one: the vote on the maxima below is also the one on
            // that; a lane that gave up goes on until then with what its row of TMEM holds.
            const bool got = mbar_wait(x.bars.s_full(q), it & 1, x.abort, KDA_WAIT_LIMIT_PAGED);
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
            for (int k = 0; k < 4; k++)
                if (32 * k < keys) tmem_ld32(ts + 32 * k, s[k]);
            loaded(s[0], s[1], s[2], s[3]);
            if (!whole) {
#pragma unroll
                for (int k = 0; k < 4; k++) {            // visible columns
                    const uint32_t seen = below(see - pos - 32 * k) & ~below(key0 - pos - 32 * k);
#pragma unroll
                    for (int j = 0; j < 32; j++)
                        if (!(seen & (1u << j))) s[k][j] = 0xff800000u;   // -inf
                }
            }
            float mx[4];
#pragma unroll
            for (int k = 0; k < 4; k++) {
                mx[k] = __uint_as_float(s[k][0]);
#pragma unroll
                for (int j = 1; j < 32; j++) mx[k] = fmaxf(mx[k], __uint_as_float(s[k][j]));
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
                for (int k = 0; k < D / 32; k++) {
                    uint32_t o[32];
                    tmem_ld32(to + 32 * k, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; j++) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                    tmem_st32(to + 32 * k, o);
                }
                tmem_wait_st();
                sum *= f;
                if (behind) m = top;
            }
            if (m == -INFINITY) m = top;                 // the row's first visible keys: its O is still zero
            const float now_c = slope<E>(m, c2), z = m == -INFINITY ? 0.f : -m * now_c;
            float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int k = 0; k < 4; k++) {
                if (k == 2) {                            // the first 64 keys are in TMEM: their product can start
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(x.bars.p_half(q));
                }
                if (32 * k < keys) {
                    uint32_t w[16];
#pragma unroll
                    for (int j = 0; j < 16; j++) {
                        float2 e = fma2(make_float2(__uint_as_float(s[k][2 * j]), __uint_as_float(s[k][2 * j + 1])),
                                        make_float2(now_c, now_c), make_float2(z, z));
                        e.x = ex2(e.x);
                        e.y = ex2(e.y);
                        part[j & 1] = add2(part[j & 1], e);
                        w[j] = Half2<E>::pack(e.x, e.y);
                    }
                    tmem_st16(ts + 16 * k, w);
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
        const int live = rows.tokens * p.G - 32 * (warp & 3);        // of this warp's rows
        const int64_t dense = (int64_t)t0 * p.Hq + hk * p.G;         // row of [T][Hq] of the tile's first row
        if (rows.seen) {
            ok = x.wait(x.bars.o_done(q), mine);
            if (!ok) break;
            tc_fence_after();
            mine++;
        }
        // What O, and that of the second pipeline, is multiplied by.  Pieces with other maxima are joined by
        // exact ones: the weights lose what slope m was rounded by, up to 2^-24 of its size.
        float f0 = 1.f, f1 = 0.f;
        auto exactly = [&](float m) { return m == -INFINITY ? 0.f : residue(m, slope<E>(m, c2)); };
        if (dealt) {
            if (q) {
                x.c.other_ml[row] = make_float2(m, sum);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(x.bars.other_done());
                continue;
            }
            ok = x.wait(x.bars.other_done(), joined++);
            if (!ok) break;
            tc_fence_after();
            const float2 other = x.c.other_ml[row];
            const float top = fmaxf(m, other.x);
            f0 = m == -INFINITY ? 0.f : ex2((m - top) * c2 - exactly(m));
            f1 = other.x == -INFINITY ? 0.f : ex2((other.x - top) * c2 - exactly(other.x));
            sum = sum * f0 + other.y * f1;
            m = top;
        } else if (where != kToOut) {
            f0 = ex2(-exactly(m));
            sum *= f0;
        }
        if (where != kToOut && lane < live) {            // the row's maximum (or what stands for it) and sum
            float2 *ml = where == kToCut ? p.cut_tiles_ml + cut + row
                                         : p.whole_ml[where == kToPrefix] + dense + token * (p.Hq - p.G) + row;
            *ml = make_float2(m, sum);
        }
        if (!rows.seen) continue;                        // nothing visible in this piece: no O
        // the room of the query tile, written and read here, for the next one's copy
        auto free_queries = [&]() {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(x.bars.q_empty(q));
        };
        // 32 columns of O, multiplied by f; after the last ones it is free for the next item
        auto load_o = [&](int h, float f, uint32_t (&o)[32]) {
            tmem_ld32(to + 32 * h, o);
            tmem_wait_ld();
            if (dealt) {
                uint32_t other[32];
                tmem_ld32(to + 128 + 32 * h, other);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; j++)
                    o[j] = __float_as_uint(fmaf(__uint_as_float(other[j]), f1 * f, __uint_as_float(o[j]) * (f0 * f)));
            } else {
#pragma unroll
                for (int j = 0; j < 32; j++) o[j] = __float_as_uint(__uint_as_float(o[j]) * (f0 * f));
            }
            if (h == D / 32 - 1) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(x.bars.o_free(q));
                    if (dealt) mbar_arrive(x.bars.o_free(1));
                }
            }
        };
        if (where != kToOut) {
            // O in fp32, 32 columns at a time through shared memory, so that a store
            // instruction writes four rows of 128 bytes
            float *out = where == kToCut ? p.cut_tiles + cut * D : p.whole[where == kToPrefix] + dense * D;
            const int skip = where == kToCut ? 0 : p.Hq - p.G;       // rows between two tokens'
#pragma unroll 1
            for (int h = 0; h < D / 32; h++) {
                uint32_t o[32];
                load_o(h, 1.f, o);
#pragma unroll
                for (int j = 0; j < 8; j++)
                    *reinterpret_cast<uint4 *>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                        make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const int rr = 4 * j + (lane >> 3), r = 32 * (warp & 3) + rr, tok = r * p.inv_G >> 16;
                    const uint4 v = *reinterpret_cast<const uint4 *>(stage + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
                    if (rr < live) *reinterpret_cast<uint4 *>(out + ((int64_t)tok * skip + r) * D + 32 * h + 4 * (lane & 7)) = v;
                }
                __syncwarp();
            }
            free_queries();
            continue;
        }
        // O / sum in 16 bits, 64 columns at a time
        const float inv = 1.f / sum;
        uint16_t *out = p.out + dense * D + 8 * (lane & 7);
#pragma unroll 1
        for (int h = 0; h < D / 64; h++) {
#pragma unroll
            for (int k = 0; k < 2; k++) {
                uint32_t o[32];
                load_o(2 * h + k, inv, o);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    uint4 r;
                    r.x = Half2<E>::pack(__uint_as_float(o[8 * j]), __uint_as_float(o[8 * j + 1]));
                    r.y = Half2<E>::pack(__uint_as_float(o[8 * j + 2]), __uint_as_float(o[8 * j + 3]));
                    r.z = Half2<E>::pack(__uint_as_float(o[8 * j + 4]), __uint_as_float(o[8 * j + 5]));
                    r.w = Half2<E>::pack(__uint_as_float(o[8 * j + 6]), __uint_as_float(o[8 * j + 7]));
                    *reinterpret_cast<uint4 *>(stage + lane * 128 + (((4 * k + j) ^ (lane & 7)) << 4)) = r;
                }
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const int rr = 4 * j + (lane >> 3), r = 32 * (warp & 3) + rr, tok = r * p.inv_G >> 16;
                const uint4 v = *reinterpret_cast<const uint4 *>(stage + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
                if (rr < live) *reinterpret_cast<uint4 *>(out + ((int64_t)tok * (p.Hq - p.G) + r) * D + 64 * h) = v;
            }
            __syncwarp();
        }
        free_queries();
    }
    if (!ok) x.give_up();
}

template <typename E, int D>
__global__ void __launch_bounds__(kThreads, 1)
paged_tiles_kernel(const __grid_constant__ Maps maps, const __grid_constant__ AttendParams p)
{
    using L = Layout<E, D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - smem_u32(smem_raw));
    Ctl &c = *reinterpret_cast<Ctl *>(smem + L::kCtl);
    const Bars bars{smem_u32(c.bars)};
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp == 8 && lane == 0) {
        c.abort = 0;
        for (int s = 0; s < kRoom; s++) {
            mbar_init(bars.full(s), 1);
            mbar_init(bars.empty(s), 2);
            mbar_init(bars.values(s), 1);
        }
        for (int q = 0; q < 2; q++) {
            mbar_init(bars.q_full(q), 1);
            mbar_init(bars.q_empty(q), 4);
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
        mbar_init(bars.other_done(), 4);
        mbar_fence_init();
        tma_prefetch_desc(&maps.q);
        tma_prefetch_desc(&maps.pages);
    }
    if (warp == 9) {
        tmem_alloc(smem_u32(&c.tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // the plan is complete, for this kernel and for the rows kernel behind it
    grid_wait();
    grid_go_on();
    const Ctx x{p, c, bars, smem, base, c.tmem, lane, &c.abort};
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == 8) load_role<E, D>(x, maps);
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

template <typename E, int D>
cudaError_t launch(const PagedAttentionArgs &a, const AttendParams &p)
{
    const int page = 1 << a.cache.page_log2, box = page < kTileKeys ? page : kTileKeys;
    Maps maps;
    if (!make_map(&maps.q, a.q, a.f16, D, a.Hq, D, a.T, a.q_stride, p.G, p.tile_tokens) ||
        !make_map(&maps.pages, a.cache.pages, a.f16, D, page, D, (int64_t)a.cache.num_pages * 2 * a.Hk, (int64_t)page * D, box, 1))
        return cudaErrorInvalidValue;
    const int smem = Layout<E, D>::kSmem;
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = once_per_device(ready, a.device, [&]() {
        cudaFuncAttributes built;
        cudaError_t r = cudaFuncGetAttributes(&built, paged_tiles_kernel<E, D>);
        if (r == cudaSuccess && built.numRegs != kRegs) r = cudaErrorInvalidConfiguration;
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(paged_tiles_kernel<E, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        return r;
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.tile_workers);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, paged_tiles_kernel<E, D>, maps, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t launch_paged_tiles(const PagedAttentionArgs &a, const AttendParams &p)
{
    if (a.d == 128) return a.f16 ? launch<__half, 128>(a, p) : launch<__nv_bfloat16, 128>(a, p);
    return a.f16 ? launch<__half, 64>(a, p) : launch<__nv_bfloat16, 64>(a, p);
}

}  // namespace kda
