"""Attention over a paged cache with shared prefixes against its 64-bit form.  Every place that holds no visible position is
NaN, so a key read where none is visible shows."""
import math
import random

import pytest

import kda_linear_attention_chunk_gb300 as kda
from gpu_util import torch
from hybrid_util import beside_pending_work, torch_dtype
from paged_util import Batch, attention64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16")])
def test_decode_contexts_around_pages_and_tiles(page, d, dtype):
    own = [(c, 1) for c in (0, 1, 14, 15, 16, 17, 63, 64, 65, 126, 127, 128, 129, 255, 256, 300, 1000, 2048)]
    b = Batch(own, page=page, d=d, dtype=dtype, seed=page)
    b.check(b.call())
    assert b.t.equal(b.call(), b.call(cu_seqlens=None))


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (8, 8), (6, 2), (5, 1), (16, 1), (17, 1), (40, 2), (128, 1), (64, 2), (33, 11)])
@pytest.mark.parametrize("d,dtype", [(128, "fp16"), (64, "bf16")])
def test_head_groups(Hq, Hk, d, dtype):
    own = [(200, 1), (5, 3), (0, 40), (77, 17), (0, 1)]
    b = Batch(own, Hq=Hq, Hk=Hk, d=d, dtype=dtype, seed=Hq)
    b.check(b.call())
    b = Batch([(20, 1), (0, 2), (130, 1), (3, 1)], [(3, 150), (1, 10)], Hq=Hq, Hk=Hk, d=d, dtype=dtype, seed=Hq)
    b.check(b.call())


@pytest.mark.parametrize("prefix", [1, 15, 16, 17, 63, 64, 127, 128, 129, 500, 2049])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_prefixes_that_end_inside_pages(prefix, page):
    """Members with nothing of their own but the new row, with a few rows, and with many."""
    own = [(0, 1), (1, 1), (3, 2), (130, 1), (0, 70), (17, 1)]
    b = Batch(own, [(6, prefix)], page=page, seed=prefix)
    b.check(b.call())


@pytest.mark.parametrize("members", [1, 2, 4, 5, 8, 31, 32, 33, 64, 65, 130])
def test_group_sizes(members):
    """From fewer than 16 query rows a key head to several query tiles."""
    r = random.Random(members)
    own = [(r.randint(0, 90), 1) for _ in range(members + 3)]
    b = Batch(own, [(members, 700), (2, 129)], Hq=8, Hk=2, seed=members)
    b.check(b.call())
    assert b.t.equal(b.call(cu_seqlens=None), b.call(cu_seqlens=None))


@pytest.mark.parametrize("N", [1, 7, 37, 150, 153, 600])
@pytest.mark.parametrize("keys", [1, 17, 100, 900, 1100])
def test_many_short_parts(N, keys):
    """Few steps a part: workers' shares end before a part's first step, at it and behind it."""
    r = random.Random(N + keys)
    own = [(r.randint(0, keys - 1), r.choice([1, 1, 2, 5]) if N < 200 else 1) for _ in range(N)]
    b = Batch(own, Hq=8, Hk=2, d=64, page=32, seed=N)
    b.check(b.call())
    b = Batch(own, [(N // 3, keys), (N // 2, 3)], Hq=8, Hk=2, d=64, page=32, seed=N)
    b.check(b.call())


@pytest.mark.parametrize("tokens", [17, 64, 65, 130])
def test_many_short_spans(tokens):
    own = [((i * 37) % 300, tokens - i % 3) for i in range(60)]
    b = Batch(own, Hq=8, Hk=2, d=64, page=64, seed=tokens)
    b.check(b.call())


def test_groups_of_all_kinds():
    """Empty groups, a group without a prefix, sequences of none, empty sequences inside a group."""
    own = [(3, 1), (0, 0), (9, 5), (0, 1), (40, 1), (0, 0), (7, 30), (300, 1)]
    b = Batch(own, [(3, 100), (0, 50), (2, 0), (2, 333)], seed=4)
    b.check(b.call())
    groups, lens, slots = b.prefixes
    none = slots.clone()
    none[1] = none[2] = -1
    assert b.t.equal(b.call(prefixes=(groups, lens, none)), b.call())


@pytest.mark.parametrize("rows", [2, 5, 31, 33, 64, 65, 127, 200, 513])
@pytest.mark.parametrize("context", [0, 1, 100, 1023])
def test_several_rows(rows, context):
    b = Batch([(context, rows), (context // 2, rows // 2), (context, 1)], Hq=8, Hk=2, seed=rows + context)
    b.check(b.call())


@pytest.mark.parametrize("own,groups", [([(60000, 1)], []), ([(33000, 1), (5, 1), (9, 1)], [(3, 20000)]),
                                        ([(0, 3000)], []), ([(40000, 9)], []), ([(0, 1500), (5, 1), (12000, 3)], [])])
def test_long_contexts(own, groups):
    b = Batch(own, groups, Hq=8, Hk=2, seed=len(own))
    b.check(b.call())


@pytest.mark.parametrize("N", [700, 2500])
def test_many_short_sequences(N):
    """More of them than the plan takes at a time."""
    r = random.Random(8)
    own = [(r.randint(0, 40), r.choice([0, 1, 1, 1, 2, 7])) for _ in range(N)]
    b = Batch(own, [(100, 60), (50, 7)] + [(3, 20)] * (N // 4 - 60), Hq=4, Hk=2, d=64, seed=8)
    b.check(b.call())


@pytest.mark.parametrize("seed", range(12))
def test_any_batch(seed):
    r = random.Random(seed + 100)
    N = r.choice([1, 3, 17, 40])
    own = [(r.choice([0, 3, 100, r.randint(0, 1500)]), r.choice([1, 1, 1, 0, 4, r.randint(1, 90)])) for _ in range(N)]
    groups, left = [], N
    while left and r.random() < 0.7:
        m = r.randint(1, left)
        groups.append((m, r.choice([0, 1, 64, r.randint(1, 2000)])))
        left -= m
    Hk = r.choice([1, 2, 3])
    b = Batch(own, groups, page=r.choice([16, 32, 64, 128, 256]), Hk=Hk, Hq=Hk * r.choice([1, 3, 4, 8, 16]),
              d=r.choice([64, 128]), dtype=r.choice(["bf16", "fp16"]), seed=seed, scale=r.choice([None, 0.02, 0.3]))
    b.check(b.call())


@pytest.mark.parametrize("groups", [[], [(4, 200)]])
def test_padded_sequences_and_rows_behind_the_last(groups):
    own = [(10, 1), (20, 4), (5, 40), (100, 1), (30, 2)]
    b = Batch(own, groups, seed=1)
    t = b.t
    slots = b.slots.clone()
    slots[1] = -1
    slots[3] = -1
    q = t.cat([b.q, t.full((7, b.Hq, b.d), math.nan, dtype=b.q.dtype, device="cuda")])
    out = t.full_like(q, 3.0)
    b.call(q=q, slots=slots, out=out)
    b.check(out, skip=(1, 3))
    for n in (1, 3):
        assert (out[b.cu[n]:b.cu[n + 1]] == 3).all()
    assert (out[b.T:] == 3).all()
    assert kda.device_error(reset=True) == 0


def test_strided_queries_and_table_rows_as_slots():
    own = [(10, 1), (200, 3), (5, 50)]
    b = Batch(own, seed=2)
    t = b.t
    wide = t.full((b.T, b.Hq + 3, b.d), math.nan, dtype=b.q.dtype, device="cuda")
    wide[:, 1:1 + b.Hq] = b.q
    want = b.call()
    assert t.equal(b.call(q=wide[:, 1:1 + b.Hq]), want)
    rows = b.table[b.slots.long()].contiguous()
    assert t.equal(b.call(page_table=rows, slots=None), want)


def test_nothing_to_do():
    b = Batch([(0, 0), (5, 0)], seed=2)
    assert b.call().shape == (0, b.Hq, b.d)
    assert b.call(cu_seqlens=None, starts=None, slots=None).shape == (0, b.Hq, b.d)


def test_bad_tables_are_reported_and_stay_in_bounds():
    own = [(100, 1), (50, 20), (200, 1), (0, 1)]
    b = Batch(own, [(2, 70)], seed=6)
    t, want = b.t, b.call()
    i32 = lambda *x: t.tensor(x, dtype=t.int32, device="cuda")   # noqa: E731

    def word(**over):
        out = t.full_like(b.q, 9.0)
        b.call(out=out, **over)
        return out, kda.device_error(reset=True)

    kda.device_error(reset=True)
    slots = b.slots.clone()
    slots[1], slots[2] = 1000, -7
    out, w = word(slots=slots)
    assert w == kda.ERR_BAD_SLOT and (out[1:22] == 9).all()
    b.check(out, skip=(1, 2))                          # (another batch is cut up in another way: not the same bytes)
    groups, lens, kept = b.prefixes
    out, w = word(prefixes=(groups, lens, i32(99)))
    assert w & kda.ERR_BAD_SLOT
    table = b.table.clone()
    table[b.ids[2], 1] = 1 << 30                       # a page in the middle of a context reads as zeros
    zeroed = Batch(own, [(2, 70)], seed=6)
    zeroed.pool[zeroed.rows[zeroed.ids[2]][1]] = 0
    out, w = word(page_table=table)
    assert w == kda.ERR_BAD_PAGE
    zeroed.check(out)
    table[b.kept[0], 0] = -1                           # and in a prefix
    zeroed.pool[zeroed.rows[zeroed.kept[0]][0]] = 0
    out, w = word(page_table=table)
    assert w == kda.ERR_BAD_PAGE
    zeroed.check(out)
    _, w = word(starts=i32(-5, 1 << 30, 0x7fffffff, 0))
    assert w & kda.ERR_BAD_POSITION
    _, w = word(prefixes=(groups, i32(-3), kept))
    assert w & kda.ERR_BAD_POSITION
    _, w = word(prefixes=(groups, i32(0x7fffffff), kept))
    assert w & kda.ERR_BAD_POSITION
    _, w = word(prefixes=(i32(-4, 900), lens, kept))
    assert w & kda.ERR_BAD_SEQLENS
    _, w = word(cu_seqlens=i32(0, 5, 1000, -4, 23))
    assert w & kda.ERR_BAD_SEQLENS
    assert t.equal(b.call(), want) and kda.device_error(reset=True) == 0


def test_a_start_inside_the_prefix_is_moved_to_its_end():
    b = Batch([(0, 1), (0, 3)], [(2, 100)], seed=3)
    want = b.call()
    got = b.call(starts=b.starts - 40)
    assert b.t.equal(got, want) and kda.device_error(reset=True) == kda.ERR_BAD_POSITION


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("size", [1e-3, 30.0])
def test_scores_of_all_sizes(dtype, size):
    """From nearly equal scores to ones of which a single key takes everything."""
    b = Batch([(300, 1), (100, 20), (2000, 1)], [(2, 260)], dtype=dtype, loud=size, seed=5)
    b.check(b.call())


def test_other_rows_stay_apart_from_values_that_are_not_finite():
    """A sequence whose values hold infinities reaches no other, nor the members of another group."""
    own = [(50, 1), (60, 20), (70, 1), (40, 1)]
    b = Batch(own, [(2, 90), (1, 33)], seed=7)
    t = b.t
    want = b.call()
    p, r = b.places(b.ids[3], 0, 30)
    b.pool[p, 1, :, r] = math.inf
    p, r = b.places(b.kept[1], 0, 33)
    b.pool[p, 1, :, r] = -math.inf
    got = b.call()
    assert t.equal(got[:21], want[:21]) and not t.isfinite(got[21:]).any()


def test_keys_that_are_not_finite_behind_the_mask():
    """Keys past a row's position: infinite and NaN ones of later rows of its sequence."""
    b = Batch([(40, 30)], seed=9)
    t, want = b.t, b.call()
    p, r = b.places(b.ids[0], 60, 70)
    b.pool[p, 0, :, r] = math.nan
    got = b.call()
    assert t.equal(got[:20], want[:20])
    b.pool[p, 0, :, r] = math.inf
    got = b.call()
    assert t.equal(got[:20], want[:20])


def test_places_beyond_2_31_elements():
    """Pages far apart in a cache of more than 2^31 elements, and rows of queries likewise."""
    t = torch()
    b = Batch([(200, 1), (10, 40)], [(1, 100)], page=256, Hq=8, Hk=8, seed=3)
    n = b.pool.shape[0]
    many = (1 << 31) // (b.pool[0].numel()) + 50
    big = t.empty(many, *b.pool.shape[1:], dtype=b.pool.dtype, device="cuda")
    at = [many - 1 - 7 * i for i in range(n)]
    big[t.tensor(at, device="cuda")] = b.pool
    table = t.where(b.table >= 0, t.tensor(at, device="cuda", dtype=t.int32)[b.table.clamp_min(0).long()], -1).int()
    want = b.call()
    assert t.equal(b.call(kv_pages=big, page_table=table), want)
    del big
    stride = (1 << 31) // 20 // 8 * 8
    wide = t.empty(b.T * stride, dtype=b.q.dtype, device="cuda").as_strided((b.T, b.Hq, b.d), (stride, b.d, 1))
    wide.copy_(b.q)
    assert t.equal(b.call(q=wide), want)


def test_repeated_and_other_streams():
    t = torch()
    b = Batch([(500, 1), (40, 33), (7000, 1)], [(2, 300)], seed=11)
    want = b.call()
    for _ in range(3):
        assert t.equal(b.call(), want)
    streams = [t.cuda.Stream() for _ in range(4)]
    t.cuda.synchronize()
    outs = []
    for s in streams * 3:                              # calls that overlap, each with a workspace of its own
        with t.cuda.stream(s):
            outs.append(b.call())
    t.cuda.synchronize()
    assert all(t.equal(o, want) for o in outs)
    got = beside_pending_work(lambda side: b.call(stream=side), want.shape, want.dtype)
    assert t.equal(got, want)


def test_replayed_graphs():
    """Two graphs of one pool, replayed in turn and at the same time on two streams where their memory is their own."""
    t = torch()
    b = Batch([(500, 1), (40, 20), (900, 1)], [(2, 300)], seed=12)
    want = b.call()
    graphs, outs = [], []
    for _ in range(2):
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            outs.append(b.call())
        graphs.append(g)
    for o in outs:
        o.zero_()
    streams = [t.cuda.Stream() for _ in range(2)]
    t.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with t.cuda.stream(s):
                g.replay()
    t.cuda.synchronize()
    assert all(t.equal(o, want) for o in outs)
    # a graph follows its inputs: longer contexts next time
    c = Batch([(700, 1), (140, 20), (200, 1)], [(2, 310)], seed=13, extra=2)
    d = Batch([(300, 1), (10, 20), (900, 1)], [(2, 310)], seed=13, extra=2)
    if c.table.shape[1] >= d.table.shape[1]:
        args = [x.clone() for x in (c.q, c.table, c.starts, c.slots)]
        pool = t.zeros(max(c.pool.shape[0], d.pool.shape[0]), *c.pool.shape[1:], dtype=c.pool.dtype, device="cuda")
        lens = c.prefixes[1].clone()
        kept = c.prefixes[2].clone()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            out = kda.paged_attention(args[0], pool, args[1], starts=args[2], cu_seqlens=c.cu_dev, slots=args[3],
                                      prefixes=(c.prefixes[0], lens, kept))
        for x in (c, d):
            pool[:x.pool.shape[0]] = x.pool
            args[0].copy_(x.q)
            args[1].fill_(-1)
            args[1][:, :x.table.shape[1]] = x.table[:, :args[1].shape[1]]
            args[2].copy_(x.starts)
            args[3].copy_(x.slots)
            lens.copy_(x.prefixes[1])
            kept.copy_(x.prefixes[2])
            g.replay()
            t.cuda.synchronize()
            x.check(out)
    assert torch_dtype("bf16") is b.q.dtype


def test_rows_past_the_tables_end_are_left_as_they_were():
    """More rows than the table has positions for: those that fit are answered."""
    b = Batch([(0, 200)], page=64, seed=14, extra=0)
    t = b.t
    table = b.table[:, :2].contiguous()
    out = t.full_like(b.q, 6.0)
    b.call(page_table=table, out=out)
    assert kda.device_error(reset=True) == kda.ERR_BAD_POSITION
    ref, bound = b.want(0)
    assert ((out[:128].double() - ref[:128]).abs() <= bound[:128]).all() and (out[128:] == 6).all()


def test_an_empty_sequence_in_a_group_may_start_anywhere():
    b = Batch([(5, 2), (0, 0), (3, 1)], [(3, 100)], seed=15)
    starts = b.starts.clone()
    starts[1] = 0
    b.check(b.call(starts=starts))
    assert kda.device_error(reset=True) == 0


def test_infinite_scores_are_masked():
    """Keys that no row sees yet hold values whose scores would be infinite; rows that do see one have no finite answer."""
    b = Batch([(70, 20), (40, 1)], seed=16, dtype="fp16")
    t, want = b.t, b.call()
    p, r = b.places(b.ids[0], 85, 90)
    b.pool[p, 0, :, r] = -math.inf
    got = b.call()
    assert t.equal(got[:15], want[:15]) and t.equal(got[20:], want[20:])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("scale", [1e-30, 0.01, 1e10, 1e30, 9e36])
def test_scores_times_scales_of_any_size(dtype, scale):
    """Whole numbers, so that the scores are exact: the largest one takes all where the scale is large, equal ones share."""
    b = Batch([(300, 1), (700, 40), (2000, 1), (0, 3)], [(2, 260)], dtype=dtype, seed=17, scale=scale)
    t = b.t
    b.q.copy_(t.randint(-2, 3, b.q.shape, device="cuda"))
    live = ~b.pool[:, 0].isnan()
    b.pool[:, 0] = t.where(live, t.randint(-2, 3, live.shape, device="cuda").to(b.pool.dtype), b.pool[:, 0])
    out = b.call()
    for n, L in enumerate(b.lens):
        k, v = b.keys(n)
        pos = t.arange(b.start[n], b.start[n] + L, device="cuda")
        ref, bound = attention64(b.q[b.cu[n]:b.cu[n + 1]].double(), k, v, pos, scale, dtype, whole=True)
        off = ((out[b.cu[n]:b.cu[n + 1]].double() - ref).abs() / bound).max().item()
        assert off <= 1, (n, off)


def test_a_query_that_is_not_finite_keeps_to_its_row():
    """Also where rows of other sequences are in its tile, as of a shared prefix."""
    b = Batch([(20, 1), (300, 1), (7, 30), (40, 1)] + [(9, 1)] * 6, [(2, 500), (7, 90)], seed=18)
    t, want = b.t, b.call()
    q = b.q.clone()
    rows = [1, 10, 34]
    q[rows] = math.nan
    q[rows[1], 0] = math.inf
    got = b.call(q=q)
    others = [i for i in range(b.T) if i not in rows]
    assert t.equal(got[others], want[others]) and got[rows].isnan().all()


def test_a_member_may_own_the_prefix():
    """The prompt's own slot goes on as one of the group."""
    b = Batch([(30, 1), (12, 2), (0, 1)], [(3, 150)], page=64, seed=19)
    t, want = b.t, b.call()
    table, pool = b.table.clone(), b.pool.clone()
    kept, own = b.kept[0], b.ids[0]
    for j in range(150 // 64 + 1, table.shape[1]):
        table[kept, j] = table[own, j]
    tail = b.rows[kept][150 // 64]                     # the page that the prefix ends in goes on with the member's rows
    pool[tail, :, :, 150 % 64:] = pool[b.rows[own][150 // 64], :, :, 150 % 64:]
    slots = b.slots.clone()
    slots[0] = kept
    assert t.equal(b.call(page_table=table, kv_pages=pool, slots=slots), want)


@pytest.mark.parametrize("cu,groups", [((0, 30, 10, 40, 41), (0, 2, 4)), ((0, 1, 21, 40, 41), (2, 1, 4)),
                                       ((40, 30, 20, 10, 0), (0, 4, 2)), ((0, 20, 41, 20, 41), (4, 0, 4))])
def test_tables_out_of_order_stay_in_bounds(cu, groups):
    """cu_seqlens and groups that go back: the results are undefined, but the call ends, writes its rows only, and the next one
    is right."""
    b = Batch([(20, 1), (30, 20), (100, 19), (50, 1)], [(2, 200), (2, 90)], seed=20)
    t = b.t
    i32 = lambda x: t.tensor(x, dtype=t.int32, device="cuda")   # noqa: E731
    room = t.full((b.T + 2, b.Hq, b.d), 4.0, dtype=b.q.dtype, device="cuda")
    b.call(cu_seqlens=i32(cu), prefixes=(i32(groups), *b.prefixes[1:]), out=room[1:-1])
    t.cuda.synchronize()
    assert (room[0] == 4).all() and (room[-1] == 4).all()
    kda.device_error(reset=True)
    b.check(b.call())
