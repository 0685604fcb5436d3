"""Appending to a paged cache: q against the 64-bit form, the pages bit for bit beside what must not change."""
import math
import random

import pytest

import kda_linear_attention_chunk_gb300 as kda
from gpu_util import torch
from hybrid_util import beside_pending_work, f64, norm_rope, torch_dtype, worst
from paged_util import Batch

pytestmark = pytest.mark.gpu


class Rows:
    def __init__(self, own, page=64, Hq=8, Hk=2, d=128, dtype="bf16", rotary=64, layout="half", norm=True, weights=True,
                 seed=0, fused=True):
        t = torch()
        self.b = b = Batch(own, page=page, Hq=Hq, Hk=Hk, d=d, dtype=dtype, seed=seed)
        g = t.Generator(device="cuda")
        g.manual_seed(seed + 1)
        qkv = (2 * t.randn(b.T, Hq + 2 * Hk, d, generator=g, device="cuda")).to(torch_dtype(dtype))
        self.q, self.k, self.v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        if not fused:
            self.q, self.k, self.v = (x.contiguous() for x in (self.q, self.k, self.v))
        self.w = [1 + 0.2 * t.randn(d, generator=g, device="cuda") for _ in range(2)] if weights else [None, None]
        self.top = max([1] + [a + n for a, n in zip(b.start, b.lens)])
        self.table = kda.rope_table(self.top, rotary) if rotary else None
        self.kw = dict(q_weight=self.w[0], k_weight=self.w[1], table=self.table, layout=layout, norm=norm)
        self.layout, self.norm, self.dtype = layout, norm, dtype

    def call(self, pool, **over):
        b = self.b
        args = dict(q=self.q, k=self.k, v=self.v, kv_pages=pool, page_table=b.table, starts=b.starts, cu_seqlens=b.cu_dev,
                    slots=b.slots, **self.kw)
        args.update(over)
        return kda.paged_append(**args)

    def check(self, out, pool, skip=()):
        """q within its bound; k as head_norm_rope gives it, v as it is, in their places; nothing else touched."""
        import numpy as np
        b, t = self.b, torch()
        pos = [a + i for a, n in zip(b.start, b.lens) for i in range(n)]
        w = self.w[0]
        ref, bound = norm_rope(f64(self.q), None if w is None else f64(w), None if self.table is None else f64(self.table),
                               np.array(pos, dtype=int), self.layout, 1e-6, self.norm, self.dtype)
        live = np.ones(b.T, dtype=bool)
        for n in skip:
            live[b.cu[n]:b.cu[n + 1]] = False
        assert worst(f64(out)[live], ref[live], bound[live]) <= 1
        turned = kda.head_norm_rope(self.q, self.k, positions=t.tensor(pos, dtype=t.int32, device="cuda"), **self.kw) \
            if b.T else (self.q, self.k)
        assert t.equal(out[t.tensor(live, device="cuda")], turned[0][t.tensor(live, device="cuda")])
        want = t.full_like(pool, 5.0)
        for n, L in enumerate(b.lens):
            if L and n not in skip:
                p, r = b.places(b.ids[n], b.start[n], b.start[n] + L)
                want[p, 0, :, r] = turned[1][b.cu[n]:b.cu[n + 1]]
                want[p, 1, :, r] = self.v[b.cu[n]:b.cu[n + 1]]
        assert t.equal(pool, want)


def run(rows, skip=(), **over):
    pool = torch().full_like(rows.b.pool, 5.0)
    out = rows.call(pool, **over)
    rows.check(out, pool, skip)
    return out


@pytest.mark.parametrize("layout,rotary", [("half", 128), ("half", 64), ("interleaved", 128), ("interleaved", 16), ("half", 0),
                                           ("half", 48)])
@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16")])
def test_layouts(layout, rotary, d, dtype):
    run(Rows([(5, 40), (0, 1), (63, 2), (64, 0), (200, 100)], d=d, dtype=dtype, rotary=min(rotary, d), layout=layout))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 3), (40, 5), (9, 9), (64, 1)])
def test_pages_and_heads(page, Hq, Hk):
    run(Rows([(page - 1, 3), (0, page + 1), (3 * page, 1)], page=page, Hq=Hq, Hk=Hk, seed=Hq))


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("N", [1, 2, 31, 33, 200])
def test_single_rows(N, fused):
    r = random.Random(N)
    rows = Rows([(r.randint(0, 300), 1) for _ in range(N)], fused=fused, seed=N)
    assert torch().equal(run(rows), run(rows, cu_seqlens=None))


def test_without_weights_norm_or_start():
    run(Rows([(7, 9)], weights=False))
    run(Rows([(7, 9)], norm=False))
    rows = Rows([(0, 9), (0, 30)])
    run(rows, starts=None)


@pytest.mark.parametrize("N", [1, 5, 40, 1500])
def test_many_sequences_some_empty(N):
    r = random.Random(N)
    run(Rows([(r.randint(0, 50), r.choice([0, 0, 1, 3, 20])) for _ in range(N)] + [(4, 2)], Hq=2, Hk=1, d=64, seed=N))


def test_padded_sequences_rows_behind_and_in_place():
    t = torch()
    rows = Rows([(10, 3), (20, 4), (30, 5)], fused=False)
    b = rows.b
    slots = b.slots.clone()
    slots[1] = -1
    pool, out = t.full_like(b.pool, 5.0), t.full_like(rows.q, 7.0)
    rows.call(pool, slots=slots, out=out)
    rows.check(out, pool, skip=(1,))
    assert (out[3:7] == 7).all()
    # rows behind the last sequence
    pad = lambda x: t.cat([x, t.full_like(x[:2], math.nan)])   # noqa: E731
    pool, out = t.full_like(b.pool, 5.0), t.full_like(pad(rows.q), 7.0)
    rows.call(pool, q=pad(rows.q), k=pad(rows.k), v=pad(rows.v), out=out)
    rows.check(out[:-2], pool)
    assert (out[-2:] == 7).all()
    # in place
    want, q = rows.call(t.full_like(b.pool, 5.0)), rows.q.clone()
    assert rows.call(t.full_like(b.pool, 5.0), q=q, out=q) is q and t.equal(q, want)
    assert kda.device_error(reset=True) == 0


def test_bad_tables_are_reported_and_stay_in_bounds():
    t = torch()
    rows = Rows([(60, 10), (0, 3)])
    b = rows.b
    i32 = lambda *x: t.tensor(x, dtype=t.int32, device="cuda")   # noqa: E731

    def word(**over):
        pool = t.full_like(b.pool, 5.0)
        out = rows.call(pool, **over)
        return out, pool, kda.device_error(reset=True)

    kda.device_error(reset=True)
    _, good, w = word()
    assert w == 0
    table = b.table.clone()
    table[b.ids[0], 1] = -1
    out, pool, w = word(page_table=table)
    assert w == kda.ERR_BAD_PAGE
    p, r = b.places(b.ids[0], 64, 70)                  # the rows of that page are dropped, all others written
    good[p, :, :, r] = 5.0
    assert t.equal(pool, good)
    table[b.ids[0], 1] = b.pool.shape[0]
    assert t.equal(word(page_table=table)[1], good)
    _, pool, w = word(slots=i32(-2, 4000))
    assert w == kda.ERR_BAD_SLOT and (pool == 5).all()
    capacity = b.table.shape[1] * b.page
    for starts in ((-1, 0), (0, capacity - 2), (0, 0x7fffffff)):
        assert word(starts=i32(*starts))[2] & kda.ERR_BAD_POSITION, starts
    assert word(cu_seqlens=i32(0, 500, 13))[2] & kda.ERR_BAD_SEQLENS
    assert word(cu_seqlens=i32(-9, 10, 13))[2] & kda.ERR_BAD_SEQLENS
    short = kda.rope_table(65, 64)
    assert word(table=short)[2] == kda.ERR_BAD_POSITION
    # more rows than the table has positions for: those that fit are cached
    many = Rows([(0, 5 * 64)])
    assert many.b.table.shape[1] == 6
    pool = t.full_like(many.b.pool, 5.0)
    many.call(pool, page_table=many.b.table[:, :3].contiguous())
    assert kda.device_error(reset=True) == kda.ERR_BAD_POSITION
    want = t.full_like(pool, 5.0)
    whole = t.full_like(pool, 5.0)
    many.call(whole)
    p, r = many.b.places(many.b.ids[0], 0, 192)
    want[p, :, :, r] = whole[p, :, :, r]
    assert t.equal(pool, want)


def test_streams_and_graphs():
    t = torch()
    rows = Rows([(60, 10), (0, 300), (9, 1)])
    pool, again = t.full_like(rows.b.pool, 5.0), t.full_like(rows.b.pool, 5.0)
    want = rows.call(pool)
    got = beside_pending_work(lambda side: rows.call(again, stream=side), want.shape, want.dtype)
    assert t.equal(got, want) and t.equal(again, pool)
    again.fill_(5)
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        out = rows.call(again)
    out.zero_()
    again.fill_(5)
    g.replay()
    t.cuda.synchronize()
    assert t.equal(out, want) and t.equal(again, pool)


def test_places_beyond_2_31_elements():
    t = torch()
    rows = Rows([(5, 3)], page=256, Hk=8, d=128)
    b = rows.b
    many = (1 << 31) // b.pool[0].numel() + 3
    big = t.zeros(many, *b.pool.shape[1:], dtype=b.pool.dtype, device="cuda")
    table = t.full_like(b.table, many - 1)
    rows.call(big, page_table=table)
    pool = t.zeros_like(b.pool)
    rows.call(pool)
    assert t.equal(big[many - 1], pool[b.rows[b.ids[0]][0]]) and not big[:many - 1].any()
