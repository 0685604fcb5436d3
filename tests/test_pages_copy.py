"""Copies of positions between slots of paged caches, bit for bit."""
import random

import pytest

import kda_linear_attention_chunk_gb300 as kda
from gpu_util import torch

pytestmark = pytest.mark.gpu


def scene(moves, page=64, heads=(2,), d=128, dtype=None, slots=20, seed=0, extra=1):
    """moves: [(src, dst, lo, hi)]; caches, the page table on host and device."""
    t = torch()
    r = random.Random(seed)
    width = max([1] + [-(-hi // page) for *_, hi in moves]) + extra
    pages = list(range(slots * width + 3))
    r.shuffle(pages)
    rows = [[pages[s * width + j] for j in range(width)] for s in range(slots)]
    g = t.Generator(device="cuda")
    g.manual_seed(seed)
    caches = [t.randn(len(pages), 2, h, page, d, generator=g, device="cuda").to(dtype or t.bfloat16) for h in heads]
    return caches, rows, t.tensor(rows, dtype=t.int32, device="cuda")


def copied(caches, rows, moves, page):
    t = torch()
    out = [c.clone() for c in caches]
    for s, to, lo, hi in moves:
        if s < 0 or to < 0 or lo >= hi:
            continue
        p = t.arange(lo, hi, device="cuda")
        a, b = (t.tensor(rows[x], device="cuda")[p // page] for x in (s, to))
        for c, o in zip(caches, out):
            o[b, :, :, p % page] = c[a, :, :, p % page]
    return out


def run(moves, **kw):
    t = torch()
    page = kw.get("page", 64)
    caches, rows, table = scene(moves, **kw)
    want = copied(caches, rows, moves, page)
    i32 = lambda x: t.tensor(x, dtype=t.int32, device="cuda")   # noqa: E731
    src, dst, lo, hi = (i32(x) for x in zip(*moves))
    kda.pages_copy(caches, table, src, dst, hi, start=lo)
    for c, w in zip(caches, want):
        assert t.equal(c, w)
    assert kda.device_error(reset=True) == 0


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("lo,hi", [(0, 1), (0, 16), (15, 17), (5, 6), (63, 65), (0, 257), (255, 256), (100, 1000), (7, 7), (9, 3)])
def test_ranges(page, lo, hi):
    run([(3, 5, lo, hi), (3, 7, 0, 2), (1, 2, lo + 1, hi + 30)], page=page, seed=lo + hi)


@pytest.mark.parametrize("d,heads", [(64, (1,)), (128, (3, 8, 1)), (64, (2,) * 5), (256, (2,)), (8, (4,))])
def test_layers_and_heads(d, heads):
    t = torch()
    run([(0, 1, 3, 200), (0, 2, 70, 90), (4, 3, 0, 0), (-1, 5, 0, 9), (6, -1, 0, 9), (7, 7, 0, 30)], d=d, heads=heads)
    run([(0, 1, 3, 50)], d=d, heads=heads, dtype=t.float32)


def test_many_moves():
    r = random.Random(5)
    slots = 3000
    ids = list(range(slots))
    r.shuffle(ids)
    moves = []
    for to in ids[:1500]:
        lo = r.randint(0, 40)
        moves.append((ids[r.randint(1500, slots - 1)], to, lo, lo + r.randint(0, 60)))
    run(moves, page=32, heads=(1, 2), d=64, slots=slots)


def test_more_moves_than_a_grid_axis_holds():
    moves = [(i, -1, 0, 5) for i in range(66000)]
    moves[0] = (0, 1, 0, 5)
    moves[65534], moves[65535], moves[65999] = (0, 2, 0, 5), (0, 3, 1, 6), (0, 4, 2, 7)
    moves = [(min(a, 19), b, c, e) for a, b, c, e in moves]
    run(moves, page=16, d=64)


def test_without_start_and_without_rows():
    t = torch()
    caches, rows, table = scene([(0, 1, 0, 100)])
    want = copied(caches, rows, [(0, 1, 0, 100)], 64)
    i32 = lambda *x: t.tensor(x, dtype=t.int32, device="cuda")   # noqa: E731
    kda.pages_copy(caches, table, i32(0), i32(1), i32(100))
    assert t.equal(caches[0], want[0])
    none = t.empty(0, dtype=t.int32, device="cuda")
    kda.pages_copy(caches, table, none, none, none)
    assert t.equal(caches[0], want[0])


def test_bad_tables_are_reported_and_stay_in_bounds():
    t = torch()
    caches, rows, table = scene([(0, 1, 0, 200)])
    i32 = lambda *x: t.tensor(x, dtype=t.int32, device="cuda")   # noqa: E731
    kda.device_error(reset=True)
    was = caches[0].clone()
    kda.pages_copy(caches, table, i32(-2, 0, 20), i32(1, 20, 2), i32(50, 50, 50))
    assert kda.device_error(reset=True) == kda.ERR_BAD_SLOT and t.equal(caches[0], was)
    capacity = table.shape[1] * 64
    kda.pages_copy(caches, table, i32(0, 3), i32(1, 4), i32(0x7fffffff, 10), start=i32(capacity - 3, -5))
    assert kda.device_error(reset=True) == kda.ERR_BAD_POSITION
    want = copied([was], rows, [(0, 1, capacity - 3, capacity), (3, 4, 0, 10)], 64)[0]
    assert t.equal(caches[0], want)
    caches[0].copy_(was)
    bad = table.clone()
    bad[0, 1], bad[1, 2] = -1, 1 << 30                 # no source: zeros; no target: nothing
    kda.pages_copy(caches, bad, i32(0), i32(1), i32(200))
    assert kda.device_error(reset=True) == kda.ERR_BAD_PAGE
    want = copied([was], rows, [(0, 1, 0, 128), (0, 1, 192, 200)], 64)[0]
    want[rows[1][1]] = 0
    assert t.equal(caches[0], want)


def test_graphs_and_streams():
    t = torch()
    moves = [(0, 1, 3, 200), (0, 2, 70, 90)]
    caches, rows, table = scene(moves, heads=(2, 3))
    want = copied(caches, rows, moves, 64)
    was = [c.clone() for c in caches]
    src, dst, lo, hi = (t.tensor(x, dtype=t.int32, device="cuda") for x in zip(*moves))
    side = t.cuda.Stream()
    t.cuda.synchronize()
    kda.pages_copy(caches, table, src, dst, hi, start=lo, stream=side)
    t.cuda.synchronize()
    assert all(t.equal(c, w) for c, w in zip(caches, want))
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        kda.pages_copy(caches, table, src, dst, hi, start=lo)
    for c, w in zip(caches, was):
        c.copy_(w)
    g.replay()
    t.cuda.synchronize()
    assert all(t.equal(c, w) for c, w in zip(caches, want))


def test_places_beyond_2_31_elements():
    t = torch()
    many = (1 << 31) // (2 * 8 * 256 * 128) + 3
    big = t.zeros(many, 2, 8, 256, 128, dtype=t.bfloat16, device="cuda")
    big[many - 1] = 1
    table = t.tensor([[many - 1], [many - 2]], dtype=t.int32, device="cuda")
    i32 = lambda *x: t.tensor(x, dtype=t.int32, device="cuda")   # noqa: E731
    kda.pages_copy([big], table, i32(0), i32(1), i32(256))
    assert bool((big[many - 2:] == 1).all()) and not big[:many - 2].any()
