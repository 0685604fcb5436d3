"""kda_slots_copy and kda_slots_compact on the GPU: bytes against host copies."""
import numpy as np
import pytest

import kda_linear_attention_chunk_gb300 as kda
from gpu_util import torch
from hybrid_util import beside_pending_work

pytestmark = pytest.mark.gpu


def make_pools(n, seed, shapes=((3, 7, 8), (16,), (2, 5, 100, 64))):
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(seed)
    dts = (t.float32, t.bfloat16, t.float16)
    return [t.randn((n,) + s, generator=g, device="cuda").to(dt) for s, dt in zip(shapes, dts)]


def int32(x):
    t = torch()
    return t.tensor(x, dtype=t.int32, device="cuda")


def host(pools):
    return [p.cpu().clone() for p in pools]


@pytest.mark.parametrize("n,src,dst", [
    (1, [0], [0]), (2, [0], [1]), (5, [3, 3, 3, -1], [0, 1, 4, 2]), (9, [2, -1, 5, 7], [-1, -1, 6, 0]),
    (40, [39] * 20, list(range(20))), (7, [-1] * 7, list(range(7)))])
def test_copies_forks_and_clears(n, src, dst):
    t = torch()
    pools = make_pools(n, seed=n)
    was = host(pools)
    kda.slots_copy(pools, int32(src), int32(dst))
    for p, w in zip(pools, was):
        want = w.clone()
        for a, b in zip(src, dst):
            if b >= 0:
                want[b] = w[a] if a >= 0 else 0
        assert t.equal(p.cpu(), want)


def test_large_entries_and_many_pools():
    """Entries over several pieces with ragged ends, more pools than a warp has lanes, an odd number of moves."""
    t = torch()
    sizes = [8, 2 * 8192 + 8, 16384, 40000] + [8 * (i + 1) for i in range(40)]
    pools = [t.arange(6 * s, device="cuda", dtype=t.int32).to(t.int16).view(6, s) for s in sizes]
    was = host(pools)
    kda.slots_copy(pools, int32([1, 1, -1]), int32([0, 5, 4]))
    for p, w in zip(pools, was):
        want = w.clone()
        want[0], want[5], want[4] = w[1], w[1], 0
        assert t.equal(p.cpu(), want)


def test_bad_ids_are_reported_and_skipped():
    t = torch()
    pools = make_pools(4, seed=2)
    was = host(pools)
    kda.device_error(reset=True)
    kda.slots_copy(pools, int32([4, 0, -2, 1]), int32([0, 9, 1, 2]))
    assert kda.device_error(reset=True) == kda.ERR_BAD_SLOT
    for p, w in zip(pools, was):
        want = w.clone()
        want[2] = w[1]
        assert t.equal(p.cpu(), want)


def compacted(table, n):
    live = sorted(x for x in table if x >= 0)
    m = len(live)
    free = [x for x in range(m) if x not in set(live)]
    to = {x: x if x < m else free.pop(0) for x in live}
    return [to[x] if x >= 0 else -1 for x in table]


def table_of(n, live, seed, pads=3):
    rng = np.random.default_rng(seed)
    table = [int(x) for x in rng.permutation(n)[:live]] + [-1] * pads
    return [table[i] for i in rng.permutation(len(table))]


@pytest.mark.parametrize("n,live", [(1, 1), (1, 0), (2, 1), (31, 30), (32, 7), (33, 20), (64, 64), (100, 1), (1000, 400),
                                    (1024, 512), (5000, 2500), (70000, 3000)])
def test_compaction(n, live):
    t = torch()
    pools = make_pools(n, seed=live, shapes=((2, 4), (24,)) if n > 100 else ((3, 7, 8), (16,), (2, 5, 100, 64)))
    table = table_of(n, live, seed=n)
    was = host(pools)
    got = kda.slots_compact(pools, int32(table))
    want = compacted(table, n)
    assert got.tolist() == want
    for p, w in zip(pools, was):
        after = w.clone()
        for a, b in zip(table, want):
            if a >= 0:
                after[b] = w[a]
        assert t.equal(p.cpu(), after)


def test_compaction_at_the_largest_number_of_slots():
    n = kda.KDA_MAX_POOL_SLOTS
    t = torch()
    pool = t.arange(n, device="cuda", dtype=t.int64)[:, None].repeat(1, 2).contiguous()
    table = table_of(n, 6000, seed=1)
    got = kda.slots_compact([pool], int32(table))
    want = compacted(table, n)
    assert got.tolist() == want
    host_pool = pool.cpu()
    assert all(host_pool[b, 0] == a for a, b in zip(table, want) if a >= 0)


def test_compaction_reports_bad_ids():
    pools = make_pools(6, seed=3)
    was = host(pools)
    kda.device_error(reset=True)
    got = kda.slots_compact(pools, int32([5, 6, -1, -7, 2]))
    assert kda.device_error(reset=True) == kda.ERR_BAD_SLOT
    assert got.tolist() == compacted([5, -1, -1, -1, 2], 6)
    for p, w in zip(pools, was):
        for a, b in zip([5, 2], [got[0].item(), got[4].item()]):
            assert torch().equal(p[b].cpu(), w[a])


def test_other_stream():
    t = torch()
    pools = make_pools(8, seed=4)
    was = host(pools)
    t.cuda.synchronize()
    src, dst = int32([1, 2]), int32([5, 6])
    t.cuda.synchronize()
    s = t.cuda.Stream()
    kda.slots_copy(pools, src, dst, stream=s)
    s.synchronize()
    for p, w in zip(pools, was):
        assert t.equal(p[5].cpu(), w[1]) and t.equal(p[6].cpu(), w[2])


def test_compact_result_on_a_given_stream():
    t = torch()
    pools, slots = make_pools(6, seed=14), int32([5, -1, 3])
    kda.slots_compact(make_pools(6, seed=14), slots)
    got = beside_pending_work(lambda s: kda.slots_compact(pools, slots, stream=s), (3,), t.int32)
    assert got.tolist() == compacted([5, -1, 3], 6)
