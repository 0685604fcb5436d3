"""kda_window_prefill where few rows a sequence on average hide long sequences: those go to the tensor-core tiles, the
others to the warp-MMA kernel, in one call.  Against softmax attention in 64 bits, and the ring cache bit for bit."""
import numpy as np
import pytest

import kda_linear_attention_chunk_gb300 as kda
from gpu_util import torch
from test_window import Batch

pytestmark = pytest.mark.gpu

PICKS = [0, 1, 2, 15, 16, 31, 63, 64, 65, 127, 128, 129, 255, 300, 511, 600]


# A sequence of more than 256 query rows a key head is long; the batch has at least 1024 of them, and 32 a sequence at
# most.
@pytest.mark.parametrize("Hq,Hk,lens", [
    (8, 2, [65, 64, 64, 66] + [0] * 40), (8, 2, [0] * 40 + [65, 64, 64, 66]), (8, 2, [64] * 4 + [0] * 40),
    (8, 2, [64, 65, 64, 0, 66] + [1] * 60), (8, 2, [0] * 31 + [300] + [0] * 100),
    (8, 2, [0] * 32 + [300, 2, 300] + [3] * 130), (2, 2, [257, 256, 255, 258] + [1] * 30),
    (2, 2, [256, 258, 600] + [0] * 60), (8, 1, [33, 32, 1, 34, 40] + [0] * 40), (128, 1, [3, 2, 1, 0, 4] + [0] * 60),
    (20, 1, [13, 12, 200] + [0] * 147), (8, 2, [600] + [0] * 90 + [70] + [1] * 40 + [0] * 30 + [129])])
def test_long_sequences_among_short_ones(Hq, Hk, lens):
    b = Batch([(37 * i) % 90 for i in range(len(lens))], Hq, Hk, 64, window=40, sinks=3, dtype="bf16", seed=len(lens))
    b.prefill(lens, check_rows=PICKS)
    b.prefill(lens[::-1], check_rows=PICKS)


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16"), (128, "fp16")])
def test_sizes_and_types(d, dtype):
    lens = [1, 0, 140, 2, 90] + [0] * 20 + [1] * 30
    b = Batch([5 * i for i in range(len(lens))], 8, 2, d, window=70, sinks=2, dtype=dtype, seed=d)
    b.prefill(lens, check_rows=PICKS)


def test_without_a_cache_and_without_starts():
    lens = [0] * 30 + [200, 1, 1, 0, 77] + [0] * 40
    Batch([0] * len(lens), 8, 2, 64, window=60, sinks=4, dtype="bf16", seed=2).prefill(lens, cached=False, check_rows=PICKS)
    Batch([0] * len(lens), 8, 2, 64, window=60, sinks=4, dtype="bf16", seed=3).prefill(lens, starts=False, check_rows=PICKS)


def test_padded_long_and_short_sequences():
    lens = [100, 1, 150, 2, 0, 66] + [1] * 60
    b = Batch([3 * i for i in range(len(lens))], 8, 2, 64, window=30, sinks=2, dtype="bf16", seed=4)
    b.prefill(lens, padded=(0, 3, 7), check_rows=PICKS)
    b.prefill(lens, padded=(0, 2, 5), check_rows=PICKS)


def test_bad_slots_and_starts_are_reported_once_and_skipped():
    t = torch()
    lens = [100, 1, 150, 2, 80] + [0] * 60
    b = Batch([4] * len(lens), 8, 2, 64, window=30, sinks=2, dtype="bf16", seed=5)
    q, k, v = b.new_rows(sum(lens))
    cu = b.int32(np.concatenate([[0], np.cumsum(lens)]).tolist())
    ids, starts = b.ids(), b.int32([4] * len(lens))
    ids[0], ids[1], starts[2] = b.pool.shape[0], -5, -1
    out, was = t.full((sum(lens), 8, 64), 7.0, dtype=q.dtype, device="cuda"), b.pool.clone()
    kda.device_error(reset=True)
    kda.window_prefill(q, k, v, cu, 30, sinks=2, kv_pool=b.pool, slots=ids, starts=starts, out=out)
    assert kda.device_error(reset=True) == kda.ERR_BAD_SLOT | kda.ERR_BAD_POSITION
    assert (out[:101] == 7.0).all() and not (out[101:] == 7.0).all(-1).any()
    changed = (b.pool.view(t.int16) != was.view(t.int16)).flatten(1).any(1).nonzero().flatten().tolist()
    assert set(changed) == {b.slots[n] for n in (2, 3, 4)}


def test_bad_sequence_tables_stay_in_bounds():
    """Rows past the call's, and a table that falls: reported, and nothing outside the outputs is written."""
    t = torch()
    b = Batch([0] * 40, 8, 2, 64, window=30, sinks=0, dtype="bf16", seed=6)
    q, k, v = b.new_rows(300)
    ids, starts = b.ids(), b.int32([0] * 40)
    for table in ([0] * 20 + [90] * 20 + [4000], [0] * 5 + [150] * 10 + [-7] * 25 + [200], [0] * 39 + [400, 200]):
        around = t.full((700, 8, 64), 7.0, dtype=q.dtype, device="cuda")
        kda.device_error(reset=True)
        kda.window_prefill(q, k, v, b.int32(table), 30, kv_pool=b.pool, slots=ids, starts=starts, out=around[200:500])
        assert kda.device_error(reset=True) & kda.ERR_BAD_SEQLENS
        assert (around[:200] == 7.0).all() and (around[500:] == 7.0).all()


def test_same_bytes_every_time_in_a_graph_and_behind_other_calls():
    """Calls of one stream follow one another closely: each one's cache is the next one's input."""
    t = torch()
    lens = [90, 1, 200] + [1] * 40 + [0] * 30
    b = Batch([50] * len(lens), 8, 2, 128, window=100, sinks=4, dtype="bf16", seed=7)
    b.pool.normal_()
    q, k, v = b.new_rows(sum(lens))
    cu, ids = b.int32(np.concatenate([[0], np.cumsum(lens)]).tolist()), b.ids()
    starts = [b.int32([50 + i * n for n in lens]) for i in range(6)]
    out = [t.empty(sum(lens), 8, 128, dtype=q.dtype, device="cuda") for _ in starts]

    def chain(pool, wait):
        for s, o in zip(starts, out):
            kda.window_prefill(q, k, v, cu, 100, sinks=4, kv_pool=pool, slots=ids, starts=s, out=o)
            if wait:
                t.cuda.synchronize()

    first = b.pool.clone()
    chain(first, True)
    want = [o.clone() for o in out]
    for _ in range(5):
        pool = b.pool.clone()
        chain(pool, False)
        assert all(t.equal(x, y) for x, y in zip(out, want)) and t.equal(pool, first)
    pool = b.pool.clone()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        chain(pool, False)
    for _ in range(3):
        pool.copy_(b.pool)
        graph.replay()
        t.cuda.synchronize()
        assert all(t.equal(x, y) for x, y in zip(out, want)) and t.equal(pool, first)


def test_long_sequences_anywhere_in_a_large_table():
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.integers(0, 4, 2500)]
    for n in (0, 31, 32, 1023, 1024, 1055, 1056, 2047, 2400, 2499):
        lens[n] = int(rng.integers(60, 200))
    b = Batch([int(x) for x in rng.integers(0, 30, 2500)], 4, 1, 64, window=20, sinks=1, dtype="bf16", seed=8)
    b.prefill(lens, padded=(1024, 1700), check_rows=[0, 1, 2, 63, 64, 127, 128, 199])
