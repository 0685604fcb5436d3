"""Beam selection over vocabularies whose last slice is short (a CTA whose threads do not all have a logit)."""
import numpy as np
import pytest

import kda_linear_attention_chunk_gb300 as kda
from gpu_util import torch
from test_beam import check, draw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [505, 511, 513, 518, 600, 1023, 1300, 1789, 1795, 2047, 32000])
@pytest.mark.parametrize("B", [1, 4, 8, 9, 16, 32, 33, 64])
def test_short_slices(V, B):
    for dtype in ("bf16", "fp16", "fp32")[:1 if V > 5000 else 3]:
        x, scores, slots = draw(1, B, V, dtype, seed=V + B)
        check(x, scores, slots=slots)


@pytest.mark.parametrize("V", [50257, 128256])
@pytest.mark.parametrize("B", [4, 8])
def test_usual_vocabularies(V, B):
    x, scores, slots = draw(2, B, V, "bf16", seed=B)
    check(x, scores, slots=slots)


def a_call(V, B, dtype):
    """Microseconds of a call, of 20 captured ones."""
    t = torch()
    x, scores, _ = draw(1, B, V, dtype, seed=1)
    s = t.tensor(scores, dtype=t.float32, device="cuda")
    kda.beam_select(x, s)
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        for _ in range(20):
            kda.beam_select(x, s)
    best = float("inf")
    for _ in range(8):
        a, b = t.cuda.Event(enable_timing=True), t.cuda.Event(enable_timing=True)
        a.record()
        g.replay()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 50)
    return best


@pytest.mark.parametrize("B", [16, 32])
@pytest.mark.parametrize("V,full", [(1300, 2048), (513, 2048)])
def test_a_short_slice_takes_no_longer_than_a_full_one(V, full, B):
    """Fewer logits in as many CTAs: at most the time of the full slices, and half of it more for what a clock does."""
    short, whole = a_call(V, B, "bf16"), a_call(full, B, "bf16")
    assert short <= 1.5 * whole, (short, whole)


@pytest.mark.parametrize("B", [16, 32, 64])
def test_many_slices_take_no_rounds_over_all_their_candidates(B):
    """Sixteen slices of 2048 logits for one, in other CTAs: a round has more lists to look at, and as many rounds."""
    many, one = a_call(32768, B, "bf16"), a_call(2048, B, "bf16")
    assert many <= 4 * one, (many, one)


@pytest.mark.parametrize("V", [32768, 100000])
@pytest.mark.parametrize("B", [16, 31, 64])
def test_many_slices(V, B):
    """Steps with one hypothesis, with ended beams, and with equal logits, whose candidates are taken from the lists."""
    r = np.random.RandomState(V)
    x, scores, slots = draw(1, B, V, "bf16", seed=B)
    check(x, scores, (r.rand(1, B) < 0.3).astype(np.int32), 17, slots)
    x[1:] = x[:1]
    check(x, 0 * scores, slots=slots)
    scores[:, 1:] = -np.inf
    check(x, scores, slots=slots)


@pytest.mark.parametrize("V", [300, 4096, 40000])
def test_equal_logits_of_many_beams(V):
    """More equal candidates than are ranked by counting, few of a beam and many."""
    x, scores, slots = draw(2, 32, V, "bf16", seed=3)
    x[:] = 0
    check(x, 0 * scores, slots=slots)
    check(x, -0.25 * np.arange(64).reshape(2, 32) % 2, slots=slots)


@pytest.mark.parametrize("V", [33, 3001, 100003])
@pytest.mark.parametrize("B", [2, 16, 31, 64])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_equal_beams_whose_rows_begin_anywhere(V, B, dtype):
    """Rows of odd length, at different places of 16 bytes: their candidates are equal all the same, the lower beam's first."""
    x, scores, slots = draw(1, B, V, dtype, seed=B)
    x[1:] = x[:1]
    if B * V < 200 * 20000:
        check(x, 0 * scores, slots=slots)
        check(x, -0.5 * (np.arange(B)[None] // 3), slots=slots)
    else:                                              # (the plain form would take long)
        best, parents, tokens = kda.beam_select(x, torch().zeros(1, B, device="cuda"))[:3]
        assert parents[0].tolist() == list(range(B)) and (tokens == x[0].float().argmax()).all() and (best == best[0, 0]).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V", [7, 9, 16, 17, 24, 25, 8191, 8192, 8193])
def test_rows_at_every_place_of_16_bytes(V, dtype):
    """The same bytes in and out, whatever the place; nothing before or behind a row enters."""
    t = torch()
    x, scores, slots = draw(2, 3, V, dtype, seed=V)
    want = check(x, scores, slots=slots)
    for at in range(16 // x.element_size()):
        for apart in (V + 3, V + 16, -(-V // 8) * 8 + 8):
            wide = t.full((6 * apart + 16,), float("nan"), dtype=x.dtype, device="cuda")
            rows = wide[at:at + 6 * apart].view(6, apart)[:, :V]
            rows.copy_(x)
            got = kda.beam_select(rows, t.tensor(scores, dtype=t.float32, device="cuda"),
                                  slots=t.tensor(slots, dtype=t.int32, device="cuda"))
            assert all(a is b is None or t.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("V", [1 << 24, (1 << 24) - 5])
def test_the_largest_vocabulary_and_beams(V):
    """As many slices and lists as there can be; the plain form a row at a time."""
    t, B = torch(), 64
    g = t.Generator(device="cuda")
    g.manual_seed(5)
    x = t.empty(B, V, device="cuda")
    for b in range(B):
        x[b] = 3 * t.randn(V, generator=g, device="cuda")
    scores = -0.02 * t.arange(B, device="cuda")[None]
    got = kda.beam_select(x, scores)
    every, tokens = [], []
    for b in range(B):
        row = x[b].double()
        top = t.sort(x[b], descending=True, stable=True)
        every.append(scores[0, b].double() + top.values[:B].double() - t.logsumexp(row, 0))
        tokens.append(top.indices[:B])
    best = t.sort(t.cat(every), descending=True, stable=True)
    at = best.indices[:B]
    assert t.equal(got[1][0].long(), at // B) and t.equal(got[2][0].long(), t.cat(tokens)[at])
    assert ((got[0][0].double() - best.values[:B]).abs() <= 2.0 ** -18 + 2.0 ** -24 * best.values[:B].abs()).all()
