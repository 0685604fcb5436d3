"""Beam selection: parents, tokens and slots equal to a plain 64-bit form's, scores within the bound of their sums.

Bound of a score: the kernel's exponentials are off by at most 2^-22 relative (2 ulp of exp2 and the rounding of its argument
x log2 e, whose error of 2^-24 |x| exp(x) stays below 2^-24), each part's fp32 sum by 2^-24 for each addition on a term's
way, at most 8 + 17 in a thread of 128 logits and 5 + 8 over the CTA, the factors on the way (where a maximum moves) likewise:
together below 2^-18 of a sum of one sign, which is the error of its logarithm; and half a last place of the result."""
import math
import random

import numpy as np
import pytest

import kda_linear_attention_chunk_gb300 as kda
from gpu_util import torch

pytestmark = pytest.mark.gpu


def plain(logits, scores, ended=None, end=-1, slots=None):
    """logits [G][B][V], scores [G][B] fp64."""
    G, B, V = logits.shape
    out = {k: np.full((G, B), -1) for k in ("parent", "token", "ended", "new", "src", "dst")}
    best = np.full((G, B), -math.inf)
    out["ended"][:] = 0
    for g in range(G):
        every = np.full((B, V), -math.inf)
        for b in range(B):
            if not scores[g, b] > -math.inf:
                continue
            if ended is not None and ended[g, b]:
                every[b, end] = scores[g, b]
                continue
            x = logits[g, b]
            with np.errstate(all="ignore"):
                m = x.max()
                z = scores[g, b] + (x - (m + np.log(np.exp(x - m).sum())))
            every[b] = np.where(z > -math.inf, z, -math.inf)
        flat = every.ravel()
        beam = np.repeat(np.arange(B), V)              # logits that are equal beside their normaliser are told apart
        order = np.lexsort((np.arange(B * V), -np.nan_to_num(logits[g].ravel(), nan=-math.inf), beam, -flat))[:B]
        for k, e in enumerate(order):
            if flat[e] > -math.inf:
                best[g, k], out["parent"][g, k], out["token"][g, k] = flat[e], e // V, e % V
                out["ended"][g, k] = int((ended is not None and ended[g, e // V]) or e % V == end)
        if slots is not None:
            parents = [int(p) for p in out["parent"][g]]
            free, seen = [b for b in range(B) if b not in parents], set()
            for k, p in enumerate(parents):
                if p >= 0:
                    out["src"][g, k] = slots[g, p]
                if p >= 0 and p not in seen:
                    seen.add(p)
                    out["new"][g, k] = slots[g, p]
                else:
                    out["new"][g, k] = slots[g, free.pop(0)]
                    if p >= 0:
                        out["dst"][g, k] = out["new"][g, k]
    return best, out


def check(logits, scores, ended=None, end=-1, slots=None, **kw):
    """logits: a tensor [G * B][V] on the GPU; the rest numpy."""
    t = torch()
    G, B = scores.shape
    dev = lambda x, dt: None if x is None else t.tensor(x, dtype=dt, device="cuda")   # noqa: E731
    got = kda.beam_select(logits, dev(scores, t.float32), dev(ended, t.int32), end, dev(slots, t.int32), **kw)
    best, want = plain(logits.double().cpu().numpy().reshape(G, B, -1), scores.astype(np.float32).astype(np.float64), ended,
                       end, slots)
    s = got[0].double().cpu().numpy()
    assert np.array_equal(s == -math.inf, best == -math.inf)
    live = best > -math.inf
    assert (np.abs(s[live] - best[live]) <= 2.0 ** -18 + 2.0 ** -24 * np.abs(best[live])).all()
    names = ["parent", "token", "ended", "new", "src", "dst"]
    for name, x in zip(names, got[1:]):
        if x is None:
            assert (name == "ended" and end < 0) or (name in ("new", "src", "dst") and slots is None)
        else:
            assert np.array_equal(x.cpu().numpy(), want[name]), name
    return got


def draw(G, B, V, dtype="fp32", seed=0, scale=3.0):
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(seed)
    dt = {"fp32": t.float32, "bf16": t.bfloat16, "fp16": t.float16}[dtype]
    x = (scale * t.randn(G * B, V, generator=g, device="cuda")).to(dt)
    r = np.random.RandomState(seed)
    scores = -5.0 - np.cumsum(r.rand(G, B) * 1.3, 1)
    slots = r.permutation(G * B + 3)[:G * B].reshape(G, B)
    return x, scores, slots


@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 31, 100, 1023, 8191, 8192, 8193, 8200, 16385, 50001])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_vocabularies(V, dtype):
    """Rows of odd length start at any alignment."""
    x, scores, slots = draw(3, 5, V, dtype, seed=V)
    check(x, scores, slots=slots)


@pytest.mark.parametrize("B", [1, 2, 3, 7, 8, 9, 16, 17, 33, 64])
@pytest.mark.parametrize("dtype,V", [("fp32", 5000), ("bf16", 20011)])
def test_beams(B, dtype, V):
    x, scores, slots = draw(4, B, V, dtype, seed=B)
    check(x, scores, slots=slots)


@pytest.mark.parametrize("G,B,V", [(1, 2, 3000001), (5000, 4, 33), (700, 1, 40), (1, 64, 100000)])
def test_few_long_and_many_short_rows(G, B, V):
    x, scores, slots = draw(G, B, V, "fp16" if V > 100 else "fp32", seed=G)
    check(x, scores, slots=slots)


@pytest.mark.parametrize("dead", [0, 1, 3, 4])
def test_beams_without_a_hypothesis(dead):
    """As in the first step, where only one beam of a prompt is live, and of padded prompts, where none is."""
    x, scores, slots = draw(3, 4, 700, seed=dead)
    scores[:, 4 - dead:] = -math.inf
    scores[1] = -math.inf
    slots[1] = -1
    check(x, scores, slots=slots)
    x[4:8] = math.nan                                  # nothing of them is looked at
    check(x, scores, slots=slots)


def test_fewer_candidates_than_beams():
    x, scores, slots = draw(2, 8, 3, seed=1)
    scores[:, 2:] = -math.inf
    check(x, scores, slots=slots)
    x[0, 1] = x[1, 0] = x[1, 2] = -math.inf            # tokens that are ruled out
    check(x, scores, slots=slots)
    x[:] = -math.inf
    check(x, scores, slots=slots)


@pytest.mark.parametrize("share", [0.0, 0.3, 1.0])
def test_ended_beams(share):
    x, scores, slots = draw(6, 5, 900, seed=3)
    r = np.random.RandomState(7)
    ended = (r.rand(6, 5) < share).astype(np.int32)
    x[:, 17] += 9.0                                    # many end now
    check(x, scores, ended, 17, slots)
    check(x, scores, None, 17, slots)
    x[np.flatnonzero(ended.ravel())] = math.nan
    check(x, scores, ended, 17, slots)


@pytest.mark.parametrize("B", [1, 4, 8, 40])
def test_equal_logits(B):
    """More equal candidates than are ranked by counting: the lowest tokens of the best beam, then of the next."""
    t = torch()
    x = t.zeros(2 * B, 20000, device="cuda")
    scores = np.zeros((2, B))
    got = check(x, scores, slots=np.arange(2 * B).reshape(2, B))
    assert got[2][0].tolist() == list(range(B)) and not got[1].any()
    x[:, 5000:] = -1.0
    x[:, :9] = -2.0
    check(x, scores - np.arange(B))


def test_equal_beams():
    """Two beams with the same logits and scores: the lower one first, token by token."""
    x, scores, slots = draw(1, 6, 3000, seed=5)
    x[3] = x[1]
    scores[0, 3] = scores[0, 1] = 0.0
    check(x, scores, slots=slots)


@pytest.mark.parametrize("where", ["front", "back", "few", "sorted"])
def test_unevenly_spread_logits(where):
    """Finite logits only in a part of the row, all the best in one thread's reach, and in order."""
    t = torch()
    x, scores, slots = draw(2, 8, 30000, seed=6)
    if where == "front":
        x[:, 1500:] = -math.inf
    elif where == "back":
        x[:, :-1700] = -math.inf
    elif where == "few":
        x[:, t.arange(30000, device="cuda") % 4999 != 3] = -math.inf
    else:
        x = x.sort(-1, descending=True).values
    check(x, scores, slots=slots)


@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_rows_without_a_normaliser(value):
    """One NaN or +inf among a beam's logits leaves it no candidate; also where nothing else of a thread's is finite."""
    x, scores, slots = draw(2, 3, 9000, seed=8)
    x[1, 8500] = value
    check(x, scores, slots=slots)
    x[2, :] = -math.inf
    x[2, 4] = value
    check(x, scores, slots=slots)


@pytest.mark.parametrize("size", [1e-30, 1e4, 1e30])
def test_logits_of_all_sizes(size):
    x, scores, slots = draw(2, 4, 4000, scale=size, seed=9)
    check(x, scores, slots=slots)


def test_strided_rows():
    t = torch()
    x, scores, slots = draw(3, 4, 777, "bf16", seed=10)
    wide = t.full((12, 1001), 50.0, dtype=x.dtype, device="cuda")
    wide[:, 3:780] = x
    check(wide[:, 3:780], scores, slots=slots)


def test_a_large_step_moves_what_it_says():
    """The copies that a step asks for bring every beam's bytes to its slot."""
    t = torch()
    x, scores, slots = draw(40, 8, 6000, seed=11)
    got = check(x, scores, slots=slots)
    pool = t.arange(323, device="cuda", dtype=t.float32)[:, None].repeat(1, 4)
    kda.slots_copy([pool], got[5].flatten(), got[6].flatten())
    want = t.tensor(slots, device="cuda").gather(1, got[1].long())
    assert t.equal(pool[got[4].flatten().long(), 0], want.flatten().float())
    assert sorted(got[4].flatten().tolist()) == sorted(slots.ravel().tolist())
    assert kda.device_error(reset=True) == 0


def test_repeated_streams_and_graphs():
    t = torch()
    x, scores, slots = draw(16, 8, 33333, "bf16", seed=12)
    s, ids = t.tensor(scores, dtype=t.float32, device="cuda"), t.tensor(slots, dtype=t.int32, device="cuda")
    call = lambda stream=None: kda.beam_select(x, s, slots=ids, stream=stream)   # noqa: E731
    want = call()
    same = lambda a: all(p is q is None or t.equal(p, q) for p, q in zip(a, want))   # noqa: E731
    assert same(call())
    sides = [t.cuda.Stream() for _ in range(3)]
    t.cuda.synchronize()
    outs = [call(side) for side in sides * 3]
    t.cuda.synchronize()
    assert all(same(o) for o in outs)
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        out = call()
    for o in out:
        if o is not None:
            o.zero_()
    g.replay()
    t.cuda.synchronize()
    assert same(out)


def test_offsets_beyond_2_31_elements():
    t = torch()
    x, scores, slots = draw(2, 2, 500, "bf16", seed=13)
    stride = (1 << 30) + 5
    wide = t.empty(3 * stride + 500, dtype=t.bfloat16, device="cuda").as_strided((4, 500), (stride, 1))
    wide.copy_(x)
    check(wide, scores, slots=slots)


def test_steps_in_a_row():
    """A short search by the operator and by hand over a fixed table of transitions."""
    t = torch()
    r = random.Random(1)
    g = t.Generator(device="cuda")
    g.manual_seed(3)
    V, B, G = 50, 4, 3
    step = t.randn(V, V, generator=g, device="cuda") * 2
    logp = t.log_softmax(step.double(), -1).cpu()
    first = [r.randrange(V) for _ in range(G)]
    scores = t.full((G, B), -math.inf, device="cuda")
    scores[:, 0] = 0
    last = t.tensor(first, device="cuda")[:, None].expand(G, B).clone()
    texts = [[[f]] + [[] for _ in range(B - 1)] for f in first]
    for _ in range(6):
        scores, parents, tokens = kda.beam_select(step[last.flatten()], scores)[:3]
        last = tokens.long().clamp_min(0)
        texts = [[texts[i][parents[i, k]] + [int(tokens[i, k])] for k in range(B)] for i in range(G)]
    for i in range(G):
        hyps = [(0.0, [first[i]])]
        for _ in range(6):
            every = [(s + logp[h[-1], v].item(), h + [v]) for s, h in hyps for v in range(V)]
            hyps = sorted(every, key=lambda e: -e[0])[:B]
        assert [h for _, h in hyps] == texts[i]
        assert np.allclose([s for s, _ in hyps], scores[i].cpu().numpy(), atol=6 * 2.0 ** -18 + 2.0 ** -18)


def test_a_batch_without_prompts():
    t = torch()
    got = kda.beam_select(t.empty(0, 50, device="cuda"), t.empty(0, 4, device="cuda"), end_token=3)
    assert [x if x is None else tuple(x.shape) for x in got] == [(0, 4)] * 4 + [None] * 3
    got = kda.beam_select(t.empty(0, 50, device="cuda"), t.empty(0, 4, device="cuda"),
                          slots=t.empty(0, 4, dtype=t.int32, device="cuda"))
    assert got[0].dtype == t.float32 and got[3] is None and got[4].dtype == t.int32 and got[6].shape == (0, 4)
