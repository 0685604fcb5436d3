"""Window attention where scale times score is far beyond what 32 bits resolve to a unit: the largest score still has
the weight 2^0, and the others what their distance from it gives.

The inputs are whole numbers small enough that every score is an exact 32-bit sum, so the distances are exact on both
sides and the bounds need no term for the scores.  With n visible keys, A = sum_j p_j |v_j| and u the half ulp of the
type, an output is off by at most
  * u |ref| and half the smallest subnormal for its own rounding,
  * u A for the probabilities' (fp16: 2^-25 sum_j |v_j| more for those below 2^-14),
  * n 2^-23 A for the sums, and 2^-18 A for the exponentials: 2 ulp each of numerator and denominator, and an argument of
    at most 2^5 that counts, off by 2^-24 of itself for the scale's rounding, its own and the distance's.
"""
import numpy as np
import pytest

import kda_linear_attention_chunk_gb300 as kda
from gpu_util import torch
from hybrid_util import BITS, f64, torch_dtype, visible, worst

pytestmark = pytest.mark.gpu

HQ, HK, WINDOW, SINKS = 4, 2, 70, 3


def rows(T, d, dtype, kind, seed):
    """Queries, keys and values of T rows, and the largest distance of two scores that share weight."""
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(seed)
    ints = lambda lo, hi, h: t.randint(lo, hi, (T, h, d), generator=g, device="cuda").float()   # noqa: E731
    v = t.randn(T, HK, d, generator=g, device="cuda")
    if kind == "small":            # entries to 3: scores to 9 d
        q, k = ints(-3, 4, HQ), ints(-3, 4, HK)
    elif kind == "wide":           # entries to 2^15, multiples of 2^11: scores are multiples of 2^22
        q, k = ints(-16, 17, HQ) * 2048, ints(-16, 17, HK) * 2048
    else:                          # scores base + j: j < 12, or ("rise") 9 now and then, else 0
        base = {"2^20": 1024, "2^21": 2048, "2^22": 4096, "rise": 4096}[kind]
        q, k = t.zeros(T, HQ, d, device="cuda"), t.zeros(T, HK, d, device="cuda")
        q[..., 0], q[..., 1] = 1024, 1
        k[..., 0] = base
        k[..., 1] = t.randint(0, 12, (T, HK), generator=g, device="cuda").float()
        if kind == "rise":
            k[..., 1] = 9 * (t.rand(T, HK, generator=g, device="cuda") < 1 / 60)
    return [x.to(torch_dtype(dtype)) for x in (q, k, v)]


def reference(q, k, v, pos, scale, dtype):
    u, tiny = BITS[dtype]
    out, bound = np.zeros((len(pos),) + q.shape[1:]), np.zeros((len(pos),) + q.shape[1:])
    for r, p in enumerate(pos):
        js = visible(p, WINDOW, SINKS)
        for h in range(HQ):
            K, V = k[js, h // (HQ // HK)], v[js, h // (HQ // HK)]
            s = K @ q[p, h]
            e = np.exp(scale * (s - s.max()))
            w = e / e.sum()
            out[r, h] = w @ V
            A = w @ np.abs(V)
            bound[r, h] = u * np.abs(out[r, h]) + tiny + (1 + u) * (u + len(js) * 2.0 ** -23 + 2.0 ** -18) * A
            if dtype == "fp16":
                bound[r, h] += 2.0 ** -25 * np.abs(V).sum(0)
    return out, bound


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind,scale", [("small", 1.0), ("small", 1e6), ("small", 1e9), ("small", 1e37), ("wide", None),
                                        ("wide", 1e9), ("2^20", 0.5), ("2^21", 1.0), ("2^22", 1.0), ("2^22", 0.7),
                                        ("2^21", 60.0), ("2^22", 100.0), ("2^22", 700.0),
                                        ("rise", 0.7)])
def test_the_largest_score_keeps_its_weight(kind, scale, d, dtype):
    """All rows at once (tiles), a few at a time behind a cache (warp MMA), one at a time (decode)."""
    t = torch()
    T, scale = 400, d ** -0.5 if scale is None else scale
    q, k, v = rows(T, d, dtype, kind, seed=d)
    real = float(np.float32(scale))
    ref, bound = reference(f64(q), f64(k), f64(v), range(T), real, dtype)
    i32 = lambda x: t.tensor(x, dtype=t.int32, device="cuda")   # noqa: E731
    whole = kda.window_prefill(q, k, v, i32([0, T]), WINDOW, sinks=SINKS, scale=scale)
    assert worst(f64(whole), ref, bound) <= 1.0
    pool = t.full((1, 2, HK, WINDOW + SINKS, d), float("nan"), dtype=q.dtype, device="cuda")
    steps, a = [], 0
    while a < T:
        n = 200 if a == 0 else min(8, T - a)           # the first rows fill the ring
        steps.append(kda.window_prefill(q[a:a + n], k[a:a + n], v[a:a + n], i32([0, n]), WINDOW, sinks=SINKS, kv_pool=pool,
                                        starts=i32([a]), scale=scale))
        a += n
    assert worst(f64(t.cat(steps)), ref, bound) <= 1.0
    pool.fill_(float("nan"))
    single = t.cat([kda.window_decode(q[a:a + 1], k[a:a + 1], v[a:a + 1], i32([a]), pool, WINDOW, sinks=SINKS, scale=scale)
                    for a in range(T)])
    assert worst(f64(single), ref, bound) <= 1.0
