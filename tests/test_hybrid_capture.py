"""Captured graphs of the calls around a hybrid stack's softmax layers: what a call needs set up on the device, any one
call before the capture does, also one that another kernel, or another sharing of keys between warps, serves."""
import os
import subprocess
import sys

import pytest

import kda_linear_attention_chunk_gb300 as kda
from gpu_util import torch

pytestmark = pytest.mark.gpu

# (query heads, key heads, rows) of a first call, then of a captured one that another kernel or another sharing of keys
# serves; dtype and d are the same
CAPTURES = {"prefill": [((4, 4, 1), (8, 2, 600)), ((8, 2, 600), (4, 4, 1)), ((8, 2, 2), (16, 2, 1)), ((4, 4, 1), (33, 1, 1))],
            "decode": [((4, 4, 1), (20, 1, 1)), ((4, 4, 1), (64, 1, 1)), ((48, 1, 1), (2, 1, 1))]}


def captured(kind, first, then):
    t = torch()

    def make(Hq, Hk, T):
        t.manual_seed(1)
        q, k, v = (t.randn(T, h, 64, device="cuda").half() for h in (Hq, Hk, Hk))
        pool = t.randn(1, 2, Hk, 40, 64, device="cuda").half()
        start, cu = t.tensor([50], dtype=t.int32, device="cuda"), t.tensor([0, T], dtype=t.int32, device="cuda")
        out = t.empty_like(q)
        if kind == "decode":
            return lambda: kda.window_decode(q, k, v, start, pool, 30, sinks=1, out=out), out
        return lambda: kda.window_prefill(q, k, v, cu, 30, sinks=1, kv_pool=pool, starts=start, out=out), out

    warm, _ = make(*first)
    call, out = make(*then)
    warm()
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        call()
    out.zero_()
    graph.replay()
    t.cuda.synchronize()
    got = out.clone()
    again, want = make(*then)
    again()
    assert t.equal(got, want)


def run_alone(what):
    """In a process of its own, where no call was made before."""
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here)]))
    r = subprocess.run([sys.executable, "-c", "import test_hybrid_capture as s; " + what], env=env, cwd=os.path.dirname(here),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("kind,at", [(k, i) for k in CAPTURES for i in range(len(CAPTURES[k]))])
def test_capture_after_another_call_of_its_kind(kind, at, kda_lib):
    """The only call before the capture is one of the same kind, dtype and d."""
    run_alone(f"s.captured({kind!r}, *s.CAPTURES[{kind!r}][{at}])")


def captured_after_a_move():
    """Each call's first time is inside a capture; the only call before was a copy of slots."""
    t = torch()
    i32 = lambda *x: t.tensor(x, dtype=t.int32, device="cuda")   # noqa: E731
    kda.slots_copy([t.zeros(2, 8, device="cuda")], i32(0), i32(1))
    t.manual_seed(1)
    q, k, v = (t.randn(300, h, 128, device="cuda").bfloat16() for h in (8, 2, 2))
    table, positions, cu, start, slots = kda.rope_table(400, 128), i32(*range(300)), i32(0, 300), i32(300), i32(1)

    def run():
        pool = t.zeros(2, 2, 2, 40, 128, dtype=t.bfloat16, device="cuda")
        a, b = kda.head_norm_rope(q, k, positions=positions, table=table)
        x = kda.window_prefill(a, b, v, cu, 30, sinks=2, kv_pool=pool, slots=slots)
        moved = kda.slots_compact([pool], slots)
        y = kda.window_decode(a[:1], b[:1], v[:1], start, pool, 30, sinks=2, slots=moved)
        return a, b, x, moved, y, pool

    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        got = run()
    graph.replay()
    t.cuda.synchronize()
    for one, other in zip(got, run()):
        assert t.equal(one, other)


def test_capture_after_a_call_of_another_kind(kda_lib):
    run_alone("s.captured_after_a_move()")
