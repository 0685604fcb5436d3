"""Captured graphs and streams of the calls around paged caches: each call's first time is inside a capture, after any one
call of the library; and whose stream the outputs' memory belongs to."""
import os
import subprocess
import sys

import pytest

import kda_linear_attention_chunk_gb300 as kda
from gpu_util import torch
from test_hybrid_streams import stream_of

pytestmark = pytest.mark.gpu


def scene(t):
    """A step of two prompts of three beams each, from raw projections to the copies of what the beams own."""
    t.manual_seed(1)
    i32 = lambda *x: t.tensor(x, dtype=t.int32, device="cuda")   # noqa: E731
    G, B, page = 2, 3, 16
    q, k, v = (t.randn(6, h, 128, device="cuda").bfloat16() for h in (8, 2, 2))
    pages = t.randn(100, 2, 2, page, 128, device="cuda").bfloat16()
    table = t.randperm(100, device="cuda")[:80].int().view(8, 10)
    starts, slots = i32(40, 40, 40, 130, 130, 130), i32(5, 1, 2, 3, 0, 4).view(G, B)
    prefixes, own = (i32(0, 3, 6), i32(33, 120), i32(6, 7)), i32(33, 33, 33, 120, 120, 120)
    logits, scores = t.randn(6, 1000, device="cuda"), t.randn(G, B, device="cuda")
    angles = kda.rope_table(200, 128)

    def run(stream=None):
        cache = pages.clone()
        a = kda.paged_append(q, k, v, cache, table, starts, slots=slots.flatten(), table=angles, stream=stream)
        o = kda.paged_attention(a, cache, table, starts, slots=slots.flatten(), prefixes=prefixes, stream=stream)
        step = kda.beam_select(logits, scores, end_token=3, slots=slots, stream=stream)
        kda.pages_copy([cache], table, step[5].flatten(), step[6].flatten(), starts + 1, start=own, stream=stream)
        return (a, o) + step + (cache,)

    return run


def captured():
    t = torch()
    i32 = lambda *x: t.tensor(x, dtype=t.int32, device="cuda")   # noqa: E731
    kda.slots_copy([t.zeros(2, 8, device="cuda")], i32(0), i32(1))
    run = scene(t)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        got = run()
    graph.replay()
    t.cuda.synchronize()
    got = [x.clone() for x in got]
    for one, other in zip(got, run()):
        assert t.equal(one, other)
    assert kda.device_error(reset=True) == 0


def test_first_calls_inside_a_capture(kda_lib):
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here)]))
    r = subprocess.run([sys.executable, "-c", "import test_paged_capture as s; s.captured()"], env=env,
                       cwd=os.path.dirname(here), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("given", ["object", "number", "default"])
def test_outputs_belong_to_the_given_stream(given):
    t = torch()
    i32 = lambda *x: t.tensor(x, dtype=t.int32, device="cuda")   # noqa: E731
    q, k = t.randn(4, 8, 128, device="cuda").bfloat16(), t.randn(4, 2, 128, device="cuda").bfloat16()
    pages, table, starts = t.zeros(9, 2, 2, 16, 128, dtype=t.bfloat16, device="cuda"), i32(*range(8)).view(4, 2), i32(0, 3, 20, 7)
    logits, scores = t.randn(4, 50, device="cuda"), t.zeros(2, 2, device="cuda")
    side = t.cuda.Stream()
    stream = {"object": side, "number": side.cuda_stream, "default": t.cuda.default_stream()}[given]
    handle = 0 if given == "default" else side.cuda_stream
    calls = [lambda: kda.paged_append(q, k, k, pages, table, starts, stream=stream),
             lambda: kda.paged_attention(q, pages, table, starts, stream=stream),
             lambda: kda.beam_select(logits, scores, stream=stream)[0]]
    for call in calls:
        t.cuda.synchronize()
        with t.cuda.stream(t.cuda.Stream()):
            out = call()
        t.cuda.synchronize()
        assert stream_of(t, out) == handle
