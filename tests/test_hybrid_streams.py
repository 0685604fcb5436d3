"""The memory of the outputs that the calls around a hybrid stack's softmax layers make on a given stream."""
import pytest

import kda_linear_attention_chunk_gb300 as kda
from gpu_util import torch

pytestmark = pytest.mark.gpu


def calls(t):
    """(name, call(stream)), each with outputs of its own making."""
    g = t.Generator(device="cuda")
    g.manual_seed(0)
    r = lambda *s: t.randn(*s, generator=g, device="cuda").bfloat16()   # noqa: E731
    i32 = lambda x: t.tensor(x, dtype=t.int32, device="cuda")   # noqa: E731
    q, k, v, pool = r(40, 8, 128), r(40, 2, 128), r(40, 2, 128), r(40, 2, 2, 64, 128)
    cu, zero, table, moved = i32(list(range(41))), i32([0] * 40), kda.rope_table(4, 64), i32([3, -1, 39])
    return [("head_norm_rope", lambda s: kda.head_norm_rope(q, k, positions=zero, table=table, stream=s)),
            ("window_prefill", lambda s: kda.window_prefill(q, k, v, cu, 60, sinks=2, kv_pool=pool, starts=zero, stream=s)),
            ("window_decode", lambda s: kda.window_decode(q, k, v, zero, pool, 60, sinks=2, stream=s)),
            ("slots_compact", lambda s: kda.slots_compact([pool], moved, stream=s))]


def stream_of(t, out):
    """The handle of the stream that the memory of a tensor belongs to."""
    for seg in t.cuda.memory_snapshot():
        if seg["address"] <= out.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("memory not found")


@pytest.mark.parametrize("given", ["object", "number", "legacy"])
def test_outputs_on_the_default_stream_beside_another(given):
    """The default stream has the handle 0 (or 1, its name in the runtime): outputs of a call on it belong to it too,
    whichever stream is current."""
    t = torch()
    default = {"object": t.cuda.default_stream(), "number": 0, "legacy": 1}[given]
    todo = calls(t)
    t.cuda.synchronize()
    for name, call in todo:
        with t.cuda.stream(t.cuda.Stream()):
            out = call(default)
        t.cuda.synchronize()
        for o in out if isinstance(out, tuple) else (out,):
            assert stream_of(t, o) == 0, name


@pytest.mark.parametrize("given", ["object", "number"])
def test_outputs_on_a_side_stream(given):
    t = torch()
    side = t.cuda.Stream()
    for name, call in calls(t):
        t.cuda.synchronize()
        out = call(side if given == "object" else side.cuda_stream)
        t.cuda.synchronize()
        for o in out if isinstance(out, tuple) else (out,):
            assert stream_of(t, o) == side.cuda_stream, name
