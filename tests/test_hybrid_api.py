"""Host-side checks of the entry points around a hybrid stack's softmax layers
(no GPU needed): every refusal, synchronously and before any device is touched.
Fake, never-dereferenced addresses are only passed in calls that must fail
validation; calls that would pass it run only on machines without a GPU."""
import ctypes

import pytest

import kda_linear_attention_chunk_gb300 as kda

A = 1 << 24
STEP = 1 << 22


def _has_gpu():
    try:
        import torch
        return torch.cuda.is_available()
    except Exception:
        return False


cpu_only = pytest.mark.skipif(_has_gpu(), reason="valid call with fake addresses: CPU-only check")


def rope(**over):
    T, Hq, Hk, d = 16, 8, 2, 128
    args = dict(q=A, q_stride=Hq * d, k=A + STEP, k_stride=Hk * d, qw=A + 2 * STEP, kw=A + 3 * STEP, table=A + 4 * STEP,
                max_pos=100, positions=A + 5 * STEP, q_out=A + 6 * STEP, k_out=A + 7 * STEP, T=T, Hq=Hq, Hk=Hk, d=d,
                rotary=64, layout=0, norm=1, eps=1e-6, dtype=0, stream=0)
    args.update(over)
    return kda.kda_head_norm_rope(*args.values())


def test_rope_refusals(kda_lib):
    for name in ("q", "k", "table", "positions", "q_out", "k_out"):
        assert rope(**{name: 0}) == kda.KDA_ERR_NULL, name
    for bad in (dict(T=-1), dict(Hq=0), dict(Hk=0), dict(d=0), dict(rotary=-16), dict(rotary=144), dict(max_pos=0),
                dict(layout=2), dict(norm=2), dict(eps=-1.0), dict(eps=float("nan")), dict(q_stride=1016),
                dict(k_stride=0), dict(q_stride=-1024), dict(q_stride=1 << 31), dict(T=1 << 30)):
        assert rope(**bad) == kda.KDA_ERR_SHAPE, bad
    for bad in (dict(d=96), dict(d=256), dict(dtype=2), dict(rotary=24)):
        assert rope(**bad) == kda.KDA_ERR_UNSUPPORTED, bad
    for bad in (dict(q=A + 8), dict(k_out=A + 7 * STEP + 2), dict(table=A + 4 * STEP + 4), dict(q_stride=1028),
                dict(positions=A + 5 * STEP + 2)):
        assert rope(**bad) == kda.KDA_ERR_ALIGN, bad
    for bad in (dict(q_out=A + 16), dict(q_out=A, q_stride=2048), dict(k_out=A), dict(q_out=A + 7 * STEP),
                dict(q_out=A + 4 * STEP), dict(k_out=A + 5 * STEP)):
        assert rope(**bad) == kda.KDA_ERR_ALIAS, bad


@cpu_only
def test_rope_valid_calls(kda_lib):
    for good in (dict(), dict(q_out=A, k_out=A + STEP), dict(qw=0, kw=0), dict(rotary=0, table=0, positions=0),
                 dict(T=0, q=0, k=0, table=0, positions=0, q_out=0, k_out=0), dict(q_stride=8192), dict(norm=0, eps=0.0),
                 dict(d=64, dtype=1, layout=1), dict(k=A + 2048, q_stride=1280, k_stride=1280)):
        assert rope(**good) == kda.KDA_ERR_DEVICE, good


def prefill(**over):
    N, T, Hq, Hk, d = 2, 16, 8, 2, 128
    args = dict(q=A, q_stride=Hq * d, k=A + STEP, k_stride=Hk * d, v=A + 2 * STEP, v_stride=Hk * d, cu=A + 3 * STEP,
                starts=A + 4 * STEP, slots=A + 5 * STEP, pool=A + 6 * STEP, num_slots=3, rows=20, out=A + 7 * STEP, N=N,
                T=T, Hq=Hq, Hk=Hk, d=d, window=16, sinks=4, scale=0.1, dtype=0, stream=0)
    args.update(over)
    return kda.kda_window_prefill(*args.values())


def decode(**over):
    N, Hq, Hk, d = 2, 8, 2, 128
    args = dict(q=A, q_stride=Hq * d, k=A + STEP, k_stride=Hk * d, v=A + 2 * STEP, v_stride=Hk * d,
                positions=A + 4 * STEP, slots=A + 5 * STEP, pool=A + 6 * STEP, num_slots=3, rows=20, out=A + 7 * STEP,
                N=N, Hq=Hq, Hk=Hk, d=d, window=16, sinks=4, scale=0.1, dtype=0, stream=0)
    args.update(over)
    return kda.kda_window_decode(*args.values())


@pytest.mark.parametrize("call", [prefill, decode])
def test_window_refusals(kda_lib, call):
    for name in ("q", "k", "v", "out"):
        assert call(**{name: 0}) == kda.KDA_ERR_NULL, name
    for bad in (dict(N=0), dict(Hq=0), dict(Hk=0), dict(Hk=3), dict(Hq=1), dict(window=0), dict(sinks=-1), dict(window=17),
                dict(sinks=5), dict(rows=19), dict(window=0x7fffffff, sinks=0x7fffffff), dict(num_slots=0),
                dict(slots=0, num_slots=1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=2e37),
                dict(scale=float("nan")), dict(q_stride=512), dict(v_stride=8), dict(num_slots=0x7fffffff)):
        assert call(**bad) == kda.KDA_ERR_SHAPE, bad
    for bad in (dict(d=96), dict(d=32), dict(dtype=2), dict(dtype=-1), dict(Hq=129, Hk=1, q_stride=129 * 128)):
        assert call(**bad) == kda.KDA_ERR_UNSUPPORTED, bad
    for bad in (dict(q=A + 8), dict(k_stride=260), dict(pool=A + 6 * STEP + 8), dict(slots=A + 5 * STEP + 1),
                dict(out=A + 7 * STEP + 4)):
        assert call(**bad) == kda.KDA_ERR_ALIGN, bad
    for bad in (dict(out=A + 16), dict(out=A + STEP), dict(pool=A + 2 * STEP), dict(out=A + 6 * STEP + 256),
                dict(slots=A + 6 * STEP + 4), dict(pool=A - 16)):
        assert call(**bad) == kda.KDA_ERR_ALIAS, bad


def test_prefill_refusals_of_its_own(kda_lib):
    assert prefill(cu=0) == kda.KDA_ERR_NULL
    assert prefill(pool=0) == kda.KDA_ERR_NULL                 # starts and slots without a cache
    assert prefill(pool=0, starts=0) == kda.KDA_ERR_NULL
    assert prefill(T=-1) == kda.KDA_ERR_SHAPE
    assert prefill(cu=A + 3 * STEP + 2) == kda.KDA_ERR_ALIGN
    assert decode(positions=0) == kda.KDA_ERR_NULL
    assert decode(pool=0) == kda.KDA_ERR_NULL
    assert decode(positions=A + 4 * STEP + 2) == kda.KDA_ERR_ALIGN


@cpu_only
def test_window_valid_calls(kda_lib):
    for good in (dict(), dict(window=1, sinks=0), dict(d=64, dtype=1), dict(slots=0), dict(Hq=128, Hk=1, q_stride=16384),
                 dict(k=A + 2048, v=A + 2560, q_stride=1536, k_stride=1536, v_stride=1536)):
        assert prefill(**good) == kda.KDA_ERR_DEVICE, good
        assert decode(**good) == kda.KDA_ERR_DEVICE, good
    assert prefill(starts=0) == kda.KDA_ERR_DEVICE
    assert prefill(pool=0, starts=0, slots=0, num_slots=0, rows=0, window=0x7fffffff) == kda.KDA_ERR_DEVICE
    assert prefill(T=0, q=0, k=0, v=0, out=0) == kda.KDA_ERR_DEVICE


def pools(*pairs):
    flat = [x for p in pairs for x in p]
    return (ctypes.c_int64 * len(flat))(*flat)


def copy(ps=((A, 4096), (A + STEP, 64)), num_slots=10, src=A + 2 * STEP, dst=A + 3 * STEP, M=4, fn="kda_slots_copy", n=None):
    arr = pools(*ps)
    return getattr(kda, fn)(ctypes.addressof(arr), len(ps) if n is None else n, num_slots, src, dst, M, 0)


@pytest.mark.parametrize("fn", ["kda_slots_copy", "kda_slots_compact"])
def test_slot_move_refusals(kda_lib, fn):
    assert getattr(kda, fn)(0, 1, 1, A, A + STEP, 1, 0) == kda.KDA_ERR_NULL
    for bad in (dict(src=0), dict(dst=0), dict(ps=((0, 64),))):
        assert copy(fn=fn, **bad) == kda.KDA_ERR_NULL, bad
    for bad in (dict(M=0), dict(num_slots=0), dict(n=0), dict(ps=((A, 0),)), dict(ps=((A, 1 << 40),))):
        assert copy(fn=fn, **bad) == kda.KDA_ERR_SHAPE, bad
    for bad in (dict(num_slots=kda.KDA_MAX_POOL_SLOTS + 1), dict(ps=tuple((A + 64 * i, 16) for i in range(129)))):
        assert copy(fn=fn, **bad) == kda.KDA_ERR_UNSUPPORTED, bad
    for bad in (dict(ps=((A + 8, 64),)), dict(ps=((A, 24),)), dict(src=A + 2 * STEP + 2), dict(dst=A + 3 * STEP + 1)):
        assert copy(fn=fn, **bad) == kda.KDA_ERR_ALIGN, bad
    for bad in (dict(ps=((A, 4096), (A + 9 * 4096, 64))), dict(src=A + 64), dict(dst=A + STEP + 16)):
        assert copy(fn=fn, **bad) == kda.KDA_ERR_ALIAS, bad
    if fn == "kda_slots_compact":
        assert copy(fn=fn, dst=A + 2 * STEP) == kda.KDA_ERR_ALIAS


@cpu_only
@pytest.mark.parametrize("fn", ["kda_slots_copy", "kda_slots_compact"])
def test_slot_move_valid_calls(kda_lib, fn):
    assert copy(fn=fn) == kda.KDA_ERR_DEVICE
    assert copy(fn=fn, ps=((A, 4096), (A + 40960, 64))) == kda.KDA_ERR_DEVICE
    assert copy(fn=fn, num_slots=kda.KDA_MAX_POOL_SLOTS, ps=((A, 16),), src=A + 16 * STEP, dst=A + 17 * STEP) == \
        kda.KDA_ERR_DEVICE


def test_wrappers_refuse_wrong_tensors():
    """The binding's own checks, which come before the library is reached (CPU tensors are refused everywhere)."""
    import torch
    x = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    i = torch.zeros(5, dtype=torch.int32)
    pool = torch.zeros(4, 2, 8, 20, 128, dtype=torch.bfloat16)
    for call in (lambda: kda.head_norm_rope(x, x), lambda: kda.head_norm_rope(x.float(), x.float()),
                 lambda: kda.window_prefill(x, x, x, i, 16), lambda: kda.window_decode(x, x, x, i, pool, 16),
                 lambda: kda.slots_copy([pool], i, i), lambda: kda.slots_compact([pool], i),
                 lambda: kda.slots_copy([], i, i), lambda: kda.slots_compact([], i),
                 lambda: kda.window_prefill(x, x, x, i, 1 << 32), lambda: kda.window_prefill(x, x, x, i, 4, sinks=1 << 31),
                 lambda: kda.window_decode(x, x, x, i, pool, 0),
                 lambda: kda.rope_table(0, 16), lambda: kda.rope_table(8, 15), lambda: kda.rope_table(8, 16, base=0.5),
                 lambda: kda.rope_table(8, 16, stretch=0.5)):
        with pytest.raises(ValueError):
            call()


def test_table_for_a_longer_context():
    """Interpolated by parts: fast pairs keep their frequency, slow ones are stretched, and the size grows."""
    import math

    import numpy as np
    plain = kda.rope_table(64, 64, base=10000.0, device="cpu").double().numpy()
    even = kda.rope_table(64, 64, base=10000.0, stretch=8.0, device="cpu").double().numpy()
    f = 10000.0 ** (-2.0 * np.arange(32) / 64)
    a = np.arange(64)[:, None] * f
    assert np.abs(plain - np.concatenate([np.cos(a), np.sin(a)], 1)).max() <= 2.0 ** -24
    assert np.abs(even - np.concatenate([np.cos(a / 8), np.sin(a / 8)], 1)).max() <= 2.0 ** -24
    parts = kda.rope_table(64, 64, base=10000.0, stretch=8.0, trained=4096, device="cpu").double().numpy()
    size = 1 + 0.1 * math.log(8.0)
    turns = 4096 * f / (2 * math.pi)
    angle = np.arctan2(parts[1, 32:], parts[1, :32])
    assert np.abs(np.hypot(parts[:, :32], parts[:, 32:]) - size).max() <= 2.0 ** -22
    fast, slow = turns >= 33, turns <= 0.9
    assert fast.sum() > 5 and slow.sum() > 5
    # one whole pair index of rounding on either side of the blended stretch
    assert np.allclose(angle[fast][:-1], f[fast][:-1], rtol=1e-6) and np.allclose(angle[slow][1:], f[slow][1:] / 8, rtol=1e-6)
    assert (np.diff(angle / f) <= 1e-6).all()
