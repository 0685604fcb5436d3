"""Host-side checks of the entry points around paged caches and beams (no GPU needed): every refusal, synchronously and
before any device is touched; and what the binding passes on and refuses, with stand-ins for CUDA tensors and for the
library.  Fake, never-dereferenced addresses are only passed in calls that must fail validation; calls that would pass it
run only on machines without a GPU."""
import ctypes

import pytest

import kda_linear_attention_chunk_gb300 as kda
from test_hybrid_api import cpu_only
from test_hybrid_tensors import OnGpu, int32, library   # noqa: F401  (a fixture)

A = 1 << 24
STEP = 1 << 24


def append(**over):
    N, T, Hq, Hk, d = 2, 16, 8, 2, 128
    args = dict(q=A, q_stride=Hq * d, k=A + STEP, k_stride=Hk * d, v=A + 2 * STEP, v_stride=Hk * d, qw=A + 3 * STEP,
                kw=A + 4 * STEP, table=A + 5 * STEP, max_pos=100, cu=A + 6 * STEP, starts=A + 7 * STEP, slots=A + 8 * STEP,
                pages=A + 9 * STEP, num_pages=10, page=64, page_table=A + 10 * STEP, num_slots=3, max_pages=4,
                q_out=A + 11 * STEP, N=N, T=T, Hq=Hq, Hk=Hk, d=d, rotary=64, layout=0, norm=1, eps=1e-6, dtype=0, stream=0)
    args.update(over)
    return kda.kda_paged_append(*args.values())


def attend(**over):
    N, T, Hq, Hk, d = 2, 16, 8, 2, 128
    args = dict(q=A, q_stride=Hq * d, cu=A + 6 * STEP, starts=A + 7 * STEP, slots=A + 8 * STEP, pages=A + 9 * STEP,
                num_pages=10, page=64, page_table=A + 10 * STEP, num_slots=3, max_pages=4, groups=A + 12 * STEP,
                lens=A + 13 * STEP, kept=A + 14 * STEP, P=1, out=A + 11 * STEP, work=A + 100 * STEP, work_bytes=1 << 30,
                N=N, T=T, Hq=Hq, Hk=Hk, d=d, scale=0.1, dtype=0, stream=0)
    args.update(over)
    return kda.kda_paged_attention(*args.values())


def expect(call, status, cases):
    for bad in cases:
        assert call(**bad) == status, bad


def test_append_refusals(kda_lib):
    expect(append, kda.KDA_ERR_NULL, [{n: 0} for n in ("q", "k", "v", "table", "pages", "page_table", "q_out")])
    expect(append, kda.KDA_ERR_SHAPE, [
        dict(N=0), dict(T=-1), dict(Hq=0), dict(Hk=0), dict(d=0), dict(rotary=-16), dict(rotary=144), dict(max_pos=0),
        dict(layout=2), dict(norm=2), dict(eps=-1.0), dict(eps=float("nan")), dict(q_stride=1016), dict(v_stride=0),
        dict(k_stride=1 << 31), dict(num_pages=0), dict(page=0), dict(num_slots=0), dict(max_pages=0),
        dict(max_pages=1 << 25), dict(slots=0, num_slots=1), dict(cu=0), dict(num_pages=0x7fffffff),
        dict(num_slots=0x7fffffff, max_pages=1 << 20, page=16)])
    expect(append, kda.KDA_ERR_UNSUPPORTED, [dict(d=96), dict(d=256), dict(dtype=2), dict(rotary=24), dict(page=8),
                                             dict(page=48), dict(page=512)])
    expect(append, kda.KDA_ERR_ALIGN, [dict(q=A + 8), dict(q_out=A + 11 * STEP + 2), dict(table=A + 5 * STEP + 4),
                                       dict(q_stride=1028), dict(pages=A + 9 * STEP + 8), dict(starts=A + 7 * STEP + 2),
                                       dict(page_table=A + 10 * STEP + 1), dict(kw=A + 4 * STEP + 4)])
    expect(append, kda.KDA_ERR_ALIAS, [dict(q_out=A + 16), dict(q_out=A, q_stride=2048), dict(q_out=A + STEP),
                                       dict(pages=A), dict(pages=A + 2 * STEP), dict(q_out=A + 9 * STEP + 256),
                                       dict(page_table=A + 9 * STEP + 4), dict(slots=A + 11 * STEP), dict(pages=A + 5 * STEP)])


def test_attention_refusals(kda_lib):
    expect(attend, kda.KDA_ERR_NULL, [{n: 0} for n in ("q", "out", "pages", "page_table", "groups", "lens", "kept")] +
           [dict(P=0), dict(P=0, groups=0, lens=0)])
    expect(attend, kda.KDA_ERR_SHAPE, [
        dict(N=0), dict(T=-1), dict(P=-1, groups=0, lens=0, kept=0), dict(Hq=0), dict(Hk=3), dict(Hk=0), dict(scale=0.0),
        dict(scale=float("inf")), dict(scale=float("nan")), dict(scale=2e37), dict(q_stride=8), dict(num_pages=0),
        dict(max_pages=0), dict(max_pages=1 << 25), dict(slots=0, num_slots=1), dict(cu=0), dict(num_pages=0x7fffffff)])
    expect(attend, kda.KDA_ERR_UNSUPPORTED, [dict(d=96), dict(dtype=2), dict(Hq=258, q_stride=258 * 128), dict(page=24),
                                             dict(page=1024)])
    expect(attend, kda.KDA_ERR_ALIGN, [dict(q=A + 8), dict(out=A + 11 * STEP + 4), dict(q_stride=1028), dict(cu=A + 2),
                                       dict(groups=A + 12 * STEP + 2), dict(pages=A + 9 * STEP + 2)])
    expect(attend, kda.KDA_ERR_ALIAS, [dict(out=A), dict(out=A + 9 * STEP), dict(out=A + 10 * STEP), dict(kept=A + 11 * STEP),
                                       dict(cu=A + 11 * STEP + 64)])


def test_attention_workspace(kda_lib):
    f = kda.kda_paged_attention_workspace
    for bad in ((0, 1, 0, 8, 2, 128), (1, -1, 0, 8, 2, 128), (1, 1, -1, 8, 2, 128), (1, 1, 0, 8, 3, 128), (1, 1, 0, 8, 2, 96),
                (1, 1, 0, 258, 2, 128), (1, 1, 0, 0, 0, 128)):
        assert f(*bad) == -1, bad
    need = f(2, 16, 1, 8, 2, 128)
    assert need >= 0
    if need:
        assert attend(work_bytes=need - 1) == kda.KDA_ERR_SHAPE and attend(work=0) == kda.KDA_ERR_NULL
        assert attend(work=A + 100 * STEP + 8) == kda.KDA_ERR_ALIGN
        assert attend(work=A + 9 * STEP) == kda.KDA_ERR_ALIAS and attend(work=A + 11 * STEP - need + 16) == kda.KDA_ERR_ALIAS


@cpu_only
def test_valid_calls(kda_lib):
    for good in (dict(), dict(q_out=A), dict(qw=0, kw=0, starts=0), dict(rotary=0, table=0), dict(slots=0),
                 dict(cu=0, N=16, slots=0, num_slots=16), dict(T=0, q=0, k=0, v=0, q_out=0, table=0), dict(page=16),
                 dict(page=256), dict(d=64, dtype=1, layout=1)):
        assert append(**good) == kda.KDA_ERR_DEVICE, good
    for good in (dict(), dict(P=0, groups=0, lens=0, kept=0), dict(starts=0), dict(slots=0), dict(T=0, q=0, out=0),
                 dict(Hq=256, q_stride=256 * 128), dict(cu=0, N=16, num_slots=16), dict(d=64, dtype=1)):
        assert attend(**good) == kda.KDA_ERR_DEVICE, good


def copy(caches=((A, 2 * 2 * 64 * 256), (A + STEP, 2 * 8 * 64 * 256)), n=None, **over):
    arr = (ctypes.c_int64 * (2 * len(caches)))(*[x for c in caches for x in c])
    args = dict(caches=ctypes.addressof(arr), n=len(caches) if n is None else n, num_pages=10, page=64, row_bytes=256,
                page_table=A + 20 * STEP, num_slots=4, max_pages=5, src=A + 21 * STEP, dst=A + 22 * STEP,
                start=A + 23 * STEP, end=A + 24 * STEP, M=4, stream=0)
    args.update(over)
    return kda.kda_pages_copy(*args.values())


def test_copy_refusals(kda_lib):
    expect(copy, kda.KDA_ERR_NULL, [{n: 0} for n in ("page_table", "src", "dst", "end")] + [dict(caches=((0, 65536),))])
    assert kda.kda_pages_copy(0, 1, 1, 64, 256, A, 1, 1, A, A, 0, A, 1, 0) == kda.KDA_ERR_NULL
    expect(copy, kda.KDA_ERR_SHAPE, [dict(M=0), dict(n=0), dict(num_pages=0), dict(page=0), dict(num_slots=0),
                                     dict(max_pages=0), dict(row_bytes=0), dict(max_pages=1 << 25), dict(caches=((A, 0),)),
                                     dict(caches=((A, 64 * 256 + 256),)), dict(caches=((A, 1 << 40),))])
    expect(copy, kda.KDA_ERR_UNSUPPORTED, [dict(page=40), dict(page=8), dict(row_bytes=1040),
                                           dict(caches=tuple((A + 65536 * i, 16384) for i in range(129)), num_pages=1)])
    expect(copy, kda.KDA_ERR_ALIGN, [dict(row_bytes=200), dict(caches=((A + 8, 65536),)), dict(src=A + 21 * STEP + 2),
                                     dict(start=A + 23 * STEP + 1), dict(end=A + 24 * STEP + 3)])
    expect(copy, kda.KDA_ERR_ALIAS, [dict(caches=((A, 65536), (A + 9 * 65536, 65536))), dict(src=A + 64),
                                     dict(page_table=A + STEP), dict(end=A + STEP + 64), dict(start=A)])


@cpu_only
def test_copy_valid_calls(kda_lib):
    for good in (dict(), dict(start=0), dict(row_bytes=1024, caches=((A, 65536),)), dict(row_bytes=16, caches=((A, 1024),))):
        assert copy(**good) == kda.KDA_ERR_DEVICE, good


def beam(**over):
    G, B, V = 3, 4, 1000
    args = dict(logits=A, row_stride=V, dtype=2, scores=A + STEP, ended=A + 2 * STEP, end=5, slots=A + 3 * STEP,
                scores_out=A + 4 * STEP, parents=A + 5 * STEP, tokens=A + 6 * STEP, ended_out=A + 7 * STEP,
                new=A + 8 * STEP, src=A + 9 * STEP, dst=A + 10 * STEP, work=A + 11 * STEP, work_bytes=1 << 23, G=G, B=B, V=V,
                stream=0)
    args.update(over)
    return kda.kda_beam_select(*args.values())


def test_beam_refusals(kda_lib):
    expect(beam, kda.KDA_ERR_NULL, [{n: 0} for n in ("logits", "scores", "scores_out", "parents", "tokens", "ended_out", "new",
                                                     "src", "dst", "work")] + [dict(slots=0), dict(slots=0, new=0)])
    expect(beam, kda.KDA_ERR_SHAPE, [dict(G=0), dict(B=0), dict(V=0), dict(end=-1), dict(end=1000), dict(end=-2, ended=0, ended_out=0),
                                     dict(row_stride=999), dict(row_stride=1 << 40), dict(G=1 << 19), dict(work_bytes=10),
                                     dict(ended=0, end=-1)])
    expect(beam, kda.KDA_ERR_UNSUPPORTED, [dict(B=65), dict(dtype=3), dict(dtype=-1), dict(V=(1 << 24) + 1, row_stride=1 << 25)])
    expect(beam, kda.KDA_ERR_ALIGN, [dict(logits=A + 2), dict(dtype=0, logits=A + 1), dict(scores=A + STEP + 2),
                                     dict(work=A + 11 * STEP + 8), dict(dst=A + 10 * STEP + 1), dict(slots=A + 3 * STEP + 2)])
    expect(beam, kda.KDA_ERR_ALIAS, [dict(scores_out=A + STEP), dict(parents=A + 5 * STEP + 4, tokens=A + 5 * STEP),
                                     dict(new=A + 3 * STEP), dict(work=A), dict(src=A + 11 * STEP), dict(tokens=A + 400)])
    f = kda.kda_beam_select_workspace
    for bad in ((0, 1, 1), (1, 0, 1), (1, 65, 1), (1, 1, 0), (1, 1, (1 << 24) + 1), (1 << 20, 2, 5)):
        assert f(*bad) == -1, bad
    assert f(3, 4, 1000) > 0 and beam(work_bytes=f(3, 4, 1000) - 1) == kda.KDA_ERR_SHAPE


@cpu_only
def test_beam_valid_calls(kda_lib):
    for good in (dict(), dict(ended=0), dict(ended=0, ended_out=0, end=-1), dict(slots=0, new=0, src=0, dst=0),
                 dict(dtype=0, logits=A + 2), dict(work_bytes=kda.kda_beam_select_workspace(3, 4, 1000)), dict(row_stride=1001)):
        assert beam(**good) == kda.KDA_ERR_DEVICE, good


def everywhere():
    """Every wrapper with its tensors on device 0: {name: (call(**tensors), tensors, C entry)}."""
    import torch
    half = lambda *s: OnGpu(torch.zeros(*s, dtype=torch.bfloat16))   # noqa: E731
    f32 = lambda *s: OnGpu(torch.zeros(*s))   # noqa: E731
    four, table = int32([0] * 4), int32([[0, 1]] * 4)
    cache = dict(kv_pages=half(3, 2, 2, 16, 64), page_table=table, starts=four, cu_seqlens=int32([0, 1, 2, 3, 4]), slots=four)
    return {
        "append": (lambda a, **kw: kda.paged_append(out=a, **kw),
                   dict(cache, q=half(4, 8, 64), k=half(4, 2, 64), v=half(4, 2, 64), q_weight=f32(64), k_weight=f32(64),
                        table=f32(9, 32), a=half(4, 8, 64)), "kda_paged_append"),
        "copy": (lambda a, b, **kw: kda.pages_copy([a, b], **kw),
                 dict(a=half(3, 2, 2, 16, 64), b=half(3, 2, 5, 16, 64), page_table=table, src=four, dst=four, end=four, start=four),
                 "kda_pages_copy"),
    }


@pytest.mark.parametrize("which", ["append", "copy"])
def test_devices_and_streams(library, which):   # noqa: F811
    class Stream:
        cuda_stream, device_index = 4096, 1

    call, tensors, entry = everywhere()[which]
    call(stream=0, **tensors)
    assert [c[0] for c in library.calls] == [entry]
    for name, x in tensors.items():
        for other in (OnGpu(x.t, 1), x.t):
            with pytest.raises(ValueError):
                call(stream=0, **dict(tensors, **{name: other}))
    with pytest.raises(ValueError, match="current device"):
        call(stream=0, **{name: OnGpu(x.t, 1) for name, x in tensors.items()})
    with pytest.raises(ValueError):
        call(stream=Stream(), **tensors)
    Stream.device_index = 0
    call(stream=Stream(), **tensors)
    assert len(library.calls) == 2 and library.calls[1][1][-1] == 4096


def test_wrappers_refuse_wrong_tensors(library):   # noqa: F811
    import torch
    bf, f16, f32 = torch.bfloat16, torch.float16, torch.float32
    z = lambda *s, dtype=bf: OnGpu(torch.zeros(*s, dtype=dtype))   # noqa: E731
    q, k, pages, table = z(4, 8, 64), z(4, 2, 64), z(3, 2, 2, 16, 64), int32([[0, 1]] * 4)
    good = dict(q=q, k=k, v=k, kv_pages=pages, page_table=table, stream=0, out=q)
    for bad in (dict(q=z(4, 8, 64, dtype=f32)), dict(k=z(4, 2, 64, dtype=f16)), dict(v=z(4, 3, 64)), dict(k=z(5, 2, 64)),
                dict(kv_pages=z(3, 2, 4, 16, 64)), dict(kv_pages=z(3, 1, 2, 16, 64)), dict(kv_pages=z(3, 2, 2, 16, 128)),
                dict(kv_pages=z(0, 2, 2, 16, 64)), dict(kv_pages=z(3, 2, 2, 16, 64, dtype=f16)), dict(page_table=int32([0, 1])),
                dict(page_table=z(4, 2)), dict(page_table=z(4, 0, dtype=torch.int32)), dict(starts=int32([0] * 3)),
                dict(slots=int32([0] * 5)), dict(cu_seqlens=z(4)), dict(layout="other"), dict(table=z(64, dtype=f32)),
                dict(q_weight=z(64)), dict(out=z(4, 7, 64))):
        with pytest.raises(ValueError):
            kda.paged_append(**dict(good, **bad))
    good = dict(q=q, kv_pages=pages, page_table=table, stream=0, out=q)
    for bad in (dict(q=z(4, 8, 64, dtype=f32)), dict(kv_pages=z(3, 2, 2, 16, 128)), dict(kv_pages=z(3, 3, 2, 16, 64)),
                dict(page_table=z(4, 2)), dict(starts=int32([0] * 3)), dict(out=z(4, 7, 64)),
                dict(prefixes=(int32([0, 4]), int32([5, 5]), int32([1]))), dict(prefixes=(int32([0]), int32([5]), int32([1])))):
        with pytest.raises(ValueError):
            kda.paged_attention(**dict(good, **bad))
    four = int32([0] * 4)
    good = dict(caches=[pages], page_table=table, src=four, dst=four, end=four, stream=0)
    for bad in (dict(caches=[]), dict(caches=[pages, z(3, 2, 2, 16, 128)]), dict(caches=[pages, z(4, 2, 2, 16, 64)]),
                dict(caches=[z(3, 2, 2, 16)]), dict(caches=[z(3, 1, 2, 16, 64)]), dict(dst=int32([0])), dict(end=int32([0])),
                dict(start=int32([0])), dict(page_table=int32([0])),
                dict(caches=[pages, z(3, 2, 2, 16, 64, dtype=f32)])):
        with pytest.raises(ValueError):
            kda.pages_copy(**dict(good, **bad))
    x, s = z(8, 50, dtype=f32), z(2, 4, dtype=f32)
    good = dict(logits=x, scores=s, stream=0)
    for bad in (dict(logits=z(7, 50)), dict(logits=z(8, 50, dtype=torch.float64)), dict(logits=z(2, 4, 50)), dict(scores=z(8, dtype=f32)),
                dict(scores=z(2, 4)), dict(ended=z(2, 4)), dict(ended=int32([0] * 8)), dict(slots=int32([0] * 8)),
                dict(logits=OnGpu(torch.zeros(50, 8).T)), dict(logits=x.t)):
        with pytest.raises(ValueError):
            kda.beam_select(**dict(good, **bad))
    assert library.calls == []


def test_empty_calls(library):   # noqa: F811
    import torch
    pages, table, none = OnGpu(torch.zeros(3, 2, 2, 16, 64, dtype=torch.bfloat16)), int32([[0, 1]] * 4), int32([])
    kda.pages_copy([pages], table, none, none, none, stream=0)
    q, k = (OnGpu(torch.zeros(0, h, 64, dtype=torch.bfloat16)) for h in (8, 2))
    assert kda.paged_append(q, k, k, pages, table, out=q, stream=0) is q
    assert kda.paged_attention(q, pages, table, out=q, stream=0) is q
    assert library.calls == []
