"""What the binding's calls around a hybrid stack's softmax layers make of the tensors that they are given: on CPU, with
stand-ins for CUDA tensors and for the library, which records its arguments; and on the GPU."""
import ctypes

import pytest

import kda_linear_attention_chunk_gb300 as kda


class OnGpu:
    """A CPU tensor that says it lies on a GPU."""

    def __init__(self, t, index=0):
        import torch
        self.t, self.index, self.is_cuda, self.device = t, index, True, torch.device("cuda", index)

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


class Library:
    """Takes every call for valid and keeps its arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or kda.KDA_OK


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(kda, "load", lambda: lib)
    monkeypatch.setattr(kda, "_current_device", lambda: 0, raising=False)
    return lib


def int32(values, index=0):
    import torch
    return OnGpu(torch.tensor(values, dtype=torch.int32), index)


def one_slot_views():
    """Contiguous tensors [1][...] whose first stride is not their entry's size."""
    import torch
    return [torch.zeros(1, 100, 10)[:, 50:55], torch.empty(5, 1, 8).transpose(0, 1), torch.zeros(6, 4, 16)[::3][:1],
            torch.zeros(4, 16).as_strided((1, 4, 16), (0, 16, 1))]


def test_entry_sizes_are_those_of_an_entry(library, monkeypatch):
    """A first axis of one may have any stride."""
    import torch
    sizes = []

    def copy(array, n, *rest):
        sizes.append(list((ctypes.c_int64 * (2 * n)).from_address(array))[1::2])
        return kda.KDA_OK

    monkeypatch.setattr(library, "kda_slots_copy", copy, raising=False)
    monkeypatch.setattr(library, "kda_slots_compact", copy, raising=False)
    views = one_slot_views()
    assert all(v.is_contiguous() for v in views)
    pools = [OnGpu(v) for v in views]
    kda.slots_copy(pools, int32([-1]), int32([0]), stream=0)
    kda.slots_compact(pools, int32([0]), int32([0]), stream=0)
    kda.slots_copy([OnGpu(torch.zeros(3, 4, 8, dtype=torch.bfloat16)), OnGpu(torch.zeros(3, 24))], int32([0]), int32([1]),
                   stream=0)
    assert sizes == [[200, 160, 256, 256]] * 2 + [[64, 96]]


def test_pools_without_entries_are_refused(library):
    import torch
    for shape in ((0, 8), (2, 0), (2, 3, 0), (8,), ()):
        for call in (lambda p: kda.slots_copy(p, int32([0]), int32([1]), stream=0),
                     lambda p: kda.slots_compact(p, int32([0]), int32([0]), stream=0)):
            with pytest.raises(ValueError):
                call([OnGpu(torch.zeros(shape))])
    assert library.calls == []


@pytest.mark.gpu
def test_a_single_slot_that_is_a_view_is_cleared_and_nothing_beside_it():
    import torch
    t = torch.ones(3, 100, 12, device="cuda")
    kda.slots_copy([t[1:2, 50:55]], torch.tensor([-1], dtype=torch.int32, device="cuda"),
                   torch.tensor([0], dtype=torch.int32, device="cuda"))
    want = torch.ones(3, 100, 12)
    want[1, 50:55] = 0
    assert torch.equal(t.cpu(), want)
    t = torch.ones(5, 1, 8, device="cuda")
    kda.slots_copy([t.transpose(0, 1)], torch.tensor([-1], dtype=torch.int32, device="cuda"),
                   torch.tensor([0], dtype=torch.int32, device="cuda"))
    assert not t.any()


def everywhere():
    """Every call with its tensors: {name: (call(tensors), tensors)}; each runs on device 0 as it is."""
    import torch
    half = lambda *s: OnGpu(torch.zeros(*s, dtype=torch.bfloat16))   # noqa: E731
    f32 = lambda *s: OnGpu(torch.zeros(*s))   # noqa: E731
    q, k, v, pool, out = half(4, 8, 64), half(4, 2, 64), half(4, 2, 64), half(4, 2, 2, 20, 64), half(4, 8, 64)
    rope = dict(q=q, k=k, q_weight=f32(64), k_weight=f32(64), positions=int32([0] * 4), table=f32(9, 32))
    window = dict(q=q, k=k, v=v, kv_pool=pool, slots=int32([0] * 4), out=out)
    return {
        "rope": (lambda a, b, **kw: kda.head_norm_rope(out=(a, b), stream=0, **kw), dict(rope, a=half(4, 8, 64), b=half(4, 2, 64))),
        "prefill": (lambda **kw: kda.window_prefill(window=16, stream=0, **kw),
                    dict(window, cu_seqlens=int32([0, 1, 2, 3, 4]), starts=int32([0] * 4))),
        "decode": (lambda **kw: kda.window_decode(window=16, stream=0, **kw), dict(window, positions=int32([0] * 4))),
        "copy": (lambda a, b, **kw: kda.slots_copy([a, b], stream=0, **kw),
                 dict(a=pool, b=f32(4, 8), src=int32([0]), dst=int32([1]))),
        "compact": (lambda a, b, **kw: kda.slots_compact([a, b], stream=0, **kw),
                    dict(a=pool, b=f32(4, 8), slots=int32([0]), new_slots=int32([0]))),
    }


@pytest.mark.parametrize("which", ["rope", "prefill", "decode", "copy", "compact"])
def test_tensors_of_two_devices_are_refused(library, which):
    call, tensors = everywhere()[which]
    call(**tensors)
    assert len(library.calls) == 1
    for name, t in tensors.items():
        with pytest.raises(ValueError):
            call(**dict(tensors, **{name: OnGpu(t.t, 1)}))
        with pytest.raises(ValueError):
            call(**dict(tensors, **{name: t.t}))
    assert len(library.calls) == 1


@pytest.mark.parametrize("which", ["rope", "prefill", "decode", "copy", "compact"])
def test_tensors_beside_the_current_device_are_refused(library, which):
    """The library launches on the current device."""
    call, tensors = everywhere()[which]
    with pytest.raises(ValueError, match="current device"):
        call(**{name: OnGpu(t.t, 1) for name, t in tensors.items()})
    assert library.calls == []


@pytest.mark.parametrize("which", ["rope", "prefill", "decode", "copy", "compact"])
def test_a_stream_of_another_device_is_refused(library, which):
    class Stream:
        cuda_stream, device_index = 4096, 1

    call, tensors = everywhere()[which]
    names = {"rope": "kda_head_norm_rope", "prefill": "kda_window_prefill", "decode": "kda_window_decode",
             "copy": "kda_slots_copy", "compact": "kda_slots_compact"}
    fn = {"rope": kda.head_norm_rope, "prefill": kda.window_prefill, "decode": kda.window_decode, "copy": kda.slots_copy,
          "compact": kda.slots_compact}[which]
    kw = dict(tensors)
    if which in ("copy", "compact"):
        kw["pools"] = [kw.pop("a"), kw.pop("b")]
    elif which == "rope":
        kw["out"] = (kw.pop("a"), kw.pop("b"))
    else:
        kw["window"] = 16
    with pytest.raises(ValueError):
        fn(stream=Stream(), **kw)
    Stream.device_index = 0
    fn(stream=Stream(), **kw)
    assert [c[0] for c in library.calls] == [names[which]] and library.calls[0][1][-1] == 4096


@pytest.mark.parametrize("shape", [(0, 2, 2, 20, 64), (4, 2, 2, 0, 64)])
def test_a_ring_cache_without_entries_is_refused(library, shape):
    """Its address is null, which would mean that nothing is cached."""
    import torch
    for which in ("prefill", "decode"):
        call, tensors = everywhere()[which]
        tensors = {k: t for k, t in tensors.items() if k not in ("slots", "starts")}
        with pytest.raises(ValueError):
            call(**dict(tensors, kv_pool=OnGpu(torch.zeros(shape, dtype=torch.bfloat16))))
    assert library.calls == []


def test_an_empty_list_of_moves_is_a_call_without_work(library):
    """A step that forks nothing and a batch without live sequences; what is wrong with the tensors is still refused."""
    import torch
    pool, none = OnGpu(torch.zeros(3, 8)), int32([])
    assert kda.slots_copy([pool], none, none, stream=0) is None
    new = int32([])
    assert kda.slots_compact([pool], none, new, stream=0) is new
    assert library.calls == []
    for call in (lambda: kda.slots_copy([pool], none, int32([0]), stream=0), lambda: kda.slots_copy([], none, none, stream=0),
                 lambda: kda.slots_copy([pool], none, int32([], index=1), stream=0),
                 lambda: kda.slots_compact([pool], none, int32([0]), stream=0)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_an_empty_table_compacts_to_an_empty_one():
    import torch
    pool = torch.ones(3, 8, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    kda.slots_copy([pool], none, none)
    got = kda.slots_compact([pool], none)
    assert got.shape == (0,) and got.dtype == torch.int32 and got.is_cuda and bool((pool == 1).all())
