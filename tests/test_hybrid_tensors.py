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
