"""Failure detection of the paged attention's tiles where a query tile's key tiles are dealt to both pipelines: a bounded wait
for scores that runs out, in both pipelines and in the second alone (the first then waits for one that never ends).

Copies of the library built here have a limit of zero polls for those waits, as in test_paged_timeout.py; the CTAs wind
down, the call returns, the copy's error word holds bit 1, and the next call (the regular library, same process and
context) is right.
"""
import ctypes

import pytest

import kda_linear_attention_chunk_gb300 as kda
from kda_linear_attention_chunk_gb300 import build as kbuild
from paged_lines import workers

OWN, GROUPS, HQ, HK = [(30, 1)] * 12, [(12, 40000)], 32, 8


def test_most_workers_begin_with_a_dealt_item():
    assert sum(items[:1] != [] and items[0][2] for items in workers(OWN, GROUPS, HQ, HK, 152)) >= 140


@pytest.mark.gpu
@pytest.mark.parametrize("tag,limit", [("paged0", "0"), ("paged_second", "(threadIdx.x < 128 ? 1u << 18 : 0u)")])
def test_a_wait_that_runs_out_in_a_dealt_item(tag, limit, monkeypatch):
    from gpu_util import torch
    from paged_util import Batch
    t = torch()
    whole, lib = kda.load(), kda.load(kbuild.build_variant(tag, [f"KDA_WAIT_LIMIT_PAGED={limit}"]))
    word = ctypes.c_int(0)
    assert lib.kda_device_error(ctypes.byref(word), 1) == kda.KDA_OK
    b = Batch(OWN, GROUPS, Hq=HQ, Hk=HK, seed=1)
    monkeypatch.setattr(kda, "_lib", lib)
    b.call()
    t.cuda.synchronize()                                  # the kernels returned
    assert lib.kda_device_error(ctypes.byref(word), 1) == kda.KDA_OK
    assert word.value & kda.ERR_WAIT_TIMEOUT, f"error word {word.value:#x}"
    monkeypatch.setattr(kda, "_lib", whole)
    b.check(b.call())
