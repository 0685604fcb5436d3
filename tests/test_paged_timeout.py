"""Failure detection of the paged attention's tiles: a bounded wait that runs out.

The copy of the library built here has a limit of zero polls for the softmax's wait for scores, so it gives up at once
although its MMAs complete; that takes every CTA through the wind-down.  The call must return, the copy's error word must
hold bit 1, and a normal call afterwards (the regular library, same process and context) must still be right.
"""
import ctypes

import pytest

import kda_linear_attention_chunk_gb300 as kda
from kda_linear_attention_chunk_gb300 import build as kbuild

pytestmark = pytest.mark.gpu


def test_wait_timeout_sets_bit_and_leaves_the_gpu_usable(monkeypatch):
    from gpu_util import torch
    from paged_util import Batch
    t = torch()
    whole, lib = kda.load(), kda.load(kbuild.build_variant("paged0", ["KDA_WAIT_LIMIT_PAGED=0"]))
    word = ctypes.c_int(0)
    assert lib.kda_device_error(ctypes.byref(word), 1) == kda.KDA_OK
    # spans of two query tiles, and of one, whose key tiles are dealt to both pipelines
    for own, groups in (([(300, 1), (100, 140), (900, 1)], []), ([(30, 1)] * 12, [(12, 600)])):
        b = Batch(own, groups, seed=1)
        monkeypatch.setattr(kda, "_lib", lib)
        b.call()
        t.cuda.synchronize()                              # the kernels returned
        assert lib.kda_device_error(ctypes.byref(word), 1) == kda.KDA_OK
        assert word.value & kda.ERR_WAIT_TIMEOUT, f"error word {word.value:#x}"
        monkeypatch.setattr(kda, "_lib", whole)
        b.check(b.call())
