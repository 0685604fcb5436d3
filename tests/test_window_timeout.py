"""Failure detection of the tiled window prefill on the GPU: a bounded wait that
runs out.

The copy of the library built here has a limit of zero polls for the softmax's
wait for scores, so it gives up at once although its MMAs complete; that takes
every CTA through the wind-down (bit 1 of the error word, the other roles
stopped, every copy and MMA in flight landed, TMEM freed).  The call must
return, the copy's error word must hold bit 1, and a normal call afterwards
(the regular library, same process and context) must still be right.
"""
import ctypes

import pytest

import kda_linear_attention_chunk_gb300 as kda
from kda_linear_attention_chunk_gb300 import build as kbuild

pytestmark = pytest.mark.gpu


def test_wait_timeout_sets_bit_and_leaves_the_gpu_usable():
    from gpu_util import torch
    from test_window import Batch
    t = torch()
    lib = kda.load(kbuild.build_variant("scores0", ["KDA_WAIT_LIMIT_SCORES=0"]))
    b = Batch([0, 90, 7], 8, 2, 128, window=150, sinks=3, dtype="bf16", seed=21)
    lens = [300, 260, 130]
    q, k, v = b.new_rows(sum(lens))
    cu = b.int32([0, 300, 560, 690])
    out, pool = t.empty((690, 8, 128), dtype=q.dtype, device="cuda"), b.pool.clone()
    starts, slots = b.int32(b.length), b.ids()
    word = ctypes.c_int(0)
    assert lib.kda_device_error(ctypes.byref(word), 1) == kda.KDA_OK
    st = lib.kda_window_prefill(q.data_ptr(), q.stride(0), k.data_ptr(), k.stride(0), v.data_ptr(), v.stride(0),
                                cu.data_ptr(), starts.data_ptr(), slots.data_ptr(), pool.data_ptr(), pool.shape[0],
                                pool.shape[3], out.data_ptr(), 3, 690, 8, 2, 128, 150, 3, 0.1, kda.KDA_BF16,
                                int(t.cuda.current_stream().cuda_stream))
    assert st == kda.KDA_OK
    t.cuda.synchronize()                                  # the kernels returned
    assert lib.kda_device_error(ctypes.byref(word), 1) == kda.KDA_OK
    assert word.value & kda.ERR_WAIT_TIMEOUT, f"error word {word.value:#x}"
    # the context is intact: the regular library still computes the right thing
    b.prefill(lens, check_rows=[0, 1, 63, 64, 129, 299], qkv=(q, k, v))
