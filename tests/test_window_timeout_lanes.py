"""A bounded wait of the tiled window prefill that runs out for some lanes of a warp only.

Lanes poll one by one, so at a limit, or beside another role that gives up, a barrier may complete between the last
poll of one lane and that of the next. The copy of the library built here gives every second softmax thread a limit of
zero polls for its scores and the others the usual one: the whole warp must give up, and the CTA wind down, as if all of
them had (bit 1 of the error word, the call returns, and the next one is right).
"""
import ctypes

import pytest

import kda_linear_attention_chunk_gb300 as kda
from kda_linear_attention_chunk_gb300 import build as kbuild

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [[300, 260, 130], [1000]])
def test_a_wait_that_runs_out_for_every_second_lane(lens):
    from gpu_util import torch
    from test_window import Batch
    t = torch()
    lib = kda.load(kbuild.build_variant("scores_lanes", ["KDA_WAIT_LIMIT_SCORES=((threadIdx.x & 1) ? 0u : (1u << 18))"]))
    b = Batch([0, 90, 7][:len(lens)], 8, 2, 128, window=150, sinks=3, dtype="bf16", seed=22)
    T, N = sum(lens), len(lens)
    q, k, v = b.new_rows(T)
    cu = b.int32([sum(lens[:i]) for i in range(N + 1)])
    out, pool = t.empty((T, 8, 128), dtype=q.dtype, device="cuda"), b.pool.clone()
    starts, slots = b.int32(b.length), b.ids()
    word = ctypes.c_int(0)
    assert lib.kda_device_error(ctypes.byref(word), 1) == kda.KDA_OK
    st = lib.kda_window_prefill(q.data_ptr(), q.stride(0), k.data_ptr(), k.stride(0), v.data_ptr(), v.stride(0),
                                cu.data_ptr(), starts.data_ptr(), slots.data_ptr(), pool.data_ptr(), pool.shape[0],
                                pool.shape[3], out.data_ptr(), N, T, 8, 2, 128, 150, 3, 0.1, kda.KDA_BF16,
                                int(t.cuda.current_stream().cuda_stream))
    assert st == kda.KDA_OK
    t.cuda.synchronize()
    assert lib.kda_device_error(ctypes.byref(word), 1) == kda.KDA_OK
    assert word.value & kda.ERR_WAIT_TIMEOUT, f"error word {word.value:#x}"
    b.prefill(lens, check_rows=[0, 1, 63, 64, 129, 299], qkv=(q, k, v))
