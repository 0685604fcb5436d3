"""kda_head_norm_rope on the GPU against its formula in 64 bits."""
import numpy as np
import pytest

import kda_linear_attention_chunk_gb300 as kda
from gpu_util import torch
from hybrid_util import beside_pending_work, f64, norm_rope, torch_dtype, worst

pytestmark = pytest.mark.gpu


def draw(T, Hq, Hk, d, dtype, rotary, seed=0, fused=True, max_pos=500):
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(seed)
    qkv = (3 * t.randn(T, Hq + 2 * Hk, d, generator=g, device="cuda")).to(torch_dtype(dtype))
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    qw, kw = (1 + 0.3 * t.randn(2, d, generator=g, device="cuda")).unbind(0)
    pos = t.randint(0, max_pos, (T,), generator=g, device="cuda", dtype=t.int32)
    table = kda.rope_table(max_pos, rotary) if rotary else None
    return q, k, qw.contiguous(), kw.contiguous(), pos, table


def check(got, x, w, table, pos, layout, eps, norm, dtype):
    ref, bound = norm_rope(f64(x), None if w is None else f64(w), None if table is None else f64(table),
                           pos.cpu().numpy(), layout, eps, norm, dtype)
    assert got.is_contiguous() and worst(f64(got), ref, bound) <= 1.0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,Hq,Hk,d,rotary", [(1, 1, 1, 128, 128), (7, 5, 1, 64, 64), (33, 32, 8, 128, 64),
                                             (130, 14, 2, 64, 16), (9, 17, 3, 128, 96), (64, 9, 9, 128, 0)])
def test_matches_the_formula(T, Hq, Hk, d, rotary, layout, dtype):
    q, k, qw, kw, pos, table = draw(T, Hq, Hk, d, dtype, rotary, seed=T)
    a, b = kda.head_norm_rope(q, k, qw, kw, pos if rotary else None, table, layout=layout)
    check(a, q, qw, table, pos, layout, 1e-6, True, dtype)
    check(b, k, kw, table, pos, layout, 1e-6, True, dtype)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_alone_and_norm_without_weights(layout):
    q, k, _, kw, pos, table = draw(21, 6, 2, 128, "bf16", 128, seed=3)
    a, b = kda.head_norm_rope(q, k, positions=pos, table=table, layout=layout, norm=False)
    check(a, q, None, table, pos, layout, 0.0, False, "bf16")
    check(b, k, None, table, pos, layout, 0.0, False, "bf16")
    a, b = kda.head_norm_rope(q, k, k_weight=kw, eps=0.25, layout=layout)
    check(a, q, None, None, pos, layout, 0.25, True, "bf16")
    check(b, k, kw, None, pos, layout, 0.25, True, "bf16")


def test_positions_without_a_table_do_not_turn():
    q, k, qw, kw, pos, _ = draw(6, 4, 2, 64, "fp16", 0, seed=4)
    a, b = kda.head_norm_rope(q, k, qw, kw, positions=pos, table=None)
    check(a, q, qw, None, pos, "half", 1e-6, True, "fp16")
    with pytest.raises(ValueError):
        kda.head_norm_rope(q, k, qw, kw, table=kda.rope_table(500, 16))


def test_in_place_equals_out_of_place():
    t = torch()
    q, k, qw, kw, pos, table = draw(77, 12, 4, 128, "bf16", 128, seed=5, fused=False)
    a, b = kda.head_norm_rope(q, k, qw, kw, pos, table)
    x, y = q.clone(), k.clone()
    kda.head_norm_rope(x, y, qw, kw, pos, table, out=(x, y))
    assert t.equal(a, x) and t.equal(b, y)


def test_zero_heads_and_large_values():
    q, k, qw, kw, pos, table = draw(5, 3, 1, 64, "fp16", 64, seed=6)
    q[0, 1] = 0
    q[1] = 60000.0
    k[2, 0] = 0
    a, b = kda.head_norm_rope(q, k, qw, kw, pos, table)
    check(a, q, qw, table, pos, "half", 1e-6, True, "fp16")
    check(b, k, kw, table, pos, "half", 1e-6, True, "fp16")
    a, _ = kda.head_norm_rope(q, k, eps=0.0)
    assert torch().isnan(a[0, 1]).all() and not torch().isnan(a[1:]).any()


def test_positions_out_of_the_table_are_clamped_and_reported():
    t = torch()
    q, k, qw, kw, pos, table = draw(9, 4, 2, 128, "bf16", 32, seed=7, max_pos=50)
    pos[3], pos[5] = -4, 50
    kda.device_error(reset=True)
    a, _ = kda.head_norm_rope(q, k, qw, kw, pos, table)
    assert kda.device_error(reset=True) == kda.ERR_BAD_POSITION
    check(a, q, qw, table, pos.clamp(0, 49), "half", 1e-6, True, "bf16")
    a, _ = kda.head_norm_rope(q, k, qw, kw, pos.clamp(0, 49).to(t.int32), table)
    assert kda.device_error(reset=True) == 0


def test_no_rows_and_another_stream():
    t = torch()
    q, k, qw, kw, pos, table = draw(40, 8, 8, 64, "bf16", 64, seed=8)
    a, b = kda.head_norm_rope(q[:0], k[:0], qw, kw, pos[:0], table)
    assert a.shape == (0, 8, 64) and b.shape == (0, 8, 64)
    want = kda.head_norm_rope(q, k, qw, kw, pos, table)
    t.cuda.synchronize()
    s = t.cuda.Stream()
    with t.cuda.stream(s):
        got = kda.head_norm_rope(q, k, qw, kw, pos, table)
    s.synchronize()
    assert t.equal(got[0], want[0]) and t.equal(got[1], want[1])


def test_outputs_on_a_given_stream():
    t = torch()
    q, k, qw, kw, pos, table = draw(300, 8, 8, 64, "bf16", 64, seed=18)
    want = kda.head_norm_rope(q, k, qw, kw, pos, table)
    got = beside_pending_work(lambda s: kda.head_norm_rope(q, k, qw, kw, pos, table, stream=s), (300, 8, 64), t.bfloat16)
    assert t.equal(got[0], want[0]) and t.equal(got[1], want[1])


def test_first_axis_of_one_row_may_have_any_stride():
    t = torch()
    q, k, qw, kw, pos, table = draw(3, 8, 2, 128, "bf16", 128, seed=9)
    want = kda.head_norm_rope(q, k, qw, kw, pos, table)
    got = kda.head_norm_rope(q[1:2].as_strided((1, 8, 128), (7, 128, 1), q[1:2].storage_offset()), k[1:2], qw, kw,
                             pos[1:2], table)
    assert t.equal(got[0], want[0][1:2]) and t.equal(got[1], want[1][1:2])


def test_table_turns_like_the_angles():
    tab = f64(kda.rope_table(300, 32, base=500.0))
    f = 500.0 ** (-2.0 * np.arange(16) / 32)
    a = np.arange(300)[:, None] * f
    assert np.abs(tab - np.concatenate([np.cos(a), np.sin(a)], 1)).max() <= 2.0 ** -24
