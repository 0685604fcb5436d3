"""kda_window_prefill and kda_window_decode on the GPU against softmax attention
in 64 bits, key by key; the ring cache against a copy kept on the host, bit for
bit.  Cache rows that hold no visible position are filled with NaN."""
import numpy as np
import pytest

import kda_linear_attention_chunk_gb300 as kda
from gpu_util import torch
from hybrid_util import attention, beside_pending_work, f64, row_of, torch_dtype, worst

pytestmark = pytest.mark.gpu


class Batch:
    """Sequences with cached contexts: the full key and value history on the host, the pool on the device."""

    def __init__(self, starts, Hq, Hk, d, window, sinks, dtype, extra=0, seed=0, entries=None, scale=None):
        t = torch()
        self.g = t.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.N, self.Hq, self.Hk, self.d = len(starts), Hq, Hk, d
        self.window, self.sinks, self.dtype, self.rows = window, sinks, dtype, window + sinks + extra
        self.scale = d ** -0.5 if scale is None else scale
        entries = entries or self.N + 2
        rng = np.random.default_rng(seed)
        self.slots = [int(x) for x in rng.permutation(entries)[:self.N]]
        self.length = list(starts)
        self.pool = t.full((entries, 2, Hk, self.rows, d), float("nan"), dtype=torch_dtype(dtype), device="cuda")
        self.keys, self.values = [], []
        for n, a in enumerate(starts):
            k, v = self.rand(a, Hk), self.rand(a, Hk)
            self.keys.append({})
            self.values.append({})
            self.keep(n, 0, f64(k), f64(v))
            for p in self.held(a):
                self.pool[self.slots[n], 0, :, row_of(p, sinks, self.rows)] = k[p]
                self.pool[self.slots[n], 1, :, row_of(p, sinks, self.rows)] = v[p]

    def rand(self, rows, heads):
        t = torch()
        return (1.5 * t.randn(rows, heads, self.d, generator=self.g, device="cuda")).to(torch_dtype(self.dtype))

    def held(self, length):
        """Positions that the cache holds of a context of that length."""
        return [p for p in range(length) if p < self.sinks or p >= length - (self.rows - self.sinks)]

    def keep(self, n, start, k, v):
        for i in range(k.shape[0]):
            self.keys[n][start + i], self.values[n][start + i] = k[i], v[i]

    def new_rows(self, T, fused=True):
        qkv = self.rand(T, self.Hq + 2 * self.Hk)
        parts = qkv[:, :self.Hq], qkv[:, self.Hq:self.Hq + self.Hk], qkv[:, self.Hq + self.Hk:]
        return parts if fused else tuple(x.contiguous() for x in parts)

    def ids(self, padded=()):
        t = torch()
        return t.tensor([-1 if n in padded else s for n, s in enumerate(self.slots)], dtype=t.int32, device="cuda")

    def int32(self, x):
        t = torch()
        return t.tensor(x, dtype=t.int32, device="cuda")

    def expected_pool(self, was, rows):
        """The pool after rows[n] = (k, v) device rows of each unpadded sequence joined its context."""
        want = was.clone()
        for n, (k, v) in rows.items():
            a, L = self.length[n], k.shape[0]
            for p in self.held(a + L):
                if p >= a:
                    want[self.slots[n], 0, :, row_of(p, self.sinks, self.rows)] = k[p - a]
                    want[self.slots[n], 1, :, row_of(p, self.sinks, self.rows)] = v[p - a]
        return want

    def prefill(self, lens, padded=(), cached=True, fused=True, check_rows=None, qkv=None, starts=True):
        t = torch()
        cu = np.concatenate([[0], np.cumsum(lens)])
        T = int(cu[-1])
        q, k, v = self.new_rows(T, fused) if qkv is None else qkv
        out = t.full((T, self.Hq, self.d), 7.0, dtype=q.dtype, device="cuda")
        was = self.pool.clone()
        kw = dict(kv_pool=self.pool, slots=self.ids(padded), starts=self.int32(self.length) if starts else None)
        kda.window_prefill(q, k, v, self.int32(cu), self.window, sinks=self.sinks, scale=self.scale, out=out,
                           **(kw if cached else {}))
        got, joined = f64(out), {}
        for n, L in enumerate(lens):
            rows = slice(int(cu[n]), int(cu[n + 1]))
            if n in padded:
                assert (got[rows] == 7.0).all()
                continue
            joined[n] = (k[rows], v[rows])
            self.keep(n, self.length[n], f64(k[rows]), f64(v[rows]))
            if L == 0:
                continue
            picks = range(L) if check_rows is None else sorted({min(L - 1, i) for i in check_rows})
            qs = f64(q[rows])[list(picks)]
            ref, bound = attention(qs, self.keys[n], self.values[n], [self.length[n] + i for i in picks], self.window,
                                   self.sinks, self.scale, self.dtype)
            assert worst(got[rows][list(picks)], ref, bound) <= 1.0, n
        if cached:
            want = self.expected_pool(was, joined)
            assert t.equal(self.pool.view(t.int16), want.view(t.int16))
        for n in joined:
            self.length[n] += lens[n]
        return out

    def decode(self, padded=(), fused=True):
        t = torch()
        q, k, v = self.new_rows(self.N, fused)
        out = t.full((self.N, self.Hq, self.d), 7.0, dtype=q.dtype, device="cuda")
        was = self.pool.clone()
        kda.window_decode(q, k, v, self.int32(self.length), self.pool, self.window, sinks=self.sinks,
                          slots=self.ids(padded), scale=self.scale, out=out)
        got, joined = f64(out), {}
        for n in range(self.N):
            if n in padded:
                assert (got[n] == 7.0).all()
                continue
            joined[n] = (k[n:n + 1], v[n:n + 1])
            self.keep(n, self.length[n], f64(k[n:n + 1]), f64(v[n:n + 1]))
            ref, bound = attention(f64(q[n:n + 1]), self.keys[n], self.values[n], [self.length[n]], self.window,
                                   self.sinks, self.scale, self.dtype)
            assert worst(got[n:n + 1], ref, bound) <= 1.0, n
        assert t.equal(self.pool.view(t.int16), self.expected_pool(was, joined).view(t.int16))
        for n in joined:
            self.length[n] += 1
        return out


HEADS = [(1, 1), (2, 2), (6, 2), (5, 1), (8, 1), (14, 2), (16, 1), (40, 2), (48, 1), (128, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hk", HEADS)
def test_prefill_heads_and_types(Hq, Hk, d, dtype):
    b = Batch([0, 30, 3], Hq, Hk, d, window=11, sinks=2, dtype=dtype, seed=Hq)
    b.prefill([37, 1, 20])


# (sequences, rows of each) with few rows a sequence, where the warp-MMA kernel runs, and with more, where the
# tensor-core tiles do: rows x query heads per key head at most 32 a sequence, or up to 256 of a single sequence
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (4, 1), (10, 2), (16, 1), (20, 1), (33, 1), (64, 1), (100, 1), (128, 1)])
@pytest.mark.parametrize("N,L", [(40, 1), (40, 2), (7, 5), (1, 3), (1, 8), (1, 70), (5, 40), (3, 300)])
def test_prefill_from_few_rows_to_many(N, L, Hq, Hk, d):
    """Both kernels and every sharing of keys between warps, over contexts around the window and the ring's wrap."""
    b = Batch([(37 * i + 5) % 90 for i in range(N)], Hq, Hk, d, window=24, sinks=3, dtype="bf16", seed=N + Hq)
    b.prefill([L + (i % 3 == 1) - (i % 4 == 2) for i in range(N)], check_rows=[0, 1, 2, 4, 7, 8, 31, 39, 64, 127, 128, 299])


@pytest.mark.parametrize("lens", [[1] * 60 + [700], [0] * 50 + [90, 0, 3], [2] * 3 + [500] + [0] * 70])
def test_prefill_mixed_lengths_under_one_rule(lens):
    """The kernel is chosen by the average: long sequences among many short ones."""
    b = Batch([20 + 3 * i for i in range(len(lens))], 8, 2, 64, window=40, sinks=2, dtype="bf16", seed=len(lens))
    b.prefill(lens, check_rows=[0, 1, 3, 15, 16, 63, 64, 130, 499, 699])


@pytest.mark.parametrize("window,sinks,extra", [(1, 0, 0), (1, 3, 0), (2, 0, 5), (16, 16, 0), (17, 1, 3), (63, 0, 1),
                                                (64, 4, 0), (128, 0, 0), (129, 5, 7), (300, 130, 0)])
def test_prefill_windows_and_contexts(window, sinks, extra):
    b = Batch([0, 1, window, window + sinks, 2 * window + 3, 500], 4, 2, 64, window, sinks, "bf16", extra=extra, seed=window)
    b.prefill([70, 0, 1, 33, 129, 65])
    b.prefill([1, 5, 0, 64, 2, 140])


@pytest.mark.parametrize("window,sinks", [(100, 3), (1024, 4), (5000, 0)])
def test_prefill_long_rows(window, sinks):
    """Thousands of rows, checked at tile edges and a few others."""
    b = Batch([0, 700], 4, 1, 128, window, sinks, "bf16", seed=1)
    edges = [0, 1, 15, 16, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 1000, 1023, 1024, 1030, 1999, 2047,
             2048, 2100, 2499]
    b.prefill([2500, 1100], check_rows=edges)


def test_prefill_in_chunks_equals_the_formula_throughout():
    b = Batch([0, 0], 8, 2, 128, window=50, sinks=5, dtype="bf16", seed=2)
    for lens in ([3, 60], [1, 1], [200, 0], [7, 90], [128, 128]):
        b.prefill(lens)


def test_prefill_without_a_cache():
    b = Batch([0, 0, 0], 6, 2, 128, window=40, sinks=6, dtype="fp16", seed=3)
    b.prefill([100, 0, 55], cached=False)


def test_prefill_wider_window_than_any_context_is_causal_attention():
    t = torch()
    small = Batch([0], 4, 4, 64, window=300, sinks=0, dtype="bf16", seed=4)
    q, k, v = small.new_rows(300)
    a = kda.window_prefill(q, k, v, small.int32([0, 300]), 300)
    c = kda.window_prefill(q, k, v, small.int32([0, 300]), 0x7fffffff)
    assert t.equal(a, c)
    small.prefill([300], cached=False, qkv=(q, k, v))


def test_prefill_sinks_and_window_beyond_everything():
    """Without a cache neither is bounded by one; both at the largest number are causal attention."""
    t = torch()
    for T in (40, 500):
        b = Batch([0], 4, 2, 64, window=T, sinks=0, dtype="bf16", seed=T)
        q, k, v = b.new_rows(T)
        want = kda.window_prefill(q, k, v, b.int32([0, T]), T)
        for window, sinks in ((0x7fffffff, 0x7fffffff), (1, 0x7fffffff), (3, T)):
            assert t.equal(kda.window_prefill(q, k, v, b.int32([0, T]), window, sinks=sinks), want)


@pytest.mark.parametrize("L", [1, 10])
def test_prefill_many_sequences(L):
    """More sequences than one round of probes tells apart, some empty, for both kernels."""
    rng = np.random.default_rng(L)
    lens = [int(x) for x in rng.integers(0, 2 * L + 1, 1200)]
    b = Batch([int(x) for x in rng.integers(0, 12, 1200)], 4, 1, 64, window=9, sinks=1, dtype="bf16", seed=L)
    b.prefill(lens, padded=(3, 700), check_rows=[0, L, 2 * L - 1])


def test_offsets_beyond_32_bits():
    """Rows, outputs and cache entries whose offsets pass 2^31 elements: rows at the end against the same rows alone."""
    t = torch()
    T, H, d = (1 << 31) // 2048 + 700, 16, 128
    free = t.cuda.mem_get_info()[0]
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    qkv = t.empty(T, H + 2, d, dtype=t.bfloat16, device="cuda").normal_()
    q, k, v = qkv[:, :H], qkv[:, H:H + 1], qkv[:, H + 1:]
    cu = t.tensor([0, T], dtype=t.int32, device="cuda")
    out = kda.window_prefill(q, k, v, cu, 50)
    tail = kda.window_prefill(q[-300:], k[-300:], v[-300:], t.tensor([0, 300], dtype=t.int32, device="cuda"), 50)
    # as far as the reduction's order goes: the tiles of the two calls start at different rows
    assert (out[-250:].float() - tail[-250:].float()).abs().max() <= 2.0 ** -5
    a, b = kda.head_norm_rope(q, k, positions=t.zeros(T, dtype=t.int32, device="cuda"), table=kda.rope_table(1, d))
    x, y = kda.head_norm_rope(q[-9:], k[-9:], positions=t.zeros(9, dtype=t.int32, device="cuda"), table=kda.rope_table(1, d))
    assert t.equal(a[-9:], x) and t.equal(b[-9:], y)
    del out, a, b
    rows, slots = 140000, 64                       # 64 x 2 x 140000 x 128 elements
    pool = t.zeros(slots, 2, 1, rows, d, dtype=t.bfloat16, device="cuda")
    assert pool.numel() > 1 << 31
    small = t.empty(1, 2, 1, rows, d, dtype=t.bfloat16, device="cuda").normal_()
    pool[slots - 1] = small[0]
    ids, start = t.tensor([slots - 1], dtype=t.int32, device="cuda"), t.tensor([200000], dtype=t.int32, device="cuda")
    for L in (1, 2, 300):
        cu = t.tensor([0, L], dtype=t.int32, device="cuda")
        p, s = pool, small.clone()
        got = kda.window_prefill(q[:L], k[:L], v[:L], cu, rows - 4, sinks=4, kv_pool=p, slots=ids, starts=start)
        want = kda.window_prefill(q[:L], k[:L], v[:L], cu, rows - 4, sinks=4, kv_pool=s, starts=start)
        assert t.equal(got, want) and t.equal(p[slots - 1], s[0])
        pool[slots - 1] = small[0]
    got = kda.window_decode(q[:1], k[:1], v[:1], start, pool, rows - 4, sinks=4, slots=ids)
    s = small.clone()
    assert t.equal(got, kda.window_decode(q[:1], k[:1], v[:1], start, s, rows - 4, sinks=4))
    assert t.equal(pool[slots - 1], s[0])
    kda.slots_copy([pool], ids, t.tensor([3], dtype=t.int32, device="cuda"))
    assert t.equal(pool[3], pool[slots - 1])


@pytest.mark.parametrize("window", [60, 1000])
@pytest.mark.parametrize("L", [1, 3, 50, 300, 700])
@pytest.mark.parametrize("Hq,Hk,d", [(1, 1, 64), (5, 1, 64), (8, 2, 128)])
def test_positions_up_to_the_largest(Hq, Hk, d, L, window):
    """Whole turns of the ring apart, contexts give the same bytes, up to the last positions that an int32 holds."""
    t = torch()
    sinks, rows = 4, window + 9
    ring, top = rows - sinks, (1 << 31) - 1 - L
    near = ring * 3 + (top - sinks) % ring + sinks
    b = Batch([0], Hq, Hk, d, window, sinks, "bf16", extra=5, seed=L)
    b.pool.normal_()
    q, k, v = b.new_rows(L)
    cu = b.int32([0, L])
    kda.device_error(reset=True)
    pools = [b.pool.clone() for _ in range(2)]
    got = [kda.window_prefill(q, k, v, cu, window, sinks=sinks, kv_pool=p, slots=b.ids(), starts=b.int32([s]))
           for p, s in zip(pools, (near, top))]
    assert b.pool.shape[3] == rows and t.isfinite(got[0]).all()
    assert t.equal(*got) and t.equal(*pools)
    for back in (0, 1):
        got = [kda.window_decode(q[:1], k[:1], v[:1], b.int32([s + L - back]), p, window, sinks=sinks, slots=b.ids())
               for p, s in zip(pools, (near, top))]
        assert t.equal(*got) and t.equal(*pools)
    assert kda.device_error() == 0


def test_prefill_padded_and_bad_slots():
    t = torch()
    b = Batch([10, 20, 30, 0], 4, 2, 128, window=9, sinks=2, dtype="bf16", seed=5)
    b.prefill([12, 40, 3, 8], padded=(1,))
    b.prefill([120, 140, 300, 8], padded=(2,))
    kda.device_error(reset=True)
    q, k, v = b.new_rows(9)
    ids = b.ids()
    ids[2] = b.pool.shape[0]
    ids[3] = -2
    was = b.pool.clone()
    out = t.full((9, 4, 128), 7.0, dtype=q.dtype, device="cuda")
    kda.window_prefill(q, k, v, b.int32([0, 2, 4, 6, 9]), 9, sinks=2, kv_pool=b.pool, slots=ids,
                       starts=b.int32(b.length), out=out)
    assert kda.device_error(reset=True) == kda.ERR_BAD_SLOT
    assert (out[4:] == 7.0).all() and not (out[:4] == 7.0).all(-1).any()
    changed = (b.pool.view(t.int16) != was.view(t.int16)).flatten(1).any(1).nonzero().flatten().tolist()
    assert set(changed) <= {b.slots[0], b.slots[1]}


def test_prefill_bad_starts_are_clamped_and_reported():
    b = Batch([0, 0], 2, 1, 64, window=8, sinks=0, dtype="bf16", seed=6)
    q, k, v = b.new_rows(10)
    kda.device_error(reset=True)
    out = kda.window_prefill(q, k, v, b.int32([0, 5, 10]), 8, kv_pool=b.pool, slots=b.ids(), starts=b.int32([-3, 0]))
    assert kda.device_error(reset=True) == kda.ERR_BAD_POSITION
    ref = kda.window_prefill(q, k, v, b.int32([0, 5, 10]), 8)
    assert torch().equal(out, ref)


def test_prefill_bad_sequence_table_stays_in_bounds():
    b = Batch([0, 0], 2, 1, 64, window=8, sinks=0, dtype="bf16", seed=7)
    q, k, v = b.new_rows(10)
    kda.device_error(reset=True)
    kda.window_prefill(q, k, v, b.int32([0, 5, 4000]), 8, kv_pool=b.pool, slots=b.ids(), starts=b.int32([0, 0]))
    assert kda.device_error(reset=True) == kda.ERR_BAD_SEQLENS


@pytest.mark.parametrize("T", [80, 400])
def test_masked_keys_never_reach_an_output(T):
    """Keys that are infinite, NaN or of the type's lowest value change only the rows that see them; rows that see
    them would give NaN."""
    t = torch()
    for bad in (float("inf"), float("-inf"), float("nan"), t.finfo(t.bfloat16).min):
        b = Batch([0], 4, 2, 128, window=6, sinks=0, dtype="bf16", seed=8)
        q, k, v = b.new_rows(T, fused=False)
        clean = kda.window_prefill(q, k, v, b.int32([0, T]), 6)
        k2 = k.clone()
        k2[3] = bad
        k2[40] = bad
        got = kda.window_prefill(q, k2, v, b.int32([0, T]), 6)
        seen = [r for r in range(T) if 3 <= r < 9 or 40 <= r < 46]
        rest = [r for r in range(T) if r not in seen]
        assert t.equal(got[rest], clean[rest])


@pytest.mark.parametrize("a,b_,c", [(19, 40, 61), (5, 12, 20), (300, 511, 700)])
def test_values_of_other_sequences_never_reach_an_output(a, b_, c):
    t = torch()
    b = Batch([0, 0, 0], 4, 2, 64, window=20, sinks=3, dtype="bf16", seed=9)
    q, k, v = b.new_rows(c, fused=False)
    cu = b.int32([0, a, b_, c])
    clean = kda.window_prefill(q, k, v, cu, 20, sinks=3)
    k[a:b_], v[a:b_] = float("nan"), float("nan")
    got = kda.window_prefill(q, k, v, cu, 20, sinks=3)
    assert t.equal(got[:a], clean[:a]) and t.equal(got[b_:], clean[b_:])


def test_large_scores_and_lowest_values():
    """Scores of thousands (one key takes all the weight) stay finite; a large scale too."""
    b = Batch([40], 4, 1, 64, window=33, sinks=2, dtype="bf16", seed=10, scale=30.0)
    b.prefill([50])
    b.decode()


def test_prefill_empty_call_and_other_stream():
    t = torch()
    b = Batch([4, 9], 4, 2, 128, window=10, sinks=1, dtype="bf16", seed=11)
    was = b.pool.clone()
    q, k, v = b.new_rows(0)
    assert kda.window_prefill(q, k, v, b.int32([0, 0, 0]), 10, sinks=1, kv_pool=b.pool, slots=b.ids(),
                              starts=b.int32(b.length)).shape == (0, 4, 128)
    assert t.equal(was.view(t.int16), b.pool.view(t.int16))
    q, k, v = b.new_rows(12)
    cu, ids, st = b.int32([0, 5, 12]), b.ids(), b.int32(b.length)
    p1, p2 = b.pool.clone(), b.pool.clone()
    want = kda.window_prefill(q, k, v, cu, 10, sinks=1, kv_pool=p1, slots=ids, starts=st)
    t.cuda.synchronize()
    s = t.cuda.Stream()
    got = kda.window_prefill(q, k, v, cu, 10, sinks=1, kv_pool=p2, slots=ids, starts=st, stream=s)
    s.synchronize()
    assert t.equal(got, want) and t.equal(p1.view(t.int16), p2.view(t.int16))


def test_outputs_on_a_given_stream():
    t = torch()
    b = Batch([0] * 40, 8, 2, 128, window=40, sinks=2, dtype="bf16", seed=25)
    q, k, v = b.new_rows(40)
    cu, ids, st = b.int32(list(range(41))), b.ids(), b.int32(b.length)
    for call in (lambda s: kda.window_prefill(q, k, v, cu, 40, sinks=2, kv_pool=b.pool, slots=ids, starts=st, stream=s),
                 lambda s: kda.window_decode(q, k, v, st, b.pool, 40, sinks=2, slots=ids, stream=s)):
        want = call(None)
        assert t.equal(beside_pending_work(call, (40, 8, 128), t.bfloat16), want)


def test_prefill_same_bytes_every_time():
    t = torch()
    b = Batch([0, 300], 8, 2, 128, window=200, sinks=4, dtype="bf16", seed=12)
    q, k, v = b.new_rows(900)
    cu, ids, st = b.int32([0, 500, 900]), b.ids(), b.int32(b.length)
    outs = [kda.window_prefill(q, k, v, cu, 200, sinks=4, kv_pool=b.pool.clone(), slots=ids, starts=st) for _ in range(3)]
    assert t.equal(outs[0], outs[1]) and t.equal(outs[0], outs[2])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hk", HEADS)
def test_decode_heads_and_types(Hq, Hk, d, dtype):
    b = Batch([0, 1, 15, 16, 40, 100], Hq, Hk, d, window=33, sinks=3, dtype=dtype, seed=Hq)
    b.decode()
    b.decode(padded=(2,))


@pytest.mark.parametrize("window,sinks,extra", [(1, 0, 0), (1, 2, 0), (7, 9, 4), (128, 0, 0), (130, 5, 0), (1000, 4, 24)])
def test_decode_windows_and_contexts(window, sinks, extra):
    b = Batch([0, window - 1, window, window + sinks, 2 * window + sinks + 1, 1500], 4, 2, 64, window, sinks, "bf16",
              extra=extra, seed=window)
    for _ in range(3):
        b.decode()


def test_decode_large_batch_and_single_sequence():
    Batch([int(x) for x in np.random.default_rng(0).integers(0, 400, 200)], 8, 2, 64, 150, 4, "bf16", seed=13).decode()
    Batch([2000], 16, 1, 128, 1500, 4, "bf16", seed=14).decode()


def test_decode_after_prefill_and_verify():
    """A prompt, single tokens, three drafted tokens of which one is kept (the ring has room for the rejected two)."""
    b = Batch([0, 0], 4, 2, 128, window=20, sinks=2, dtype="bf16", extra=2, seed=15)
    b.prefill([45, 9])
    b.decode()
    lens = list(b.length)
    b.prefill([3, 3])
    b.length = [x + 1 for x in lens]      # one draft kept; the positions of the others are taken again
    b.decode()
    b.decode()


def test_decode_bad_position_and_slot():
    b = Batch([5, 6, 7], 2, 1, 64, window=8, sinks=0, dtype="bf16", seed=16)
    q, k, v = b.new_rows(3)
    kda.device_error(reset=True)
    ids = b.ids()
    ids[1] = 99
    out = torch().full((3, 2, 64), 7.0, dtype=q.dtype, device="cuda")
    kda.window_decode(q, k, v, b.int32([-1, 6, 7]), b.pool, 8, slots=ids, out=out)
    assert kda.device_error(reset=True) == kda.ERR_BAD_POSITION | kda.ERR_BAD_SLOT
    assert (out[1] == 7.0).all()
    assert torch().equal(out[0], v[0].expand(2, 64))     # position 0 sees itself alone


def test_decode_other_stream_and_same_bytes():
    t = torch()
    b = Batch([300, 20], 8, 1, 128, window=200, sinks=4, dtype="bf16", seed=17)
    q, k, v = b.new_rows(2)
    pos, ids = b.int32(b.length), b.ids()
    want = kda.window_decode(q, k, v, pos, b.pool, 200, sinks=4, slots=ids)
    t.cuda.synchronize()
    s = t.cuda.Stream()
    got = kda.window_decode(q, k, v, pos, b.pool, 200, sinks=4, slots=ids, stream=s)
    s.synchronize()
    assert t.equal(got, want)


def test_entries_without_a_table_and_graph_replay():
    """slots None means entry n; a captured decode step replays."""
    t = torch()
    b = Batch([50, 3], 4, 2, 64, window=30, sinks=1, dtype="bf16", seed=18)
    b.slots = [0, 1]
    b.pool.normal_()
    q, k, v = b.new_rows(2)
    pos = b.int32([50, 3])
    want = kda.window_decode(q, k, v, pos, b.pool.clone(), 30, sinks=1, slots=b.int32([0, 1]))
    out = t.empty_like(want)
    kda.window_decode(q, k, v, pos, b.pool, 30, sinks=1, out=out)
    assert t.equal(out, want)
    cu = b.int32([0, 1, 2])
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph, stream=s):
        kda.window_decode(q, k, v, pos, b.pool, 30, sinks=1, out=out)
        kda.window_prefill(q, k, v, cu, 30, sinks=1, kv_pool=b.pool)
    out.zero_()
    graph.replay()
    t.cuda.synchronize()
    assert t.equal(out, want)

