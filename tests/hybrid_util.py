"""Plain 64-bit forms of the operators around a hybrid stack's softmax layers,
and the element-wise bounds of their tests.

Rounding: a 16-bit result is off by at most u |ref| with u = 2^-8 (bf16, eight
significant bits) or 2^-11 (fp16, eleven), plus half the smallest subnormal.

Attention: with p_j the exact probabilities and A = sum_j p_j |v_j|,
  * the kernels round each unnormalised probability to 16 bits (its own u), so
    the sum is off by at most u A; fp16 probabilities below 2^-14 are off by up to
    2^-25 of the largest one, together 2^-25 sum_j |v_j|;
  * a score s is a d-term fp32 sum, off by at most d 2^-23 sum |q_i k_i| scale
    (round-to-nearest would give 2^-24; the tensor cores may truncate), and its
    exponential by that plus 2^-20 for exp2 and the fp32 arithmetic of its
    argument (2^-23 of an argument whose size the same sum bounds); numerator
    and denominator both carry it, so twice;
  * fp32 accumulation over n keys: n 2^-23 A.
"""
import math

import numpy as np

BITS = {"bf16": (2.0 ** -8, 2.0 ** -134), "fp16": (2.0 ** -11, 2.0 ** -25)}


def torch_dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[name]


def f64(t):
    return t.detach().to("cpu").double().numpy()


def row_of(p, sinks, rows):
    return p if p < sinks else sinks + (p - sinks) % (rows - sinks)


def visible(p, window, sinks):
    return [j for j in range(p + 1) if j > p - window or j < sinks]


def attention(q, keys, values, pos, window, sinks, scale, dtype):
    """q [rows][Hq][d] at positions pos; keys, values: {position: [Hk][d]}.  Returns out and its bound, fp64."""
    u, tiny = BITS[dtype]
    R, Hq, d = q.shape
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for r in range(R):
        js = visible(pos[r], window, sinks)
        K = np.stack([keys[j] for j in js])
        V = np.stack([values[j] for j in js])
        G = Hq // K.shape[1]
        for h in range(Hq):
            k, v = K[:, h // G], V[:, h // G]
            s = scale * (k @ q[r, h])
            size = scale * (np.abs(k) @ np.abs(q[r, h]))
            e = np.exp(s - s.max())
            p = e / e.sum()
            out[r, h] = p @ v
            A = p @ np.abs(v)
            off = 2 * ((d + 4) * 2.0 ** -23 * size.max() + 2.0 ** -20) + len(js) * 2.0 ** -23 + u
            bound[r, h] = u * np.abs(out[r, h]) + tiny + off * (1 + u) * A
            if dtype == "fp16":
                bound[r, h] += 2.0 ** -25 * np.abs(v).sum(0)
    return out, bound


def norm_rope(x, w, table, pos, layout, eps, norm, dtype):
    """x [T][H][d] fp64; table [max_pos][r] or None.  Returns out and its bound."""
    u, tiny = BITS[dtype]
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) if norm else x.copy()
    if w is not None:
        y = y * w
    size = np.abs(y)
    if table is not None:
        r = table.shape[1]
        i = np.arange(r // 2)
        a, b = (i, i + r // 2) if layout == "half" else (2 * i, 2 * i + 1)
        c, s = table[pos][:, None, :r // 2], table[pos][:, None, r // 2:]
        ya, yb = y[..., a].copy(), y[..., b].copy()
        y[..., a], y[..., b] = ya * c - yb * s, yb * c + ya * s
        size[..., a] = np.abs(ya * c) + np.abs(yb * s)
        size[..., b] = np.abs(yb * c) + np.abs(ya * s)
    # fp32: at most 8 roundings of 2^-24 after the norm, whose d-term sum of squares of one
    # sign is off by (d / 2) 2^-24 after the square root at most, and 2 ulp of rsqrt
    return y, u * np.abs(y) + tiny + (x.shape[-1] / 2 + 16) * 2.0 ** -24 * size


def worst(got, ref, bound):
    """Largest |got - ref| / bound: <= 1 passes; NaN anywhere fails."""
    x = np.abs(got - ref) / bound
    return float(x.max()) if x.size and not np.isnan(x).any() else (math.inf if x.size else 0.0)


def beside_pending_work(call, shape, dtype):
    """call(stream) on a stream of its own while the current one still has writes before it into blocks of the given
    size that were handed back: the outputs must not lie in one of those."""
    import torch

    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.empty(shape, dtype=dtype, device="cuda") for _ in range(512)]
    blocks[0].fill_(0)                             # loads the kernel: later that would wait for the sleep
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(60_000_000)                  # some 30 ms
    for b in blocks:
        b.fill_(7)
    del b, blocks[::2]                             # holes of just that size
    got = call(side)
    side.synchronize()
    torch.cuda.synchronize()
    return got
