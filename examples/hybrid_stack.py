"""A small hybrid decoder served with this library: linear-attention layers and window-attention layers in turn.

Every layer keeps a fixed-size entry per sequence in a pool (recurrent state and conv window, or keys and values of the
window and the sinks), and one slot id addresses a sequence in all of them.  The script prefills packed prompts, forks
each prompt's slots into parallel samples, decodes, retires some samples and compacts the pools, decodes on, and checks
the samples against a prefill of their whole texts.

    python examples/hybrid_stack.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kda_linear_attention_chunk_gb300 as kda  # noqa: E402


def rms_norm(x, eps=1e-6):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + eps)).to(x.dtype)


class LinearLayer:
    """A KDA layer: projections, short conv, L2 norm, recurrence, output projection."""

    def __init__(self, dim, heads, slots, g):
        self.heads, d = heads, 128
        w = lambda *s: (torch.randn(*s, generator=g, device="cuda") / math.sqrt(s[0])).bfloat16()   # noqa: E731
        self.qkv, self.gate, self.beta, self.out = w(dim, 3 * heads * d), w(dim, heads * d), w(dim, heads), w(heads * d, dim)
        self.conv = 0.5 * torch.randn(3, heads * d, 4, generator=g, device="cuda")
        self.windows = torch.zeros(slots, 3, 3, heads * d, dtype=torch.bfloat16, device="cuda")
        self.states = torch.zeros(slots, heads, d, d, device="cuda")
        self.pools = [self.windows, self.states]

    def _project(self, x):
        T, h = x.shape[0], self.heads
        y = rms_norm(x)
        q, k, v = (p.contiguous().view(T, h, 128) for p in (y @ self.qkv).chunk(3, -1))
        decay = -0.15 * torch.sigmoid((y @ self.gate).float()).view(T, h, 128)
        return q, k, v, decay, torch.sigmoid((y @ self.beta).float())

    def prefill(self, x, cu, starts, slots):
        q, k, v, g, beta = self._project(x)
        o = kda.chunk_prefill_conv(q, k, v, self.conv, g, beta, cu, self.windows, self.states, slots=slots)
        return x + o.flatten(1) @ self.out

    def decode(self, x, positions, slots):
        q, k, v, g, beta = self._project(x)
        o = kda.decode_conv(q, k, v, self.conv, self.windows, g, beta, self.states, conv_slots=slots, state_slots=slots)
        return x + o.flatten(1) @ self.out


class WindowLayer:
    """A softmax layer over a sliding window and sinks: fused projection, norm and rotation per head, ring cache."""

    def __init__(self, dim, heads, kv_heads, window, sinks, slots, table, g):
        self.hq, self.hk, self.window, self.sinks, self.table = heads, kv_heads, window, sinks, table
        w = lambda *s: (torch.randn(*s, generator=g, device="cuda") / math.sqrt(s[0])).bfloat16()   # noqa: E731
        self.qkv, self.out = w(dim, (heads + 2 * kv_heads) * 128), w(heads * 128, dim)
        self.qw, self.kw = (1 + 0.1 * torch.randn(2, 128, generator=g, device="cuda")).unbind(0)
        self.cache = torch.empty(slots, 2, kv_heads, sinks + window, 128, dtype=torch.bfloat16, device="cuda")
        self.pools = [self.cache]

    def _project(self, x, positions):
        y = (rms_norm(x) @ self.qkv).view(x.shape[0], -1, 128)
        q, k = kda.head_norm_rope(y[:, :self.hq], y[:, self.hq:self.hq + self.hk], q_weight=self.qw, k_weight=self.kw,
                                  positions=positions, table=self.table)
        return q, k, y[:, self.hq + self.hk:]

    def prefill(self, x, cu, starts, slots):
        n = torch.repeat_interleave(torch.arange(len(cu) - 1, device="cuda"), cu.diff())
        positions = (torch.arange(x.shape[0], device="cuda") - cu[n] + starts[n]).int()
        q, k, v = self._project(x, positions)
        o = kda.window_prefill(q, k, v, cu, self.window, sinks=self.sinks, kv_pool=self.cache, slots=slots, starts=starts)
        return x + o.flatten(1) @ self.out

    def decode(self, x, positions, slots):
        q, k, v = self._project(x, positions)
        o = kda.window_decode(q, k, v, positions, self.cache, self.window, sinks=self.sinks, slots=slots)
        return x + o.flatten(1) @ self.out


class HybridStack:
    def __init__(self, dim=512, heads=4, kv_heads=2, window=96, sinks=4, depth=2, slots=32, max_pos=4096, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        table = kda.rope_table(max_pos, 128, stretch=4.0, trained=max_pos // 4)
        self.slots = slots
        self.layers = []
        for _ in range(depth):
            self.layers += [LinearLayer(dim, heads, slots, g),
                            WindowLayer(dim, heads, kv_heads, window, sinks, slots, table, g)]
        self.pools = [p for layer in self.layers for p in layer.pools]

    def ids(self, values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    def prefill(self, x, lens, slots, starts=None):
        """x: [T][dim], the packed new tokens of each sequence; returns the last layer's outputs."""
        cu = self.ids([0] + torch.tensor(lens).cumsum(0).tolist())
        starts = self.ids([0] * len(lens)) if starts is None else starts
        for layer in self.layers:
            x = layer.prefill(x, cu, starts, slots)
        return x

    def decode(self, x, positions, slots):
        for layer in self.layers:
            x = layer.decode(x, positions, slots)
        return x

    def fork(self, src, dst):
        """Entries src become entries dst in every pool; src -1 clears."""
        kda.slots_copy(self.pools, self.ids(src), self.ids(dst))

    def compact(self, slots):
        return kda.slots_compact(self.pools, slots)


def main(seed=0, dim=512, steps=12):
    """Runs the whole story; returns the largest relative error of the decoded outputs against a prefill of the same
    texts, which must stay at what 16-bit layers leave."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    net = HybridStack(dim=dim, seed=seed)
    lens, copies = [150, 1, 37], 3
    prompts = [torch.randn(n, dim, generator=g, device="cuda").bfloat16() for n in lens]
    origin = [20, 9, 30]
    net.fork([-1] * 3, origin)                                    # fresh entries
    # the first prompt in two chunks, the second one packed with the others
    net.prefill(torch.cat([prompts[0][:100], prompts[1], prompts[2]]), [100, 1, 37], net.ids(origin))
    net.prefill(prompts[0][100:], [50], net.ids(origin[:1]), starts=net.ids([100]))
    # three samples of each prompt, in any free slots
    slots = [2, 31, 5, 17, 8, 25, 11, 14, 3]
    owner = [i // copies for i in range(9)]
    net.fork([origin[i] for i in owner], slots)
    texts = [prompts[i] for i in owner]
    table, live = net.ids(slots), list(range(9))
    outputs = [[] for _ in range(9)]
    for step in range(steps):
        if step == steps // 2:                                    # some samples end; the others move to the front
            keep = [True, False, True, True, False, False, True, True, True]
            table = net.compact(torch.where(torch.tensor(keep, device="cuda"), table, -1))
            live = [i for i in live if keep[i]]
        x = torch.randn(9, dim, generator=g, device="cuda").bfloat16()
        positions = net.ids([len(texts[i]) for i in range(9)])
        y = net.decode(x, positions, table)                       # retired rows carry slot -1 and are skipped
        for i in live:
            texts[i] = torch.cat([texts[i], x[i:i + 1]])
            outputs[i].append(y[i])
    # the same texts by one packed prefill into fresh entries
    check = HybridStack(dim=dim, seed=seed)
    whole = check.prefill(torch.cat([texts[i] for i in live]), [len(texts[i]) for i in live], check.ids(list(range(len(live)))))
    worst, end = 0.0, 0
    for i in live:
        end += len(texts[i])
        want = whole[end - len(outputs[i]):end].float()
        got = torch.stack(outputs[i]).float()
        worst = max(worst, float((got - want).norm() / want.norm()))
    assert sorted(s for s in table.tolist() if s >= 0) == list(range(len(live)))
    return worst


if __name__ == "__main__":
    print(f"decoded outputs against a prefill of the same texts: relative L2 error {main():.2e}")
