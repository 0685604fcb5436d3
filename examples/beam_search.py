"""Beam search over a small hybrid decoder: linear-attention layers and softmax layers that see the whole context in turn.

A prompt's keys and values stay in the pages of its own slot and are read once for all of its beams; a beam owns the
pages of what it has generated, its recurrent state and its conv window, all reached by one slot id.  Each step appends
the beams' new tokens, attends, selects, and lets states and pages follow: most beams stay where they are, and only the
further children of a beam are copied.  In the end every hypothesis is run again as one prefill.

    python examples/beam_search.py
"""
import math
import os
import sys

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path[:0] = [os.path.dirname(HERE), HERE]
import kda_linear_attention_chunk_gb300 as kda  # noqa: E402
from hybrid_stack import LinearLayer, rms_norm  # noqa: E402


class PagedLayer:
    """A softmax layer over the whole context: fused projection, norm and rotation per head, paged cache."""

    def __init__(self, dim, heads, kv_heads, pages, page, angles, g):
        self.hq, self.hk, self.angles = heads, kv_heads, angles
        w = lambda *s: (torch.randn(*s, generator=g, device="cuda") / math.sqrt(s[0])).bfloat16()   # noqa: E731
        self.qkv, self.out = w(dim, (heads + 2 * kv_heads) * 128), w(heads * 128, dim)
        self.qw, self.kw = (1 + 0.1 * torch.randn(2, 128, generator=g, device="cuda")).unbind(0)
        self.cache = torch.empty(pages, 2, kv_heads, page, 128, dtype=torch.bfloat16, device="cuda")

    def __call__(self, x, table, starts, cu, slots, prefixes=None):
        y = (rms_norm(x) @ self.qkv).view(x.shape[0], -1, 128)
        q = kda.paged_append(y[:, :self.hq], y[:, self.hq:self.hq + self.hk], y[:, self.hq + self.hk:], self.cache, table,
                             starts, cu_seqlens=cu, slots=slots, q_weight=self.qw, k_weight=self.kw, table=self.angles)
        o = kda.paged_attention(q, self.cache, table, starts, cu_seqlens=cu, slots=slots, prefixes=prefixes)
        return x + o.flatten(1) @ self.out


class Decoder:
    def __init__(self, vocab=500, dim=512, heads=4, kv_heads=2, depth=2, slots=32, page=16, max_pages=24, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        angles = kda.rope_table(page * max_pages, 128)
        self.embed, self.head = torch.randn(2, vocab, dim, generator=g, device="cuda").bfloat16().unbind(0)
        self.layers = []
        for _ in range(depth):
            self.layers += [LinearLayer(dim, heads, slots, g),
                            PagedLayer(dim, heads, kv_heads, slots * max_pages, page, angles, g)]
        # every slot owns as many pages as a row of the table has entries, in any order
        order = torch.randperm(slots * max_pages, generator=g, device="cuda")
        self.table = order.int().view(slots, max_pages)
        self.states = [p for layer in self.layers[::2] for p in layer.pools]
        self.caches = [layer.cache for layer in self.layers[1::2]]

    def ids(self, values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    def clear(self, slots):
        kda.slots_copy(self.states, self.ids([-1] * len(slots)), self.ids(slots))

    def prefill(self, tokens, lens, slots):
        """The packed texts of fresh slots; returns the hidden rows."""
        cu, starts, ids = self.ids([0] + torch.tensor(lens).cumsum(0).tolist()), self.ids([0] * len(lens)), self.ids(slots)
        x = self.embed[tokens]
        for linear, paged in zip(self.layers[::2], self.layers[1::2]):
            x = paged(linear.prefill(x, cu, starts, ids), self.table, starts, cu, ids)
        return x

    def step(self, tokens, starts, slots, prefixes):
        x = self.embed[tokens]
        for linear, paged in zip(self.layers[::2], self.layers[1::2]):
            x = paged(linear.decode(x, starts, slots), self.table, starts, None, slots, prefixes)
        return x

    def logits(self, x):
        return rms_norm(x) @ self.head.T / 8


def search(net, prompts, origin, slots, beams, steps, end):
    """Beam search of all prompts at once; returns scores, texts and the last hidden rows, all [prompts][beams]."""
    G, lens = len(prompts), [len(p) for p in prompts]
    net.clear(origin)
    x = net.prefill(torch.cat(prompts), lens, origin)
    last = x[torch.tensor(lens, device="cuda").cumsum(0) - 1].repeat_interleave(beams, 0)
    # each beam starts from its prompt's state; the prompt's pages are shared as they are
    kda.slots_copy(net.states, net.ids([o for o in origin for _ in range(beams)]), net.ids(slots))
    table = net.ids(slots).view(G, beams)
    prefixes = net.ids([i * beams for i in range(G + 1)]), net.ids(lens), net.ids(origin)
    before = net.ids(lens).repeat_interleave(beams)
    scores = torch.full((G, beams), -math.inf, device="cuda")
    scores[:, 0] = 0                                              # all beams are the same text still
    ended = torch.zeros(G, beams, dtype=torch.int32, device="cuda")
    texts = torch.empty(G, beams, 0, dtype=torch.int32, device="cuda")
    for i in range(steps):
        scores, parents, tokens, ended, table, src, dst = kda.beam_select(net.logits(last), scores, ended, end, table)
        src, dst = src.flatten(), dst.flatten()
        kda.slots_copy(net.states, src, dst)
        kda.pages_copy(net.caches, net.table, src, dst, before + i, start=before)
        texts = torch.cat([texts.gather(1, parents.long()[..., None].expand_as(texts)), tokens[..., None]], 2)
        last = net.step(tokens.flatten().long(), before + i, table.flatten(), prefixes)
    return scores, texts, last.view(G, beams, -1)


def main(seed=0, beams=4, steps=10):
    """Searches, and runs every hypothesis again as one prefill; returns the largest relative error of the last hidden
    rows, which must stay at what 16-bit layers leave, and the scores."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    net = Decoder(seed=seed)
    vocab, end = net.embed.shape[0], 7
    prompts = [torch.randint(8, vocab, (n,), generator=g, device="cuda") for n in (45, 1, 130)]
    slots = torch.randperm(32, generator=g, device="cuda").tolist()
    scores, texts, last = search(net, prompts, slots[:3], slots[3:3 + 3 * beams], beams, steps, end)
    check, worst = Decoder(seed=seed), 0.0
    for i, p in enumerate(prompts):
        whole = [torch.cat([p, t.long()]) for t in texts[i]]
        n = len(whole[0])
        used = list(range(beams))
        check.clear(used)
        x = check.prefill(torch.cat(whole), [n] * beams, used).view(beams, n, -1)
        for k, t in enumerate(texts[i].tolist()):
            if end not in t[:-1]:                                 # (an ended beam is carried along, not continued)
                want = x[k, -1].float()
                worst = max(worst, float((last[i, k].float() - want).norm() / want.norm()))
    assert bool((scores.diff(dim=1) <= 0).all())
    return worst, scores


if __name__ == "__main__":
    error, found = main()
    print(f"hidden rows against a prefill of the same texts: relative L2 error {error:.2e}\nscores:\n{found}")
