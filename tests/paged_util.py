"""Paged caches for tests: a page table in random order with NaN wherever no position is visible, and the plain 64-bit
attention over it with the element-wise bound of hybrid_util (whose derivation holds part by part: joining parts of the
keys in fp32 adds a few roundings of 2^-24 for each part, fewer than the keys that n 2^-23 A counts)."""
import math
import random

from hybrid_util import BITS, torch_dtype


class Batch:
    """Sequences with a paged cache.  own: [(positions before the new rows, new rows)] of each sequence, the first counted
    from its prefix's end; groups: [(sequences, prefix length)], in order, from the first sequence on."""

    def __init__(self, own, groups=(), page=64, Hq=8, Hk=2, d=128, dtype="bf16", seed=0, scale=None, extra=1, loud=1.0):
        import torch
        self.t, r = torch, random.Random(seed)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.page, self.Hq, self.Hk, self.d, self.dtype = page, Hq, Hk, d, dtype
        self.scale = d ** -0.5 if scale is None else scale
        N = len(own)
        self.prefix, self.group = [0] * N, [-1] * N
        cut = [0]
        for i, (members, length) in enumerate(groups):
            for n in range(cut[-1], cut[-1] + members):
                self.prefix[n], self.group[n] = length, i
            cut.append(cut[-1] + members)
        self.lens = [b for _, b in own]
        self.start = [a + p for (a, _), p in zip(own, self.prefix)]
        slots = N + len(groups) + 2
        ids = list(range(slots))
        r.shuffle(ids)
        self.ids, self.kept = ids[:N], ids[N:N + len(groups)]
        needs = {ids[n]: (self.prefix[n], self.start[n] + self.lens[n]) for n in range(N)}
        needs.update({ids[N + i]: (0, length) for i, (_, length) in enumerate(groups)})
        width = max([1] + [-(-hi // page) for _, hi in needs.values()]) + extra
        spots = [(s, j) for s, (lo, hi) in needs.items() for j in range(lo // page, -(-hi // page)) if hi > lo]
        pages = list(range(len(spots) + 2))
        r.shuffle(pages)
        self.rows = [[-1] * width for _ in range(slots)]
        for (s, j), i in zip(spots, pages):
            self.rows[s][j] = i
        dt = torch_dtype(dtype)
        self.pool = torch.full((len(spots) + 2, 2, Hk, page, d), math.nan, dtype=dt, device="cuda")
        for s, (lo, hi) in needs.items():
            if hi > lo:
                p, row = self.places(s, lo, hi)
                self.pool[p, :, :, row] = torch.randn(hi - lo, 2, Hk, d, generator=g, device="cuda").to(dt) * loud
        self.T = sum(self.lens)
        self.q = (torch.randn(self.T, Hq, d, generator=g, device="cuda") * loud).to(dt)
        self.cu = [0]
        for n in self.lens:
            self.cu.append(self.cu[-1] + n)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
        self.table, self.slots, self.starts, self.cu_dev = i32(self.rows), i32(self.ids), i32(self.start), i32(self.cu)
        self.prefixes = (i32(cut), i32([n for _, n in groups]), i32(self.kept)) if groups else None

    def places(self, slot, lo, hi):
        """Pages and rows in them of the positions [lo, hi) of a slot."""
        t, page = self.t, self.page
        p = t.arange(lo, hi, device="cuda")
        return t.tensor(self.rows[slot], device="cuda")[p // page], p % page

    def call(self, **over):
        import kda_linear_attention_chunk_gb300 as kda
        args = dict(q=self.q, kv_pages=self.pool, page_table=self.table, starts=self.starts, cu_seqlens=self.cu_dev,
                    slots=self.slots, prefixes=self.prefixes, scale=self.scale)
        args.update(over)
        return kda.paged_attention(**args)

    def keys(self, n):
        """Keys and values [positions][Hk][d] of sequence n, in 64 bits."""
        t = self.t
        p, r = self.places(self.ids[n], self.prefix[n], self.start[n] + self.lens[n])
        kv = self.pool[p, :, :, r]
        if self.prefix[n]:
            p, r = self.places(self.kept[self.group[n]], 0, self.prefix[n])
            kv = t.cat([self.pool[p, :, :, r], kv])
        return kv[:, 0].double(), kv[:, 1].double()

    def want(self, n):
        """Output of sequence n's rows and its bound."""
        k, v = self.keys(n)
        pos = self.t.arange(self.start[n], self.start[n] + self.lens[n], device="cuda")
        return attention64(self.q[self.cu[n]:self.cu[n + 1]].double(), k, v, pos, self.scale, self.dtype)

    def check(self, out, skip=()):
        for n, L in enumerate(self.lens):
            if L and n not in skip:
                ref, bound = self.want(n)
                got = out[self.cu[n]:self.cu[n + 1]].double()
                off = ((got - ref).abs() / bound).max().item()
                assert off <= 1, (n, off)              # NaN fails too


def attention64(q, k, v, pos, scale, dtype, whole=False):
    """whole: the scores are whole numbers that fp32 holds, which leaves no error of theirs."""
    import torch
    u, tiny = BITS[dtype]
    n, Hk, d = k.shape
    G = q.shape[1] // Hk
    out, bound = torch.empty_like(q), torch.empty_like(q)
    hide = torch.arange(n, device=q.device) > pos[:, None]
    for h in range(q.shape[1]):
        kk, vv = k[:, h // G], v[:, h // G]
        s = (scale * (q[:, h] @ kk.T)).masked_fill(hide, -math.inf)
        size = 0.0 if whole else (scale * (q[:, h].abs() @ kk.abs().T)).masked_fill(hide, 0.0).amax(-1, keepdim=True)
        p = torch.softmax(s, -1)
        out[:, h] = p @ vv
        A = p @ vv.abs()
        off = 2 * ((d + 4) * 2.0 ** -23 * size + 2.0 ** -20) + n * 2.0 ** -23 + u
        bound[:, h] = u * out[:, h].abs() + tiny + off * (1 + u) * A
        if dtype == "fp16":
            bound[:, h] += 2.0 ** -25 * (~hide).double() @ vv.abs()
    return out, bound
