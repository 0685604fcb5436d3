"""Decoding several continuations of a prompt over a paged cache, as measured cases: appending normed and rotated keys
and values to pages, attention over the pages with prefixes that groups of sequences share, the selection of a beam
step, and copies of pages between slots.

With ``own`` false, ``run`` computes each operator in its plain form (elementary torch operations in float32, a beam's
candidates in float64, rounded once at the end); with ``own`` true it makes the library's calls.  ``exact`` gives the
same outputs in 64 bits.

A paged cache is one tensor [num_pages][2 (k, v)][Hk][page][d] with a table [num_slots][max_pages]: position p of a
slot lives in row p % page of the page that entry p // page of the slot's table row names.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


def _dev():
    return torch.device("cuda")


# ---------------------------------------------------------------- shapes of a case
def _lens(case):
    """New rows of each sequence: one, or a split of T drawn from the case's own number ``mix`` (0: equal parts)."""
    N, T = case["N"], case["T"]
    if case["single"]:
        return [1] * N
    if case["mix"] == 0:
        cuts = [T * i // N for i in range(N + 1)]
    else:
        r = random.Random(case["mix"])
        cuts = [0] + sorted(r.randint(0, T) for _ in range(N - 1)) + [T]
    return [cuts[i + 1] - cuts[i] for i in range(N)]


def _groups(case):
    """First sequence of each group of those that share a prefix (and the end of the last), and the prefixes' lengths."""
    N, P = case["N"], case.get("P", 0)
    if not P:
        return [], []
    r = random.Random(case["mix"] + 2)
    if case["mix"] == 0:
        cuts = [N * i // P for i in range(P + 1)]
    else:
        cuts = [0] + sorted(r.randint(0, N) for _ in range(P - 1)) + [N]
    lens = [max(1, int(case["prefix"] * (0.5 + 0.5 * r.random()))) for _ in range(P)]
    lens[r.randrange(P)] = case["prefix"]
    return cuts, lens


def _prefix_of(case):
    """The length of each sequence's shared prefix."""
    cuts, lens = _groups(case)
    out = [0] * case["N"]
    for g, n in enumerate(lens):
        for i in range(cuts[g], cuts[g + 1]):
            out[i] = n
    return out


def _starts(case):
    """Positions before each sequence's new rows: its prefix, and of its own ``context`` (mix 0) or up to as many."""
    N, c = case["N"], case["context"]
    r = random.Random(case["mix"] + 1)
    got = [c if case["mix"] == 0 else int(c * r.random() ** 0.5) for _ in range(N)]
    if c:
        got[r.randrange(N)] = c
    return [a + b for a, b in zip(got, _prefix_of(case))]


def _copied(case):
    """Positions of each move of a copy of pages: whole contexts (fork), or a beam's own part."""
    r = random.Random(case["mix"])
    out = []
    for _ in range(case["moves"]):
        lo = r.randint(case["lo"] // 2, case["lo"])
        out.append((lo, lo + r.randint(case["rows"] // 2, case["rows"])))
    return out


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of 64 sequences before its attention: only latency counts
        dict(name="append_step64", op="append", N=64, T=64, single=True, mix=11, context=9000, page=64, Hq=32, Hk=8,
             d=128, rotary=64, layout="interleaved", dtype="bf16"),
        # 16 prompts packed into 8192 rows, q, k and v as slices of one fused projection
        dict(name="append_packed8192", op="append", N=16, T=8192, single=False, mix=7, context=0, page=64, Hq=32, Hk=8,
             d=128, rotary=128, layout="half", dtype="bf16"),
        # one user's decode step in a long chat: latency and the split of one context over the card
        dict(name="attend_one", op="attend", N=1, T=1, single=True, mix=0, context=20000, page=64, Hq=32, Hk=8, d=128,
             dtype="bf16"),
        # the decode step of a full batch of unrelated contexts: bandwidth
        dict(name="attend_64", op="attend", N=64, T=64, single=True, mix=5, context=16384, page=64, Hq=32, Hk=8, d=128,
             dtype="bf16"),
        # a beam-search step: 16 prompts of 8 beams each, every prompt's cache kept once
        dict(name="prefix_beams", op="attend", N=128, T=128, single=True, mix=0, context=150, P=16, prefix=8192, page=64,
             Hq=32, Hk=8, d=128, dtype="bf16"),
        # 64 samples of one very long prompt
        dict(name="prefix_samples64", op="attend", N=64, T=64, single=True, mix=21, context=1000, P=1, prefix=131072,
             page=64, Hq=32, Hk=8, d=128, dtype="bf16"),
        # a chunk of a long prompt over the pages already filled: the largest amount of work
        dict(name="attend_chunk2048", op="attend", N=1, T=2048, single=False, mix=0, context=32768, page=128, Hq=32,
             Hk=8, d=128, dtype="bf16"),
        # drafted tokens, single ones and short prompts of three ragged groups; small heads in groups of five, small pages
        dict(name="attend_odd", op="attend", N=11, T=301, single=False, mix=3, context=1777, P=3, prefix=777, page=16,
             Hq=20, Hk=4, d=64, dtype="fp16"),
        # a beam step of one prompt: latency
        dict(name="beam_one", op="beam", G=1, B=4, V=32000, ended=0.0, dead=0, dtype="fp32"),
        # a beam step of 16 prompts with 8 beams each, some ended: bandwidth
        dict(name="beam_16x8", op="beam", G=16, B=8, V=131072, ended=0.05, dead=1, dtype="bf16"),
        # what the beams of that step own moves to other beams' pages, in the caches of four layers
        dict(name="pages_beams", op="copy", layers=4, slots=128, moves=60, lo=8000, rows=300, page=64, Hk=8, d=128,
             mix=4, dtype="bf16"),
        # whole contexts forked within one layer's cache, odd lengths
        dict(name="pages_fork", op="copy", layers=1, slots=40, moves=13, lo=0, rows=5001, page=16, Hk=5, d=64, mix=6,
             dtype="fp16"),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(hi, max(lo, n))
    return n + 1 if n % 1024 == 0 and n < hi else n


def _heads(rng):
    while True:
        Hk, G = rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 32])
        if Hk * G <= 64:
            return Hk * G, Hk


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "attend", "beam", "beam", "copy"])
    if op == "beam":
        while True:
            case = dict(op=op, G=_log(rng, 1, 64), B=rng.choice([1, 2, 3, 4, 5, 8, 8, 10, 16, 32]), V=_log(rng, 50, 262144),
                        ended=rng.choice([0.0, 0.0, 0.1, 0.5]), dead=rng.choice([0, 0, 1, 100]),
                        dtype=rng.choice(["bf16", "fp16", "fp32", "fp32"]))
            if case["G"] * case["B"] * case["V"] <= 64e6:
                return case
    d, dtype, page = rng.choice([64, 128, 128]), rng.choice(["bf16", "bf16", "fp16"]), rng.choice([16, 32, 64, 64, 128, 256])
    Hq, Hk = _heads(rng)
    mix = rng.randrange(1, 1 << 20)
    if op == "copy":
        while True:
            slots = _log(rng, 4, 256)
            case = dict(op=op, layers=rng.choice([1, 2, 4]), slots=slots, moves=rng.randint(1, slots // 2),
                        lo=rng.choice([0, 100, 5000]), rows=_log(rng, 2, 6000), page=page, Hk=Hk, d=d, mix=mix, dtype=dtype)
            if case["layers"] * slots * (case["rows"] + 2 * page) * Hk * d <= 4e9:
                return case
    single = rng.random() < 0.6
    if op == "append":
        N = _log(rng, 1, 512)
        return dict(op=op, N=N, T=N if single else _log(rng, 1, 16384), single=single, mix=mix,
                    context=_log(rng, 1, 3000) if single or rng.random() < 0.5 else 0, page=page, Hq=Hq, Hk=Hk, d=d,
                    rotary=rng.choice([0, 16, 32, d // 2, d]), layout=rng.choice(["half", "interleaved"]), dtype=dtype)
    while True:
        N = _log(rng, 1, 256)
        case = dict(op=op, N=N, T=N if single else _log(rng, 1, 4096), single=single, mix=mix,
                    context=_log(rng, 1, 65536), page=page, Hq=Hq, Hk=Hk, d=d, dtype=dtype)
        if rng.random() < 0.5:
            case.update(P=rng.randint(1, max(1, N // 2)), prefix=_log(rng, 1, 100000), context=_log(rng, 1, 2000))
        cuts, lens = _groups(case)
        rows, most = max(_lens(case)), max(a - b for a, b in zip(_starts(case), _prefix_of(case)))
        held = sum(_starts(case)) + case["T"] + sum(lens)
        members = max([cuts[g + 1] - cuts[g] for g in range(len(lens))] or [0])
        scores = N * rows * (most + rows) + len(lens) * members * rows * case.get("prefix", 0)
        gathered = (N * (most + rows) + len(lens) * case.get("prefix", 0)) * Hk * d
        if scores * Hq <= 5e9 and gathered <= 3e9 and held * Hk * d <= 2e9 and work(case)["flops"] <= 1.2e12:
            return case


# ---------------------------------------------------------------- inputs
def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    """Normal values in pieces, so that a large cache needs no float32 copy of itself."""
    out = torch.empty(shape, dtype=dtype, device=_dev())
    flat = out.view(-1)
    step = 1 << 27
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device=_dev(), dtype=torch.float32) * scale
    return out


def _table(positions, rotary, base=10000.0, stretch=4.0):
    """cos | sin of every position, fp32 [positions][rotary]: frequencies stretched for a long context."""
    if rotary == 0:
        return None
    f = base ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device=_dev()) / rotary) / stretch
    a = torch.arange(positions, dtype=torch.float64, device=_dev())[:, None] * f[None, :]
    return torch.cat([a.cos(), a.sin()], 1).float()


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device=_dev())


def _pages(r, needs, slots, page, spare=3):
    """A page table: slot s gets pages for its positions [lo, hi), in random order; -1 elsewhere."""
    width = max([1] + [(hi + page - 1) // page for _, hi in needs.values()]) + 1
    spots = [(s, j) for s, (lo, hi) in needs.items() for j in range(lo // page, (hi + page - 1) // page)]
    ids = list(range(len(spots) + spare))
    r.shuffle(ids)
    rows = [[-1] * width for _ in range(slots)]
    for (s, j), i in zip(spots, ids):
        rows[s][j] = i
    return _int(rows), rows, len(spots) + spare


def _prepare_beam(case, s, g, r):
    G, B, V = case["G"], case["B"], case["V"]
    s["logits"] = _randn(g, G * B, V, dtype=DTYPES[case["dtype"]], scale=3.0)
    # cumulated scores of beams some steps in: a few units apart; the last `dead` beams of a prompt without a hypothesis
    scores = -10.0 - 2.0 * torch.rand(G, B, generator=g, device=_dev()).cumsum(1)
    if case["dead"] and B > 1:
        scores[:, max(1, B - case["dead"]):] = -math.inf
    s["scores"] = scores
    s["end"] = V // 7
    s["ended"] = (torch.rand(G, B, generator=g, device=_dev()) < case["ended"]).int()
    ids = list(range(G * B + 5))
    r.shuffle(ids)
    s["slots"] = _int(ids[:G * B]).view(G, B)
    return s


def _prepare_copy(case, s, g, r):
    ids, of_case = list(range(case["slots"])), random.Random(case["mix"] + 1)   # as many pages with any seed
    r.shuffle(ids)
    m, spans = case["moves"], _copied(case)
    dst, rest = ids[:m], ids[m:]
    src = [rest[of_case.randrange(len(rest))] for _ in range(m)]
    needs = {}
    for (lo, hi), a, b in zip(spans, src, dst):
        needs[b] = (lo, hi)
        was = needs.get(a, (lo, hi))
        needs[a] = (min(lo, was[0]), max(hi, was[1]))
    s["table"], s["rows"], n = _pages(r, needs, case["slots"], case["page"])
    s["caches"] = [_randn(g, n, 2, case["Hk"], case["page"], case["d"], dtype=DTYPES[case["dtype"]])
                   for _ in range(case["layers"])]
    for i in range(m):                             # as from a beam step: rows without a copy among the others
        if i % 9 == 8:
            dst[i] = -1
    s["src"], s["dst"] = _int(src), _int(dst)
    s["from"], s["to"] = _int([lo for lo, _ in spans]), _int([hi for _, hi in spans])
    return s


def prepare(case, seed):
    g = torch.Generator(device=_dev())
    g.manual_seed(seed)
    r = random.Random(seed)
    s = {"case": case}
    if case["op"] == "beam":
        return _prepare_beam(case, s, g, r)
    if case["op"] == "copy":
        return _prepare_copy(case, s, g, r)
    dt, N, Hq, Hk, d = DTYPES[case["dtype"]], case["N"], case["Hq"], case["Hk"], case["d"]
    lens, starts = _lens(case), _starts(case)
    cuts, shared = _groups(case)
    before = _prefix_of(case)
    slots = N + len(shared) + 2
    ids = list(range(slots))
    r.shuffle(ids)
    needs = {ids[n]: (before[n], starts[n] + lens[n]) for n in range(N)}
    needs.update({ids[N + p]: (0, n) for p, n in enumerate(shared)})
    s["table"], s["table_host"], pages = _pages(r, needs, slots, case["page"])
    s["pool"] = _randn(g, pages, 2, Hk, case["page"], d, dtype=dt)
    s["slots_host"], s["slots"] = ids[:N], _int(ids[:N])
    s["starts_host"], s["starts"] = starts, _int(starts)
    s["lens"] = lens
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    s["cu"] = None if case["single"] else _int(cu)
    if case["op"] == "append":
        qkv = _randn(g, sum(lens), Hq + 2 * Hk, d, dtype=dt, scale=2.0)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        s["qw"] = 1.0 + _randn(g, d, scale=0.2)
        s["kw"] = 1.0 + _randn(g, d, scale=0.2)
        s["angles"] = _table(max(a + b for a, b in zip(starts, lens)) + 1, case["rotary"])
        return s
    # as after the per-head norm: entries of unit size, so logits of a few units after the scale
    s["q"] = _randn(g, sum(lens), Hq, d, dtype=dt)
    if shared:
        s["groups_host"], s["shared_host"] = cuts, shared
        s["groups"], s["shared"], s["shared_slots"] = _int(cuts), _int(shared), _int(ids[N:N + len(shared)])
        s["shared_slots_host"] = ids[N:N + len(shared)]
    return s


# ---------------------------------------------------------------- the plain forms
def _plain_append(s):
    case = s["case"]
    rd, half, page = case["rotary"], case["rotary"] // 2, case["page"]
    t = torch.arange(s["q"].shape[0], device=s["q"].device)
    if s["cu"] is None:
        n, pos = t, s["starts"].long()
    else:
        n = torch.searchsorted(s["cu"].long(), t, right=True) - 1
        pos = s["starts"].long()[n] + t - s["cu"].long()[n]

    def one(x, w):
        y = x.float()
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w
        if rd:
            row = s["angles"][pos]
            cos, sin = row[:, None, :half], row[:, None, half:]
            p = y[..., :rd]
            if case["layout"] == "half":
                a, b = p[..., :half], p[..., half:]
                p = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
            else:
                a, b = p[..., 0::2], p[..., 1::2]
                p = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
            y = torch.cat([p, y[..., rd:]], -1)
        return y.to(x.dtype)

    where = s["table"].long()[s["slots"].long()[n], pos // page]
    s["pool"][where, 0, :, pos % page] = one(s["k"], s["kw"])
    s["pool"][where, 1, :, pos % page] = s["v"]
    return one(s["q"], s["qw"]), s["pool"]


def _keys(s, slots, pos):
    """Keys and values [A][K][Hk][d], in float32, of the positions pos [A][K] of slots [A]; anything past the table."""
    page = s["case"]["page"]
    ids = s["table"].long()[slots[:, None], (pos // page).clamp_max(s["table"].shape[1] - 1)].clamp_min(0)
    return s["pool"][ids, 0, :, pos % page].float(), s["pool"][ids, 1, :, pos % page].float()


def _part(q, k, v, mask, scale):
    """q [A, Q, Hk, G, d], k and v [A, K, Hk, d], mask [A, Q, K]: maxima, sums and sums of values of a part of the keys."""
    z = torch.einsum("aqhgd,akhd->ahgqk", q, k) * scale
    z = z.masked_fill(~mask[:, None, None], float("-inf"))
    m = z.amax(-1, keepdim=True)
    e = (z - m).exp().masked_fill(~mask[:, None, None], 0.0)
    o = torch.einsum("ahgqk,akhd->aqhgd", e, v)
    return m.permute(0, 3, 1, 2, 4), e.sum(-1, keepdim=True).permute(0, 3, 1, 2, 4), o


def _plain_attend(s):
    case = s["case"]
    N, Hq, Hk, d = case["N"], case["Hq"], case["Hk"], case["d"]
    dev, G, scale = s["q"].device, Hq // Hk, d ** -0.5
    cu = torch.arange(N + 1, device=dev) if s["cu"] is None else s["cu"].long()
    lens, starts, Q = cu.diff(), s["starts"].long(), max(s["lens"])
    off = torch.arange(Q, device=dev)
    live = off < lens[:, None]                                   # [N, Q]
    row = torch.where(live, cu[:-1, None] + off, 0)
    q = s["q"].float()[row].view(N, Q, Hk, G, d)
    before = torch.zeros_like(starts)
    if "groups" in s:
        groups, shared = s["groups"].long(), s["shared"].long()
        mine = torch.repeat_interleave(torch.arange(case["P"], device=dev), groups.diff())    # every sequence has a group
        before = shared[mine]
    most = max(a - b + n for a, b, n in zip(s["starts_host"], _prefix_of(case), s["lens"]))
    pos = before[:, None] + torch.arange(most, device=dev)
    k, v = _keys(s, s["slots"].long(), pos)
    mask = pos[:, None, :] <= (starts[:, None] + off)[:, :, None]
    m, l, o = _part(q, k, v, mask, scale)
    if "groups" in s:
        del k, v, mask
        width = max(b - a for a, b in zip(s["groups_host"], s["groups_host"][1:]))
        member = groups[:-1, None] + torch.arange(width, device=dev)
        inside = member < groups[1:, None]
        member = torch.where(inside, member, 0)
        pos = torch.arange(case["prefix"], device=dev).expand(case["P"], -1)
        k, v = _keys(s, s["shared_slots"].long(), pos)
        mask = (pos < shared[:, None])[:, None, :].expand(-1, width * Q, -1)
        m2, l2, o2 = _part(q[member].flatten(1, 2), k, v, mask, scale)
        at = torch.arange(N, device=dev) - groups[mine]
        m2, l2, o2 = (x.view(case["P"], width, Q, *x.shape[2:])[mine, at] for x in (m2, l2, o2))
        top = torch.maximum(m, m2)
        a, b = (m - top).exp(), (m2 - top).exp()
        l, o = l * a + l2 * b, o * a + o2 * b
    out = torch.empty(s["q"].shape[0], Hq, d, dtype=s["q"].dtype, device=dev)
    out[row[live]] = (o / l).reshape(N, Q, Hq, d)[live].to(s["q"].dtype)
    return out


def _plain_beam(s):
    case = s["case"]
    G, B, V = case["G"], case["B"], case["V"]
    dev = s["logits"].device
    x = s["logits"].view(G, B, V).double()                       # candidates of different beams lie close together
    x = x - torch.logsumexp(x, -1, keepdim=True)
    total = s["scores"].double()[..., None] + x
    token = torch.arange(V, device=dev)
    stays = torch.where(token == s["end"], s["scores"].double()[..., None], -math.inf)
    total = torch.where(s["ended"].bool()[..., None], stays, total).view(G, B * V)
    best, at = torch.sort(total, descending=True, stable=True)
    best, at = best[:, :B], at[:, :B]
    if B * V < B:
        raise ValueError("fewer candidates than beams")
    found = best > -math.inf
    parent, token = torch.where(found, at // V, -1), torch.where(found, at % V, -1)
    safe = parent.clamp_min(0)
    ended = found & (s["ended"].bool().gather(1, safe) | (token == s["end"]))
    # a parent's first child keeps its slot; the others take those of the beams without a child
    same = (parent[:, :, None] == parent[:, None, :]) & found[:, :, None]
    again = same.tril(-1).any(-1) | ~found
    beams = torch.arange(B, device=dev)
    childless = ~((parent[:, :, None] == beams) & found[:, :, None]).any(1)
    free = torch.sort(torch.where(childless, beams, B), -1).values            # childless beams first, ascending
    nth = (again.long().cumsum(-1) - 1).clamp_min(0)
    slots = s["slots"].long()
    new = torch.where(again, slots.gather(1, free.gather(1, nth).clamp_max(B - 1)), slots.gather(1, safe))
    src = torch.where(found, slots.gather(1, safe), -1)
    dst = torch.where(again & found, new, -1)
    return (best.float(), parent.int(), token.int(), ended.int(), new.int(), src.int(), dst.int())


def _plain_copy(s):
    page, table = s["case"]["page"], s["table"].long()
    longest = s["case"]["rows"]
    pos = s["from"].long()[:, None] + torch.arange(longest, device=table.device)
    live = (pos < s["to"].long()[:, None]) & (s["dst"] >= 0)[:, None]
    column = (pos // page).clamp_max(table.shape[1] - 1)
    a = table[s["src"].long()[:, None], column][live]
    b = table[s["dst"].long().clamp_min(0)[:, None], column][live]
    r = (pos % page)[live]
    everything = torch.stack(s["caches"])
    everything[:, b, :, :, r] = everything[:, a, :, :, r]
    return list(everything.unbind(0))


def _own(s):
    import kda_linear_attention_chunk_gb300 as kda

    case = s["case"]
    op = case["op"]
    if op == "append":
        q = kda.paged_append(s["q"], s["k"], s["v"], s["pool"], s["table"], s["starts"], cu_seqlens=s["cu"],
                             slots=s["slots"], q_weight=s["qw"], k_weight=s["kw"], table=s["angles"],
                             layout=case["layout"], eps=EPS)
        return q, s["pool"]
    if op == "attend":
        shared = (s["groups"], s["shared"], s["shared_slots"]) if "groups" in s else None
        return kda.paged_attention(s["q"], s["pool"], s["table"], s["starts"], cu_seqlens=s["cu"], slots=s["slots"],
                                   prefixes=shared)
    if op == "beam":
        return kda.beam_select(s["logits"], s["scores"], ended=s["ended"], end_token=s["end"], slots=s["slots"])
    kda.pages_copy(s["caches"], s["table"], s["src"], s["dst"], s["to"], start=s["from"])
    return list(s["caches"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return {"append": _plain_append, "attend": _plain_attend, "beam": _plain_beam, "copy": _plain_copy}[op](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "beam":
        live = case["B"] - min(case["dead"], case["B"] - 1)
        rows = case["G"] * live * (1.0 - case["ended"])          # nothing of the others' logits is needed
        return {"bytes": rows * case["V"] * (4 if case["dtype"] == "fp32" else 2) + case["G"] * case["B"] * 36,
                "flops": 4 * rows * case["V"]}
    if op == "copy":
        rows = sum(hi - lo for i, (lo, hi) in enumerate(_copied(case)) if i % 9 != 8)
        return {"bytes": 2 * case["layers"] * rows * 2 * case["Hk"] * case["d"] * 2, "flops": 0}
    Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
    lens, starts = _lens(case), _starts(case)
    T = sum(lens)
    if op == "append":
        return {"bytes": T * ((Hq + 2 * Hk) * d * 2 * 2 + case["rotary"] * 4) + 8 * d,
                "flops": T * (Hq + Hk) * (4 * d + 3 * case["rotary"])}
    pairs = sum(n * a + n * (n + 1) // 2 for a, n in zip(starts, lens))
    held = sum(_groups(case)[1]) + sum(a - b + n for a, b, n in zip(starts, _prefix_of(case), lens) if n)
    return {"bytes": 2 * T * Hq * d * 2 + held * Hk * 2 * d * 2, "flops": 4 * d * Hq * pairs}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, page = case["op"], case.get("page")

    def spots(row, lo, hi):
        """Pages and rows in them of the positions [lo, hi) of a table row."""
        return (torch.tensor([row[p // page] for p in range(lo, hi)], device=_dev()),
                torch.tensor([p % page for p in range(lo, hi)], device=_dev()))

    def append():
        pos = torch.tensor([a + i for a, n in zip(s["starts_host"], s["lens"]) for i in range(n)], device=_dev())
        rd, outs = case["rotary"], []
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            y = x.double()
            y = y / (y.pow(2).sum(-1, keepdim=True) / case["d"] + EPS).sqrt() * w.double()
            if rd:
                angle = s["angles"].double()[pos]
                c, n = angle[:, :rd // 2].unsqueeze(1), angle[:, rd // 2:].unsqueeze(1)
                if case["layout"] == "half":
                    i = torch.arange(rd // 2, device=y.device)
                    j = i + rd // 2
                else:
                    i = torch.arange(0, rd, 2, device=y.device)
                    j = i + 1
                a, b = y[..., i].clone(), y[..., j].clone()
                y[..., i] = a * c - b * n
                y[..., j] = a * n + b * c
            outs.append(y)
        pool, t = s["pool"].double(), 0
        for slot, a, n in zip(s["slots_host"], s["starts_host"], s["lens"]):
            if n:
                ids, rows = spots(s["table_host"][slot], a, a + n)
                pool[ids, 0, :, rows] = outs[1][t:t + n]
                pool[ids, 1, :, rows] = s["v"][t:t + n].double()
            t += n
        return outs[0], pool

    def attend():
        """Each sequence by itself: all its keys laid out by position, then blocks of its rows."""
        Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
        out, t = torch.zeros(sum(s["lens"]), Hq, d, dtype=torch.float64, device=_dev()), 0
        before = _prefix_of(case)
        kept = (None, None, None)
        for n, L in enumerate(s["lens"]):
            if not L:
                continue
            a = s["starts_host"][n]
            ids, rows = spots(s["table_host"][s["slots_host"][n]], before[n], a + L)
            k, v = s["pool"][ids, 0, :, rows], s["pool"][ids, 1, :, rows]
            if before[n]:
                g = max(i for i, c in enumerate(s["groups_host"][:-1]) if c <= n)
                if kept[0] != g:
                    ids, rows = spots(s["table_host"][s["shared_slots_host"][g]], 0, before[n])
                    kept = (g, s["pool"][ids, 0, :, rows], s["pool"][ids, 1, :, rows])
                k, v = torch.cat([kept[1], k]), torch.cat([kept[2], v])
            for lo in range(0, L, 256):
                hi = min(L, lo + 256)
                see = a + hi
                hide = torch.arange(see, device=_dev()) > torch.arange(a + lo, a + hi, device=_dev())[:, None]
                for h in range(Hk):
                    q = s["q"][t + lo:t + hi, h * (Hq // Hk):(h + 1) * (Hq // Hk)].double().transpose(0, 1)
                    z = q @ k[:see, h].double().T / math.sqrt(d)
                    p = torch.softmax(z.masked_fill(hide, -math.inf), -1)
                    out[t + lo:t + hi, h * (Hq // Hk):(h + 1) * (Hq // Hk)] = (p @ v[:see, h].double()).transpose(0, 1)
            t += L
        return out

    def beam():
        G, B, V = case["G"], case["B"], case["V"]
        best = torch.full((G, B), -math.inf, dtype=torch.float64, device=_dev())
        for g in range(G):
            every = []
            for b in range(B):
                score = float(s["scores"][g, b])
                if score == -math.inf:
                    continue
                if int(s["ended"][g, b]):
                    every.append(torch.tensor([score], dtype=torch.float64, device=_dev()))
                    continue
                x = s["logits"][g * B + b].double()
                p = torch.exp(x - x.max())
                every.append(score + torch.log(p / p.sum()))
            if every:
                top = torch.topk(torch.cat(every), min(B, sum(e.numel() for e in every))).values
                best[g, :top.numel()] = top
        return best, None, None, None, None, None, None

    def copy():
        caches = [c.double() for c in s["caches"]]
        for a, b, lo, hi in zip(s["src"].tolist(), s["dst"].tolist(), s["from"].tolist(), s["to"].tolist()):
            if b < 0:
                continue
            ia, r = spots(s["rows"][a], lo, hi)
            ib, _ = spots(s["rows"][b], lo, hi)
            for c, was in zip(caches, s["caches"]):
                c[ib, :, :, r] = was[ia, :, :, r].double()
        return caches

    return {"append": append, "attend": attend, "beam": beam, "copy": copy}[op]()
