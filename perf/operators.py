"""The softmax-attention side of a hybrid stack, as measured cases: per-head norm and rotation of q and k,
attention over a sliding window with sinks (packed prefill and decode on slot-addressed ring caches), and moves of
slot entries (fork, clear, compact).

With ``own`` false, ``run`` computes each operator in its plain form (elementary torch operations in float32, rounded
once at the end); with ``own`` true it makes the library's calls.  ``exact`` gives the same outputs in 64 bits.

A ring cache is one tensor [num_slots][2 (k, v)][Hk][rows][d]: position p of a sequence lives in row p while
p < sinks, and in row sinks + (p - sinks) % (rows - sinks) otherwise.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
QBLOCK = 128           # queries per block of the plain prefill
EPS = 1e-6


def _dev():
    return torch.device("cuda")


# ---------------------------------------------------------------- shapes of a case
def _lens(case):
    """Rows of each sequence of a prefill: a split of T drawn from the case's own number ``mix`` (0: equal parts)."""
    N, T = case["N"], case["T"]
    if case["mix"] == 0:
        cuts = [T * i // N for i in range(N + 1)]
    else:
        r = random.Random(case["mix"])
        cuts = [0] + sorted(r.randint(0, T) for _ in range(N - 1)) + [T]
    return [cuts[i + 1] - cuts[i] for i in range(N)]


def _starts(case):
    """Positions already in each sequence's cache: ``context`` for all (mix 0) or spread over [0, context]."""
    N, c = case["N"], case["context"]
    if case["mix"] == 0 or c == 0:
        return [c] * N
    r = random.Random(case["mix"] + 1)
    got = [int(c * r.random() ** 0.5) for _ in range(N)]
    got[r.randrange(N)] = c
    return got


def _visible(case, lo, hi):
    """Keys that the positions lo .. hi-1 see, summed (window of W, and the first S)."""
    W, S = case["window"], case["sinks"]

    def upto(p):                                   # sum over positions 0 .. p-1
        near = p * (p + 1) // 2 if p <= W else W * (W + 1) // 2 + (p - W) * W
        out = max(0, p - W)                        # positions with something behind the window: 1, 2, ... tokens
        far = out * (out + 1) // 2 if out <= S else S * (S + 1) // 2 + (out - S) * S
        return near + far

    return upto(hi) - upto(lo)


def _reach(case, start, n):
    """Distinct cached positions (< start) that n new rows from ``start`` on read."""
    if n == 0:
        return 0
    lo = max(0, start - case["window"] + 1)
    return start - lo + min(case["sinks"], lo)


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of 64 sequences before its attention: only latency counts
        dict(name="rope_step64", op="rope", T=64, Hq=32, Hk=8, d=128, rotary=64, layout="interleaved", dtype="bf16",
             fused=True, context=262144),
        # the packed 8192-row prefill of 16 sequences, q and k as slices of one fused projection
        dict(name="rope_packed8192", op="rope", T=8192, Hq=32, Hk=8, d=128, rotary=128, layout="half", dtype="bf16",
             fused=True, context=262144),
        # 16 fresh prompts packed into 8192 rows
        dict(name="prefill_packed16", op="prefill", N=16, T=8192, mix=7, context=0, Hq=32, Hk=8, d=128, window=1024,
             sinks=4, dtype="bf16", cached=True),
        # one 8192-row chunk in the middle of a 262,144-row context
        dict(name="prefill_chunk8192", op="prefill", N=1, T=8192, mix=0, context=131072, Hq=32, Hk=8, d=128,
             window=4096, sinks=4, dtype="bf16", cached=True),
        # a long document at once, nothing cached: the largest amount of work
        dict(name="prefill_long32768", op="prefill", N=1, T=32768, mix=0, context=0, Hq=32, Hk=8, d=128, window=4096,
             sinks=0, dtype="bf16", cached=False),
        # the verification of 8 drafted tokens for each of 64 sequences
        dict(name="prefill_verify64x8", op="prefill", N=64, T=512, mix=0, context=5000, Hq=32, Hk=8, d=128,
             window=1024, sinks=4, dtype="bf16", cached=True),
        # ragged prompts, a small window, small heads in groups of five
        dict(name="prefill_odd", op="prefill", N=11, T=4099, mix=3, context=777, Hq=20, Hk=4, d=64, window=100,
             sinks=3, dtype="fp16", cached=True),
        # one user's decode step: latency
        dict(name="decode_one", op="decode", N=1, mix=0, context=20000, Hq=32, Hk=8, d=128, window=1024, sinks=4,
             dtype="bf16"),
        # the decode step of a full batch over a long window: bandwidth
        dict(name="decode_64", op="decode", N=64, mix=5, context=262144, Hq=32, Hk=8, d=128, window=4096, sinks=4,
             dtype="bf16"),
        # a ragged batch with groups of seven small heads, some sequences shorter than the window
        dict(name="decode_odd", op="decode", N=37, mix=9, context=1500, Hq=14, Hk=2, d=64, window=500, sinks=3,
             dtype="fp16"),
        # parallel sampling: prompts' slots forked to 16 others in the pools of two layer pairs, some slots cleared
        dict(name="slots_fork", op="fork", layers=2, H=32, Hk=8, rows=1028, slots=64, moves=18, dtype="bf16"),
        # the batch shrank: the live slots move to the front of the pools
        dict(name="slots_compact", op="compact", layers=1, H=32, Hk=8, rows=516, slots=64, moves=33, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(hi, max(lo, n))
    return n + 1 if n % 1024 == 0 else n           # odd sizes rather than round ones


def _heads(rng, d):
    while True:
        Hk, G = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
        if Hk * G <= 64 and all(h * d % 1024 or h * d // 1024 != 3 for h in (Hk, Hk * G, Hk * (G + 2))):
            return Hk * G, Hk


def draw(rng):
    op = rng.choice(["rope", "prefill", "prefill", "prefill", "decode", "decode", "fork", "compact"])
    d, dtype = rng.choice([64, 128, 128]), rng.choice(["bf16", "bf16", "fp16"])
    Hq, Hk = _heads(rng, d)
    if op == "rope":
        return dict(op=op, T=_log(rng, 1, 16384), Hq=Hq, Hk=Hk, d=d, rotary=rng.choice([0, 16, 32, d // 2, d]),
                    layout=rng.choice(["half", "interleaved"]), dtype=dtype, fused=rng.random() < 0.7,
                    context=_log(rng, 64, 300000))
    if op == "prefill":
        while True:
            T = _log(rng, 1, 16384)
            case = dict(op=op, N=min(_log(rng, 1, 64), T + 2), T=T, mix=rng.randrange(1, 1 << 20),
                        context=_log(rng, 1, 200000) if rng.random() < 0.6 else 0, Hq=Hq, Hk=Hk, d=d,
                        window=_log(rng, 16, 8191), sinks=rng.choice([0, 0, 1, 4, 5, 64, 130]), dtype=dtype)
            case["cached"] = case["context"] > 0 or rng.random() < 0.5
            cols = case["sinks"] + min(case["window"] + QBLOCK, case["context"] + T)
            if (T + case["N"] * QBLOCK) * cols * Hq <= 5e9 and work(case)["flops"] <= 2e12:
                return case
    if op == "decode":
        while True:
            case = dict(op=op, N=_log(rng, 1, 256), mix=rng.randrange(1, 1 << 20), context=_log(rng, 1, 300000),
                        Hq=Hq, Hk=Hk, d=d, window=_log(rng, 16, 16383), sinks=rng.choice([0, 0, 1, 4, 5, 64, 130]),
                        dtype=dtype)
            if case["N"] * (case["window"] + case["sinks"]) * Hk * d <= 300e6:
                return case
    slots = _log(rng, 4, 80)
    moves = rng.randint(1, slots // 2 if op == "fork" else slots)
    return dict(op=op, layers=rng.choice([1, 2]), H=rng.choice([8, 16, 32]), Hk=rng.choice([1, 2, 8]),
                rows=_log(rng, 16, 1028), slots=slots, moves=moves, dtype=dtype)


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


def _ring_rows(case):
    return case["sinks"] + case["window"]


def prepare(case, seed):
    g = torch.Generator(device=_dev())
    g.manual_seed(seed)
    r = random.Random(seed)
    s = {"case": case}
    dt = DTYPES[case["dtype"]]
    op = case["op"]
    if op in ("fork", "compact"):
        n, pools = case["slots"], []
        for _ in range(case["layers"]):            # a layer pair: linear-attention state, conv window, ring cache
            pools.append(_randn(g, n, case["H"], 128, 128, scale=0.3))
            pools.append(_randn(g, n, 3, 3, case["H"] * 128, dtype=torch.bfloat16))
            pools.append(_randn(g, n, 2, case["Hk"], case["rows"], 128, dtype=dt))
        s["pools"] = pools
        ids = list(range(n))
        r.shuffle(ids)
        if op == "fork":                           # few sources, many targets; some entries cleared, some rows padded
            m = case["moves"]
            dst, rest = ids[:m], ids[m:]
            src = [rest[r.randrange(max(1, min(4, len(rest))))] for _ in range(m)]
            for i in range(m):
                if i % 9 == 4:
                    src[i] = -1
                if i % 9 == 8:
                    dst[i] = -1
            s["src"], s["dst"] = _int(src), _int(dst)
        else:                                      # a table of live slots in any order, with padded rows
            table = ids[:case["moves"]]
            for i in range(len(table) // 8):
                table.insert(r.randrange(len(table) + 1), -1)
            s["slots"] = _int(table)
        return s
    Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
    if op == "rope":
        T = case["T"]
        if case["fused"]:
            qkv = _randn(g, T, Hq + 2 * Hk, d, dtype=dt, scale=2.0)
            s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        else:
            s["q"], s["k"] = _randn(g, T, Hq, d, dtype=dt, scale=2.0), _randn(g, T, Hk, d, dtype=dt, scale=2.0)
        s["qw"] = 1.0 + _randn(g, d, scale=0.2)
        s["kw"] = 1.0 + _randn(g, d, scale=0.2)
        s["table"] = _table(case["context"], case["rotary"])
        base = torch.randint(0, case["context"], (T,), generator=g, device=_dev(), dtype=torch.int32)
        run_ = torch.arange(T, device=_dev(), dtype=torch.int32)
        s["pos"] = ((base[run_ // 512] + run_) % case["context"]).to(torch.int32) if T >= 512 else base
        return s
    rows = case["T"] if op == "prefill" else case["N"]
    # as after the per-head norm: entries of unit size, so logits of a few units after the scale
    qkv = _randn(g, rows, Hq + 2 * Hk, d, dtype=dt)
    s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    N = case["N"]
    s["starts_host"] = _starts(case)
    s["starts"] = _int(s["starts_host"])
    if op == "decode" or case["cached"]:
        entries = N + 2
        s["pool"] = _randn(g, entries, 2, Hk, _ring_rows(case), d, dtype=dt)
        ids = list(range(entries))
        r.shuffle(ids)
        s["slots_host"] = ids[:N]
        s["slots"] = _int(ids[:N])
    if op == "prefill":
        s["lens"] = _lens(case)
        cu = [0]
        for n in s["lens"]:
            cu.append(cu[-1] + n)
        s["cu"] = _int(cu)
    return s


# ---------------------------------------------------------------- the plain forms
def _plain_rope(s):
    case = s["case"]
    rd, half = case["rotary"], case["rotary"] // 2

    def one(x, w):
        y = x.float()
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w
        if rd:
            row = s["table"][s["pos"].long()]
            cos, sin = row[:, None, :half], row[:, None, half:]
            r = y[..., :rd]
            if case["layout"] == "half":
                a, b = r[..., :half], r[..., half:]
                r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
            else:
                a, b = r[..., 0::2], r[..., 1::2]
                r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
            y = torch.cat([r, y[..., rd:]], -1)
        return y.to(x.dtype)

    return one(s["q"], s["qw"]), one(s["k"], s["kw"])


def _row_of(p, case):
    """The cache row of positions p."""
    S = case["sinks"]
    return torch.where(p < S, p, S + (p - S) % case["window"])


def _attend(q, k, v, mask, scale):
    """q [B, Q, Hk, G, d], k and v [B, K, Hk, d], mask [B, Q, K]: softmax attention in float32."""
    z = torch.einsum("bqhgd,bkhd->bhgqk", q, k) * scale
    z = z.masked_fill(~mask[:, None, None], float("-inf"))
    z = z - z.amax(-1, keepdim=True)
    e = z.exp()
    o = torch.einsum("bhgqk,bkhd->bqhgd", e, v)
    return o / e.sum(-1).permute(0, 3, 1, 2)[..., None]


def _plain_prefill(s):
    case = s["case"]
    T, Hq, Hk, d, W, S = (case[x] for x in ("T", "Hq", "Hk", "d", "window", "sinks"))
    dev, G = s["q"].device, Hq // Hk
    lens, starts = s["cu"].long().diff(), s["starts"].long()
    blocks = (lens + QBLOCK - 1) // QBLOCK                       # query blocks of each sequence
    seq = torch.repeat_interleave(torch.arange(case["N"], device=dev), blocks)
    first = blocks.cumsum(0) - blocks
    at = (torch.arange(seq.numel(), device=dev) - first[seq]) * QBLOCK
    off = torch.arange(QBLOCK, device=dev)
    live = at[:, None] + off < lens[seq][:, None]                # [B, Q]
    row = torch.where(live, s["cu"].long()[seq][:, None] + at[:, None] + off, 0)
    qpos = starts[seq][:, None] + at[:, None] + off
    near = min(W - 1, max(a + b for a, b in zip(s["starts_host"], s["lens"]))) + QBLOCK
    lo = (starts[seq] + at + QBLOCK - near).clamp_min(0)         # first position of the block's window columns
    kpos = torch.cat([torch.arange(S, device=dev).expand(seq.numel(), S),
                      lo[:, None] + torch.arange(near, device=dev)], 1)
    sink = torch.arange(S + near, device=dev) < S
    end = (starts + lens)[seq][:, None]
    fresh = kpos >= starts[seq][:, None]
    new = (s["cu"].long()[seq][:, None] + kpos - starts[seq][:, None]).clamp(0, max(T - 1, 0))
    k, v = s["k"].float()[new], s["v"].float()[new]              # [B, K, Hk, d]
    if case["cached"]:
        ent, old = s["slots"].long()[seq][:, None], _row_of(kpos, case)
        k = torch.where(fresh[..., None, None], k, s["pool"][ent, 0, :, old].float())
        v = torch.where(fresh[..., None, None], v, s["pool"][ent, 1, :, old].float())
    q, kp = qpos[:, :, None], kpos[:, None, :]
    inside = torch.where(sink, kp <= q - W, (kp <= q) & (kp > q - W))
    mask = inside & (kp < end[:, :, None]) | ~live[:, :, None]   # rows past the end see anything: they are dropped
    o = _attend(s["q"].float()[row].view(seq.numel(), QBLOCK, Hk, G, d), k, v, mask, d ** -0.5)
    out = torch.zeros(T, Hq, d, dtype=s["q"].dtype, device=dev)
    out[row[live]] = o.reshape(seq.numel(), QBLOCK, Hq, d)[live].to(s["q"].dtype)
    if not case["cached"]:
        return out
    t = torch.arange(T, device=dev)
    n = torch.searchsorted(s["cu"].long(), t, right=True) - 1
    p = starts[n] + t - s["cu"].long()[n]
    kept = (p < S) | (p >= (starts + lens)[n] - W)               # a later row of the call takes the others' places
    s["pool"][s["slots"].long()[n][kept], 0, :, _row_of(p, case)[kept]] = s["k"][kept]
    s["pool"][s["slots"].long()[n][kept], 1, :, _row_of(p, case)[kept]] = s["v"][kept]
    return out, s["pool"]


def _plain_decode(s):
    case = s["case"]
    N, Hq, Hk, d, W, S = (case[x] for x in ("N", "Hq", "Hk", "d", "window", "sinks"))
    dev, pos, ent = s["q"].device, s["starts"].long(), s["slots"].long()
    s["pool"][ent, 0, :, _row_of(pos, case)] = s["k"]
    s["pool"][ent, 1, :, _row_of(pos, case)] = s["v"]
    near = min(W, max(s["starts_host"]) + 1)
    lo = (pos - near + 1).clamp_min(0)
    kpos = torch.cat([torch.arange(S, device=dev).expand(N, S), lo[:, None] + torch.arange(near, device=dev)], 1)
    sink = torch.arange(S + near, device=dev) < S
    k = s["pool"][ent[:, None], 0, :, _row_of(kpos, case)].float()
    v = s["pool"][ent[:, None], 1, :, _row_of(kpos, case)].float()
    q, kp = pos[:, None, None], kpos[:, None, :]
    mask = torch.where(sink, kp <= q - W, (kp <= q) & (kp > q - W))
    o = _attend(s["q"].float().reshape(N, 1, Hk, Hq // Hk, d), k, v, mask, d ** -0.5)
    return o.reshape(N, Hq, d).to(s["q"].dtype), s["pool"]


def _plain_fork(s):
    src, dst = s["src"].long(), s["dst"].long()
    keep = dst >= 0
    src, dst = src[keep], dst[keep]
    for pool in s["pools"]:
        rows = pool[src.clamp_min(0)]
        rows[src < 0] = 0
        pool[dst] = rows
    return list(s["pools"])


def _plain_compact(s):
    table = s["slots"].long()
    live = table >= 0
    count = live.sum()
    n = s["case"]["slots"]
    used = torch.zeros(n, dtype=torch.bool, device=table.device)
    used[table[live]] = True
    ids = torch.arange(n, device=table.device)
    free, high = ids[~used & (ids < count)], ids[used & (ids >= count)]
    to = ids.clone()
    to[high] = free                                              # the k-th high slot takes the k-th free one
    for pool in s["pools"]:
        pool[free] = pool[high]
    table = torch.where(live, to[table.clamp_min(0)], table).int()
    return [table] + [p[:s["case"]["moves"]] for p in s["pools"]]


def _own(s):
    import kda_linear_attention_chunk_gb300 as kda

    case = s["case"]
    op = case["op"]
    if op == "rope":
        return kda.head_norm_rope(s["q"], s["k"], q_weight=s["qw"], k_weight=s["kw"], positions=s["pos"],
                                  table=s["table"], layout=case["layout"], eps=EPS)
    if op == "prefill":
        if not case["cached"]:
            return kda.window_prefill(s["q"], s["k"], s["v"], s["cu"], case["window"], sinks=case["sinks"])
        out = kda.window_prefill(s["q"], s["k"], s["v"], s["cu"], case["window"], sinks=case["sinks"],
                                 kv_pool=s["pool"], slots=s["slots"], starts=s["starts"])
        return out, s["pool"]
    if op == "decode":
        out = kda.window_decode(s["q"], s["k"], s["v"], s["starts"], s["pool"], case["window"],
                                sinks=case["sinks"], slots=s["slots"])
        return out, s["pool"]
    if op == "fork":
        kda.slots_copy(s["pools"], s["src"], s["dst"])
        return list(s["pools"])
    table, count = kda.slots_compact(s["pools"], s["slots"]), case["moves"]
    return [table] + [p[:count] for p in s["pools"]]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return {"rope": _plain_rope, "prefill": _plain_prefill, "decode": _plain_decode, "fork": _plain_fork,
            "compact": _plain_compact}[op](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("fork", "compact"):
        entry = case["layers"] * (case["H"] * 128 * 128 * 4 + case["H"] * 128 * 9 * 2
                                  + 2 * case["Hk"] * case["rows"] * 128 * 2)
        n, m = case["slots"], case["moves"]
        if op == "fork":                           # at most four sources read once, every target written
            skip, clear = sum(i % 9 == 8 for i in range(m)), sum(i % 9 == 4 for i in range(m))
            return {"bytes": entry * (m - skip + min(4, m - skip - clear)), "flops": 0}
        high = m * (n - m) / n                     # of m live slots anywhere, so many lie past the first m
        return {"bytes": max(8 * m, 2 * entry * high), "flops": 0}
    Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
    if op == "rope":
        T = case["T"]
        return {"bytes": T * ((Hq + Hk) * d * 2 * 2 + case["rotary"] * 4 + 4) + 8 * d,
                "flops": T * (Hq + Hk) * (4 * d + 3 * case["rotary"])}
    starts = _starts(case)
    lens = _lens(case) if op == "prefill" else [1] * case["N"]
    pairs = sum(_visible(case, a, a + n) for a, n in zip(starts, lens))
    rows = sum(lens)
    moved = rows * (2 * Hq + 2 * Hk) * d * 2
    if op == "decode" or case["cached"]:
        old = sum(_reach(case, a, n) for a, n in zip(starts, lens))
        kept = sum(min(n, case["window"] + max(0, min(case["sinks"], a + n - case["window"]) - a))
                   for a, n in zip(starts, lens))
        moved += (old + kept) * Hk * 2 * d * 2
    return {"bytes": moved, "flops": 4 * d * Hq * pairs}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    def rope(s):
        case, outs = s["case"], []
        rd = case["rotary"]
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            y = x.double()
            y = y / (y.pow(2).sum(-1, keepdim=True) / case["d"] + EPS).sqrt() * w.double()
            if rd:
                angle = s["table"].double()[s["pos"].long()]
                c = angle[:, :rd // 2].unsqueeze(1)
                n = angle[:, rd // 2:].unsqueeze(1)
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
        return tuple(outs)

    def place(p, case):
        return p if p < case["sinks"] else case["sinks"] + (p - case["sinks"]) % case["window"]

    def attention(s):
        """Each sequence by itself: its keys laid out by position, then blocks of queries against what they see."""
        case = s["case"]
        Hq, Hk, d, W, S = (case[x] for x in ("Hq", "Hk", "d", "window", "sinks"))
        decode = case["op"] == "decode"
        lens = [1] * case["N"] if decode else s["lens"]
        dev = s["q"].device
        out = torch.zeros(sum(lens), Hq, d, dtype=torch.float64, device=dev)
        pool = s["pool"].double() if "pool" in s else None
        row = 0
        for n, L in enumerate(lens):
            if L == 0:
                continue
            a = s["starts_host"][n]
            base = max(0, a - W + 1)                   # oldest cached position in any window
            old = list(range(min(S, base))) + list(range(base, a))
            pos = torch.tensor(old + list(range(a, a + L)), device=dev)
            k, v = s["k"][row:row + L].double(), s["v"][row:row + L].double()
            if old:
                places = torch.tensor([place(p, case) for p in old], device=dev)
                e = s["slots_host"][n]
                k = torch.cat([s["pool"][e, 0][:, places].transpose(0, 1).double(), k])
                v = torch.cat([s["pool"][e, 1][:, places].transpose(0, 1).double(), v])
            step = 1024
            for b in range(0, L, step):
                m = min(step, L - b)
                qp = torch.arange(a + b, a + b + m, device=dev)
                want = (pos <= a + b + m - 1) & ((pos > a + b - W) | (pos < S))
                kp = pos[want]
                see = (kp[None] <= qp[:, None]) & ((kp[None] > qp[:, None] - W) | (kp[None] < S))
                for h in range(Hk):
                    kk, vv = k[want, h], v[want, h]
                    for j in range(Hq // Hk):
                        hq = h * (Hq // Hk) + j
                        z = s["q"][row + b:row + b + m, hq].double() @ kk.T / math.sqrt(d)
                        z = torch.where(see, z, -math.inf)
                        out[row + b:row + b + m, hq] = torch.softmax(z, -1) @ vv
            if pool is not None:
                e = s["slots_host"][n]
                kept = [i for i in range(L) if a + i < S or i >= L - W]
                places = torch.tensor([place(a + i, case) for i in kept], device=dev)
                rows = torch.tensor(kept, device=dev) + row
                pool[e, 0][:, places] = s["k"][rows].double().transpose(0, 1)
                pool[e, 1][:, places] = s["v"][rows].double().transpose(0, 1)
            row += L
        return out if pool is None else (out, pool)

    def moves(s):
        case = s["case"]
        pools = [p.double() for p in s["pools"]]
        if case["op"] == "fork":
            for i, j in zip(s["src"].tolist(), s["dst"].tolist()):
                if j >= 0:
                    for p, was in zip(pools, s["pools"]):
                        p[j] = was[i].double() if i >= 0 else 0.0
            return pools
        table = s["slots"].tolist()
        live = sorted(x for x in table if x >= 0)
        free = [x for x in range(len(live)) if x not in live]
        to = {x: x if x < len(live) else free.pop(0) for x in live}
        for x, y in to.items():
            for p, was in zip(pools, s["pools"]):
                p[y] = was[x].double()
        return [None] + [p[:len(live)] for p in pools]

    s = prepare(case, seed)
    if case["op"] == "rope":
        return rope(s)
    return attention(s) if case["op"] in ("prefill", "decode") else moves(s)
