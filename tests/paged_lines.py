"""What the workers of the paged attention's tiles kernel do with a batch: the line of key tiles, cut up on the host by
the rules of kda_paged_attend.cuh.  Tests assert with it that their batches reach the items that they are there for."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kda_linear_attention_chunk_gb300", "csrc")


def constant(name):
    for f in ("kda_paged_attend.cuh", "kda_paged_tiles.cu"):
        with open(os.path.join(CSRC, f)) as fh:
            found = re.search(rf"\b{name} = (\d+)\b", fh.read())
        if found:
            return int(found.group(1))
    raise KeyError(name)


def spans(own, groups, G):
    """(rows, first key tile, key tiles, set-up) of each span of a key head's line.  own, groups: as of paged_util.Batch."""
    few, rows = constant("kFewRows"), constant("kTileRows")
    keys, short, set_up = constant("kTileKeys"), constant("kShortTiles"), constant("kTilesSetUp")
    span = 2 * (rows // G)
    prefix = [length for members, length in groups for _ in range(members)]
    prefix += [0] * (len(own) - len(prefix))
    parts, n = [], 0                                   # rows, position of the first one (None: all see all keys), keys
    for members, length in groups:
        parts.append((sum(b for _, b in own[n:n + members]), None, 0, length))
        n += members
    parts += [(b, a + p, p, a + p + b) for (a, b), p in zip(own, prefix)]
    out = []
    for tokens, first, key0, key1 in parts:
        if tokens <= 0 or key1 <= key0 or tokens * G <= few:
            continue
        for j in range(-(-tokens // span)):
            end = key1 if first is None else min(key1, first + min((j + 1) * span, tokens))
            out.append((min(span, tokens - j * span), key0 // keys, -(-end // keys) - key0 // keys,
                        set_up if key1 - key0 <= short * keys else 0))
    return out


def workers(own, groups, Hq, Hk, sms):
    """The items (rows, key tiles, dealt) of each worker, one after the other."""
    G = Hq // Hk
    line = spans(own, groups, G)
    total = sum(tiles + set_up for _, _, tiles, set_up in line)
    share = max(-(-total * Hk // sms), constant("kTilesSetUp") + 1)
    out, at, dealt = [[] for _ in range(sms)], 0, constant("kDealt")
    for _ in range(Hk):
        for rows, _, tiles, set_up in line:
            at += set_up
            while tiles:
                worker = at // share
                n = min(tiles, (worker + 1) * share - at)
                out[worker].append((rows, n, rows <= constant("kTileRows") // G and n >= dealt))
                at += n
                tiles -= n
    return out
