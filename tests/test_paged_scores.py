"""Paged attention where scale times score is large and its pieces (prefixes and own keys, spans that workers share, the two
pipelines of a dealt query tile) have unequal maxima that share weight.

Scores are whole numbers that fp32 holds, base + j with j < 12, so their distances are exact and the bound has no term for
them: attention64's with whole=True.  Its 2^-19 covers what is left of the exponentials: an argument of at most 12 log2 e < 2^5
off by 2^-24 of itself for its rounding and 2^-25 for the scale's (below 2^-19 log 2 of the probability together), 2 ulp
of exp2; what a maximum's product with the scale was rounded by is a number that fp32 holds, and its exponential has 2 ulp more."""
import pytest

from paged_lines import workers
from test_paged_dealt import BEAMS, DRAFTS

BATCHES = {
    "dealt": (*BEAMS, 32, 8),
    "drafts": (DRAFTS[:64], [], 32, 8),
    "two query tiles, cut": ([(5000, 300), (700, 140)], [], 8, 2),
    "prefix and own": ([(300, 40), (100, 33), (5, 1), (600, 1)], [(2, 260), (2, 3000)], 8, 2),
}


def test_the_first_batch_has_dealt_items_cut_and_whole():
    own, groups, Hq, Hk = BATCHES["dealt"]
    tiles = [-(-length // 128) for _, length in groups]
    dealt = [n for items in workers(own, groups, Hq, Hk, 152) for _, n, d in items if d]
    assert len(dealt) > 100 and any(n in tiles for n in dealt) and any(n not in tiles for n in dealt)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("base,scale", [(128, 1.0), (1024, 0.5), (2048, 1.0), (4096, 1.0)])
@pytest.mark.parametrize("name", BATCHES)
def test_pieces_join_by_the_weights_of_their_scores(name, base, scale, dtype):
    from paged_util import Batch, attention64
    own, groups, Hq, Hk = BATCHES[name]
    b = Batch(own, groups, page=128, Hq=Hq, Hk=Hk, dtype=dtype, seed=31, scale=scale)
    t = b.t
    g = t.Generator(device="cuda")
    g.manual_seed(32)
    b.q.zero_()
    b.q[..., 0], b.q[..., 1] = 1024, 1
    live = ~b.pool[:, 0, :, :, 0].isnan()              # [pages][Hk][page]
    keys = t.zeros_like(b.pool[:, 0])
    keys[..., 0] = base
    # a page's scores lie close together, and those of the next one elsewhere
    page = t.randint(0, 10, (live.shape[0], 1, 1), generator=g, device="cuda")
    keys[..., 1] = (page + t.randint(0, 3, live.shape, generator=g, device="cuda")).to(keys.dtype)
    b.pool[:, 0] = t.where(live[..., None], keys, b.pool[:, 0])
    out = b.call()
    for n, L in enumerate(b.lens):
        k, v = b.keys(n)
        pos = t.arange(b.start[n], b.start[n] + L, device="cuda")
        ref, bound = attention64(b.q[b.cu[n]:b.cu[n + 1]].double(), k, v, pos, scale, dtype, whole=True)
        off = ((out[b.cu[n]:b.cu[n + 1]].double() - ref).abs() / bound).max().item()
        assert off <= 1, (n, off)
