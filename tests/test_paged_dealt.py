"""Paged attention where key tiles of one query tile are dealt to both pipelines of a CTA: alone, and behind items of one
or two key tiles, whose queries may still be on their way when such an item begins."""
import random

import pytest

from paged_lines import workers

# own, groups, Hq, Hk, d, page, dtype; how many of 152 workers have a dealt item, and one directly behind another item of
# one query tile and at most two key tiles that is not their first
DRAFTS = [((200, 1500)[i % 2], 8) for i in range(128)]
RAGGED = [(int(20 * 400 ** random.Random(i).random()), 8) for i in range(128)]
BEAMS = [(i * 11 % 150, 1) for i in range(128)], [(8, 1000 + 467 * i) for i in range(16)]
MIXED = ([(i * 29 % 200, 1) for i in range(64)] + [((150, 1300, 90, 40)[i % 4], (8, 8, 1, 40)[i % 4]) for i in range(160)],
         [(16, (90, 1100, 250, 3000)[i % 4]) for i in range(4)])
BATCHES = {
    "drafts": (DRAFTS, [], 32, 8, 128, 64, "bf16", 150, 150),
    "ragged": (RAGGED, [], 32, 8, 128, 128, "fp16", 120, 80),
    "beams": (*BEAMS, 32, 8, 128, 64, "bf16", 140, 0),
    "mixed": (*MIXED, 32, 8, 64, 16, "bf16", 80, 60),
    "one query tile full": ([(180 + i, 16) if i % 3 else (1900, 16) for i in range(90)], [], 64, 8, 64, 256, "fp16", 80, 60),
}


@pytest.mark.parametrize("name", BATCHES)
def test_batches_have_such_items(name):
    own, groups, Hq, Hk, *_, dealt, behind = BATCHES[name]
    got = workers(own, groups, Hq, Hk, 152)
    one = 128 // (Hq // Hk)
    assert sum(any(d for _, _, d in items) for items in got) >= dealt
    assert sum(any(b[2] and a[0] <= one and a[1] <= 2 for a, b in zip(items[1:], items[2:])) for items in got) >= behind


@pytest.mark.gpu
@pytest.mark.parametrize("name", BATCHES)
def test_dealt_items(name):
    """Every row against 64 bits, and the same bytes time after time, with the queries in L2 and not."""
    from paged_util import Batch
    own, groups, Hq, Hk, d, page, dtype, *_ = BATCHES[name]
    b = Batch(own, groups, page=page, Hq=Hq, Hk=Hk, d=d, dtype=dtype, seed=23)
    t, want = b.t, b.call()
    b.check(want)
    room = t.empty(1 << 26, device="cuda")             # twice what L2 holds
    for i in range(24):
        if i % 2:
            room.fill_(i)
        assert t.equal(b.call(), want)
