"""Paged attention of single rows (no cu_seqlens) with shared prefixes, against 64 bits."""
import random

import pytest

from gpu_util import torch
from paged_util import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("members", [1, 4, 5, 8, 33, 65, 130])
@pytest.mark.parametrize("Hq,Hk", [(8, 2), (16, 1), (17, 1)])
def test_single_rows_behind_prefixes(members, Hq, Hk):
    """Groups of one query row to several tiles, a sequence of none, another cut of the work than with cu_seqlens."""
    r = random.Random(members)
    own = [(r.randint(0, 90), 1) for _ in range(members + 3)]
    b = Batch(own, [(members, 700), (2, 129)], Hq=Hq, Hk=Hk, seed=members)
    b.check(b.call(cu_seqlens=None))


def test_single_rows_of_padded_sequences():
    own = [(5 + 9 * i, 1) for i in range(20)]
    b = Batch(own, [(6, 300), (0, 40), (9, 50)], seed=3)
    t = torch()
    slots = b.slots.clone()
    slots[[0, 7, 19]] = -1
    out = t.full_like(b.q, 2.0)
    b.call(cu_seqlens=None, slots=slots, out=out)
    b.check(out, skip=(0, 7, 19))
    assert (out[[0, 7, 19]] == 2).all()
