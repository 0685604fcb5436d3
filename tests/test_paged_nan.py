"""NaN among the keys that a row of the paged attention sees: its answer is NaN, however its keys are cut into pieces, and
the others' stay what they were."""
import math

import pytest

pytestmark = pytest.mark.gpu


def nan_keys(b, slot, lo, hi):
    p, r = b.places(slot, lo, hi)
    b.pool[p, 0, :, r] = math.nan


# a row of few and of many (query tiles), and so many that the join gives a head eight lanes
@pytest.mark.parametrize("own,members", [([(0, 1), (4, 1)], 2), ([(0, 17), (0, 40), (9, 1)], 3), ([(0, 1)] * 700, 700),
                                         ([(0, 30)] * 40, 40)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_own_keys_behind_a_prefix(own, members, dtype):
    """The only keys of a row's own."""
    from paged_util import Batch
    b = Batch(own, [(members, 300)], dtype=dtype, seed=41)
    t, want = b.t, b.call()
    nan_keys(b, b.ids[0], 300, b.start[0] + b.lens[0])
    got = b.call()
    rows = b.cu[1]
    assert got[:rows].isnan().all() and t.equal(got[rows:], want[rows:])


@pytest.mark.parametrize("own", [[(3, 1), (0, 1)], [(8, 20), (3, 1)], [(8, 20)] * 40])
@pytest.mark.parametrize("prefix", [1, 40, 700])
def test_a_prefix(own, prefix):
    """All of its keys: every member's answer is NaN."""
    from paged_util import Batch
    b = Batch(own + [(50, 3)], [(len(own), prefix)], seed=42)
    t, want = b.t, b.call()
    nan_keys(b, b.kept[0], 0, prefix)
    got = b.call()
    rows = b.cu[len(own)]
    assert got[:rows].isnan().all() and t.equal(got[rows:], want[rows:])


@pytest.mark.parametrize("context,rows", [(60000, 1), (60000, 6), (30000, 300)])
@pytest.mark.parametrize("lo,hi", [(0, 8000), (20000, 28000), (28500, 28501)])
def test_a_stretch_of_a_long_context(context, rows, lo, hi):
    """All the keys that some worker has of it, or one."""
    from paged_util import Batch
    b = Batch([(context, rows), (200, 1)], seed=43)
    t, want = b.t, b.call()
    nan_keys(b, b.ids[0], lo, hi)
    got = b.call()
    assert got[:rows].isnan().all() and t.equal(got[rows:], want[rows:])


def test_both_pipelines_of_a_dealt_item():
    """Key tiles without a number in one of them, in the other, and in both."""
    from paged_util import Batch
    from test_paged_dealt import BEAMS
    for stretch in ([(0, 128)], [(128, 256)], [(0, 900)]):
        b = Batch(*BEAMS, Hq=32, Hk=8, seed=44)
        t, want = b.t, b.call()
        for lo, hi in stretch:
            nan_keys(b, b.kept[9], lo, hi)
        got = b.call()
        other = [i for i in range(b.T) if b.group[i] != 9]
        assert got[72:80].isnan().all() and t.equal(got[other], want[other])
