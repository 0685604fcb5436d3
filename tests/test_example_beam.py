"""The beam-search example: it runs, and each hypothesis' last hidden row is that of a prefill of its text.

Bound: four layers, each with 16-bit outputs and operands: a relative error of 2^-8 at most each, and projections that keep
its size, so 4 x 2^-8 of the residual stream bounds it."""
import importlib.util
import os

import pytest

import kda_linear_attention_chunk_gb300 as kda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed,beams", [(0, 4), (1, 1), (2, 7)])
def test_hypotheses_match_a_prefill_of_their_texts(seed, beams):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "beam_search.py")
    spec = importlib.util.spec_from_file_location("beam_search", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    worst, scores = module.main(seed=seed, beams=beams)
    assert worst <= 4 * 2.0 ** -8 and scores.isfinite().all()
    assert kda.device_error(reset=True) == 0
