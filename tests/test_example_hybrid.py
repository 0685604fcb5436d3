"""The hybrid-stack example: prefill in chunks, fork, decode, compaction and decode again against one prefill."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", [0, 1])
def test_decoded_samples_match_a_prefill_of_their_texts(seed):
    """Four layers, each with 16-bit outputs and operands (fp16 in the linear layers' prefill): a relative error of
    2^-8 at most each, and projections that keep its size, so 4 x 2^-8 of the residual stream bounds it."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_stack.py")
    spec = importlib.util.spec_from_file_location("hybrid_stack", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    assert module.main(seed=seed) <= 4 * 2.0 ** -8
