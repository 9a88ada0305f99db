"""The example block trains, and its decode steps continue a prefill as one pass would."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_block_trains_and_decodes():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "delta_block.py")
    spec = importlib.util.spec_from_file_location("delta_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses, off = mod.main()
    assert losses[-1] < 0.9 * losses[0]
    # bf16 activations rounded at the same places; products of other shapes round differently
    assert off < 2.0 ** -6
