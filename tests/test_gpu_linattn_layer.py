"""The example layer: its operators together train, and serve a prompt and then single tokens."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_layer_trains_and_serves():
    spec = importlib.util.spec_from_file_location("layer", os.path.join(ROOT, "examples", "linear_attention_layer.py"))
    layer = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(layer)
    losses, off = layer.main()
    assert losses[-1] < 0.9 * losses[0]
    # two bf16 projections and the operators' roundings on either side: a few times 2^-8
    assert max(off) < 8 * 2.0 ** -8
