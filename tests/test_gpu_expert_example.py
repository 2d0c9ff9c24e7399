"""The expert-layer example runs, and its results are those of the float64 arithmetic."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("sizes", [dict(), dict(tokens=5, experts=3, pool=4, h_in=1056, h_out=520,
                                                train_tokens=77)])
def test_expert_lora_layer(sizes):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location(
        "expert_lora_layer", os.path.join(ROOT, "examples", "expert_lora_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # each result is rounded to bfloat16 (2^-8) at most three times on its way
    assert max(example.main(**sizes)) < 3 * 2.0 ** -8
