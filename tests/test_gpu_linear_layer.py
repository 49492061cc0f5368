"""The example layer: linear attention and group norm together, trained and decoded."""
import importlib.util
import os

import pytest

from util import cuda_device

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_example_trains_and_decodes():
    cuda_device()
    spec = importlib.util.spec_from_file_location("layer", os.path.join(ROOT, "examples", "linear_attention_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    first, last, off = module.main(steps=12)
    assert last < 0.9 * first
    # Outputs of order one. The prompt and the step round o, the norm and the products to bf16, each by up to
    # 2^-9 of values up to about 4, and the prompt its weights and states too: a few times 2^-7.
    assert off <= 8 * 2.0 ** -7
