"""The example's decoding loop: trees verified in one pass give the logits of
plain decoding along the same tokens, whatever was drafted, accepted and
moved in the caches on the way."""

import importlib.util
import os

import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "verify_tree.py")


def example():
    spec = importlib.util.spec_from_file_location("verify_tree", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("depth", [1, 3, 5])
def test_trees_give_plain_decodings_logits(depth):
    count, drafts, worst = example().main(steps=8, depth=depth)
    assert count == 3 * 9 + drafts and drafts > 0
    # logits of size about 1; two layers of bfloat16 roundings (2^-8 each) of activations of size about 1
    # reach them through sums of 256 products
    assert worst < 0.15
