"""examples/attention_block.py: the layer, attention, cache and decoding run together (GPU)."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_block.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("attention_block", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_training_step_lowers_the_loss(example):
    losses = example.train(example.AttentionBlock(), steps=15)
    assert losses[-1] < 0.8 * losses[0], losses


def test_decoding_continues_the_prefill(example):
    # bf16 rows, filters and outputs on both paths, each rounded on its own: a few 2^-8 of the largest output
    assert example.serve(example.AttentionBlock(seed=3)) < 2e-2
