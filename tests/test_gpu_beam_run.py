"""The operators of beam search together, as a server runs them."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("seed", [0, 1])
def test_beam_search_example(seed):
    """Its own assertions: the choices over the step's logits, no page lost.  Its logits pass bf16 roundings, each off by
    at most 2^-8 of a value: of the embedding none, per layer of x, qkv, the attention's output, its projection and their sum,
    then of the logits' product and sum: 2 * 5 + 2 in a row, were all of them the largest and of one sign."""
    spec = importlib.util.spec_from_file_location("beam_search", os.path.join(ROOT, "examples", "beam_search.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.main(steps=10, seed=seed) <= 12 * 2.0 ** -8
    torch.cuda.synchronize()
