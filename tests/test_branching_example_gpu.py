"""The operators for several continuations together, as examples/branching_decoder.py uses them: trees grown,
checked and accepted in a hybrid decoder, and beam search, against the same tokens read in order."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def model():
    from branching_decoder import Branching
    return Branching()


@pytest.mark.parametrize("seed", [1, 2])
@pytest.mark.parametrize("shape", [(4, 5), (1, 1), (2, 32), (16, 4)])
def test_drafts(model, seed, shape):
    """The bound of the served example: sums in other orders, roundings to bf16 and of the norm's 8-bit output at
    other places (2^-4 of a value, a few per cent of one layer of four); no room for a wrong place, path or state."""
    import gated_deltanet_linear_05_gb300 as gdn
    from branching_decoder import drafts
    free = model.free
    assert drafts(model, levels=shape[0], width=shape[1], seed=seed) < 0.1
    model.free = free
    assert gdn.gdn_device_status() == 0


@pytest.mark.parametrize("seed", [2, 3])
@pytest.mark.parametrize("width", [1, 4, 7])
def test_beams(model, seed, width):
    """The same bound for the hidden states; of five tokens' scores, 0.1 of a logit's standard deviation (1) each,
    three times over."""
    from branching_decoder import beams
    free = model.free
    hidden, scores = beams(model, width=width, seed=seed)
    assert hidden < 0.1 and scores < 5 * 0.3
    model.free = free
