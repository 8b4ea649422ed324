"""The attention-layer calls and the delta-rule calls together, as a decoder uses them: a batch
served behind a shared prefix (packed prompts, then token by token) against the same sequences
read in one piece.  The two differ in the order of sums and in where bf16 and e4m3 round: a
rounding of the norm's 8-bit output is 2^-4 of a value and takes a share of a few per cent of the
attention layer's result, one layer of four; a bound of 0.1 on the relative difference leaves that
room and none for a wrong place, position, page or state."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_decoder.py")


@pytest.fixture(scope="module")
def example():
    from gated_deltanet_linear_05_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("hybrid_decoder", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("prompts,system", [((7, 40, 1, 23, 64), 100), ((130,), 33), ((1, 1, 16), 16)])
def test_served_batch_equals_whole_sequences(example, prompts, system):
    import torch
    import gated_deltanet_linear_05_gb300 as gdn
    error = example.main(requests=len(prompts), system=system, prompts=prompts, steps=5)
    torch.cuda.synchronize()
    assert error < 0.1
    assert gdn.gdn_device_status() == 0


def test_prompt_as_long_as_the_shared_prefix(example):
    """Plain and prefixed batches of one size in turn: each with a workspace of its own."""
    import torch
    error = example.main(requests=1, system=33, prompts=(33,), steps=3)
    torch.cuda.synchronize()
    assert error < 0.1
