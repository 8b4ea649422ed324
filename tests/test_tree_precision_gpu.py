"""How exact the delta rule over trees is: float32 for inputs of either type."""
import pytest
import torch

import gated_deltanet_linear_05_gb300 as gdn
from tree_testlib import DeltaBatch, delta_rule

pytestmark = pytest.mark.gpu

# Errors' rms beside the values'.  Operands have three terms of 8 bits, and of the nine products of terms the six above
# 2^-24 are taken, the largest last.  Of a sum of 128 products only the last 8 steps, each of 16 products of the leading
# terms, add to a sum of its full size, and each loses at most 2^-23 of it: 4.8e-7 on average.  Three such sums follow one
# another (with the state, of the keys, with the tree's matrix): 1.5e-6, and some float32 roundings of 2^-24 each.  Two
# terms in place of three would leave up to 2^-15 of each operand, some 1e-5.
FLOAT32 = 2e-6


def rms_error(got, want):
    return float((got.cpu().double() - want).square().mean().sqrt() / want.square().mean().sqrt())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["chain", "bushy", "narrow"])
@pytest.mark.parametrize("t,chunk", [([16, 9], 16), ([32, 20], 32), ([64, 45], 64)])
@pytest.mark.parametrize("decay", [0.01, 1.0])
def test_the_delta_rule_is_float32(dtype, kind, t, chunk, decay):
    b = DeltaBatch(t, 2, 4, dtype, seed=chunk, decay=decay, kinds=(kind,))
    o, delta = gdn.gdn_verify_tree(*b.args(), o=torch.empty(b.v.shape, device="cuda"), chunk=chunk)
    want_o, want_d, _ = delta_rule(b)
    assert rms_error(o, want_o) <= FLOAT32 and rms_error(delta, want_d) <= FLOAT32
