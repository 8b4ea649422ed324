"""The delta rule over trees writes its outputs' rows and nothing around them."""
import pytest
import torch

import gated_deltanet_linear_05_gb300 as gdn
from tree_testlib import DeltaBatch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [[0, 30, 10], [0, 500, 40], [-7, 20, 1 << 30], [40, 40, 0]])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("wide", [False, True])
def test_a_malformed_cu_seqlens_leaves_what_lies_around(bad, dtype, wide):
    """Both outputs of the delta rule between rows that are looked at again: the kernel keeps tokens within their number."""
    b = DeltaBatch([20, 20], 1, 2, dtype, seed=53)
    room = torch.full((48, 2, 128), 7.0, dtype=torch.float32 if wide or dtype == "f32" else torch.bfloat16, device="cuda")
    deltas = torch.full((48, 2, 128), 7.0, device="cuda")
    cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
    o, delta = gdn.gdn_verify_tree(b.q, b.k, b.v, b.g, b.beta, b.state, cu, b.up, o=room[4:44], delta=deltas[4:44])
    assert o.data_ptr() == room[4:].data_ptr() and delta.data_ptr() == deltas[4:].data_ptr()
    for x in (room, deltas):
        assert (x[:4] == 7).all() and (x[44:] == 7).all()
    assert gdn.gdn_device_status() == 0
