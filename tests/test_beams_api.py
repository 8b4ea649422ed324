"""Selection over beams: what the binding passes on for logits whose rows lie over each other, and the workspace's size.
Made-up devices and addresses: nothing is launched."""
import pytest
import torch

import gated_deltanet_linear_05_gb300 as gdn
from gated_deltanet_linear_05_gb300 import build as gdn_build
from test_branching_marshal import world, zeros  # noqa: F401 (the fixture)


@pytest.fixture(scope="module", autouse=True)
def _built():
    gdn_build.build()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("have,groups,beams,vocab", [
    ((1, 1), 1, 4, 100), ((1, 1), 3, 4, 100), ((3, 1), 3, 4, 100), ((1, 4), 3, 4, 100), ((1, 1), 4, 1, 100), ((1, 1), 2, 2, 1)])
def test_rows_over_each_other_are_refused(world, dtype, have, groups, beams, vocab):  # noqa: F811
    """Expanded logits hold fewer values than the call would read."""
    x = zeros(*have, vocab, dtype=dtype).expand(groups, beams, vocab)
    s, ws = zeros(groups, beams), zeros(1 << 20, dtype=torch.uint8)
    for kw in (dict(), dict(workspace=ws)):
        for _ in range(2):  # also where it has been seen
            with pytest.raises(ValueError):
                gdn.gdn_beam_select(x, s, 1, **kw)
    assert not world.calls
    gdn.gdn_beam_select(x.contiguous(), s, 1, workspace=ws)
    assert gdn.GdnBeamShape.from_buffer_copy(world.calls.pop()[1][0]).row_stride == vocab


def test_rows_closer_than_their_length_are_refused(world):  # noqa: F811
    flat, s = zeros(1000), zeros(2, 3)
    for stride in ((120, 40, 1), (3, 1, 1), (0, 100, 1), (300, 100, 2)):
        with pytest.raises(ValueError):
            gdn.gdn_beam_select(flat.as_strided((2, 3, 100), stride), s, 4)
    assert not world.calls


def test_a_row_alone_has_no_stride(world):  # noqa: F811
    """A single row is taken whatever torch says of its strides."""
    flat, ws = zeros(1000), zeros(1 << 20, dtype=torch.uint8)
    gdn.gdn_beam_select(flat.as_strided((1, 1, 100), (0, 3, 1)), zeros(1, 1), 4, workspace=ws)
    gdn.gdn_beam_select(flat.as_strided((2, 1, 100), (200, 3, 1)), zeros(2, 1), 4, workspace=ws)
    gdn.gdn_beam_select(flat.as_strided((1, 3, 100), (7, 150, 1)), zeros(1, 3), 4, workspace=ws)
    assert [gdn.GdnBeamShape.from_buffer_copy(a[0]).row_stride for _, a in world.calls] == [100, 200, 150]
