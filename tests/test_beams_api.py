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


# ------------------------------------------------------------------ the workspace

def _size(groups, beams, vocab, top, dtype=gdn.GDN_F32):
    return gdn.gdn_beam_workspace_size(gdn.make_beam_shape(groups, beams, vocab, top, dtype))


@pytest.mark.parametrize("dtype", [gdn.GDN_BF16, gdn.GDN_F32])
@pytest.mark.parametrize("beams,vocab,top", [(8, 151936, 8), (48, 99999, 48), (4, 32000, 4), (1, 1 << 24, 64), (64, 40000, 64), (3, 500, 2)])
def test_a_workspace_serves_fewer_requests(dtype, beams, vocab, top):
    size = [_size(g, beams, vocab, top, dtype) for g in range(700)]
    assert size == sorted(size) and size[0] == 0


def test_a_workspace_serves_smaller_sizes():
    """Larger values of any of the four never need less."""
    ladder = dict(groups=[1, 2, 5, 17, 64, 300, 5000], beams=[1, 2, 3, 7, 8, 31, 32, 33, 48, 63, 64],
                  vocab=[64, 500, 4096, 4097, 8192, 8193, 32000, 99999, 151936, 262144, 1 << 22, 1 << 24], top=[1, 2, 7, 32, 33, 64])
    for dtype in (gdn.GDN_BF16, gdn.GDN_F32):
        for name, values in ladder.items():
            for at in ([0] * 4, [2, 4, 6, 2], [4, 8, 8, 3], [5, 10, 10, 5], [6, 0, 4, 0], [3, 6, 11, 4]):
                case = {n: ladder[n][i] for n, i in zip(ladder, at)}
                size = [_size(**{**case, name: v}, dtype=dtype) for v in values]
                assert size == sorted(size), (name, case, size)


def test_workspaces_stay_small():
    """Beside the logits that a call reads."""
    for groups, beams, vocab, top in ((64, 8, 151936, 8), (4, 48, 99999, 48), (256, 16, 262144, 16), (65, 2, 1 << 24, 6), (1, 64, 1 << 22, 64)):
        assert _size(groups, beams, vocab, top) <= groups * beams * vocab * 4 * 0.03
