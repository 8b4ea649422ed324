"""Selection over beams whose logits are all far below 0, as masks by a large finite value leave them: a row's level
cancels in its log-softmax, so the scores are those of the same row at any level."""
import math

import pytest
import torch

import gated_deltanet_linear_05_gb300 as gdn
from test_beams_gpu import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [1000, 40961])
@pytest.mark.parametrize("level", ["lowest", -1e30, -1e16, -1e12, 1e30, "highest"])
def test_a_beam_of_masked_tokens_alone_does_not_win(dtype, vocab, level):
    """A beam without a token left has score - ln V for each, and stands behind the beams that are better."""
    info = torch.finfo(dtype)
    level = {"lowest": info.min, "highest": info.max}.get(level, level)
    x = torch.randn(3, 4, vocab, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").to(dtype)
    x[0, 1] = x[1, 0] = x[1, 3] = level
    x[2] = level
    s = torch.tensor([[-5.0, -5.0, -6.0, -20.0], [-5.0, -0.5, -40.0, -30.0], [-3.0, -2.0, -1.0, -2.0]], device="cuda")
    for top in (1, 4, 17, 64):
        score, parent, token = check(x, s, top)
        assert (parent[2] == 2).all() and token[2].tolist() == list(range(top))
        # -1 - ln V, of which ln V comes from V equal powers (SCORE of test_beams_gpu), rounded to float32 once
        assert (score[2].double() + 1 + math.log(vocab)).abs().max() <= 2.0 ** -22 + 85 * 2.0 ** -24 + 2.0 ** -24 * 12
    fin = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    fin[:, 2] = True
    for top in (1, 4, 17):
        check(x, s, top, fin, vocab // 2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("level", [-1e4, -1e7, -1e12, -1e16, -3e37, 1e7, 3e37])
def test_rows_far_from_zero(dtype, level):
    """Distinct values at any level: their steps are then large, and the first few decide."""
    g = torch.Generator(device="cuda").manual_seed(4)
    step = abs(level) * torch.finfo(dtype).eps
    x = level + step * torch.randint(-9, 10, (2, 5, 9001), generator=g, device="cuda").double()
    x[0, 2] -= level
    x[1, 1, 100:] = -math.inf
    s = -9 * torch.rand(2, 5, generator=g, device="cuda")
    for top in (1, 5, 64):
        check(x.to(dtype), s, top)


def test_ties_at_a_level():
    """Equal rows at a far level: beams tie where score and logit do, and the lower place comes first."""
    x = torch.full((1, 3, 700), -1e30, device="cuda")
    x[:, :, 5:] = torch.finfo(torch.float32).min
    s = torch.tensor([[-2.0, -1.0, -1.0]], device="cuda")
    _, parent, token = gdn.gdn_beam_select(x, s, 12)
    assert parent[0].tolist() == [1] * 5 + [2] * 5 + [0] * 2 and token[0].tolist() == [0, 1, 2, 3, 4] * 2 + [0, 1]
