"""Selection over beams and vocabulary and the reordering of rows, against their definitions."""
import math

import numpy as np
import pytest
import torch

import gated_deltanet_linear_05_gb300 as gdn

pytestmark = pytest.mark.gpu

# Of a score: the powers are exact to 2^-22 and summed over at most 32 values a step, 40 steps and 13
# levels in float32 (2^-24 each, relative to the sum, which the logarithm makes absolute).
SCORE = 2.0 ** -22 + 85 * 2.0 ** -24


def definition(logits, scores, finished, pad):
    """All scores [G, W V] in 64 bits on the CPU."""
    x = logits.cpu().double()
    s = scores.cpu().double()[..., None]
    m = x.amax(-1, keepdim=True)
    x = s + (x - m - torch.log(torch.exp(x - m).sum(-1, keepdim=True)))
    x = torch.where(torch.isnan(x) | ~torch.isfinite(s), -math.inf, x)
    if finished is not None:
        f = finished.cpu()
        x[f] = -math.inf
        for g, w in torch.nonzero(f).tolist():
            if math.isfinite(scores[g, w]):
                x[g, w, pad] = scores[g, w].double().item()
    return x.flatten(1)


def check(logits, scores, top, finished=None, pad=0, **kw):
    got_s, parent, token = (x.cpu() for x in gdn.gdn_beam_select(logits, scores, top, finished=finished, pad_token=pad, **kw))
    groups, beams, vocab = logits.shape
    every = definition(logits, scores, finished, pad)
    want, at = torch.sort(every, dim=1, descending=True, stable=True)
    want, at = want[:, :top + 1], at[:, :top + 1]
    got = parent.long() * vocab + token
    assert ((parent >= 0) & (parent < beams) & (token >= 0) & (token < vocab)).all()
    here = torch.gather(every, 1, got)
    dead = torch.isinf(want[:, :top])
    assert torch.equal(dead, torch.isinf(got_s)) and (got_s[dead] == -math.inf).all()
    tol = SCORE + 2.0 ** -24 * want[:, :top][~dead].abs()
    assert ((got_s.double() - want[:, :top])[~dead].abs() <= tol).all()
    # no continuation twice, and every one as good as the definition's
    assert all(len(set(row)) == top for row in got.tolist())
    assert ((here - want[:, :top])[~dead].abs() <= 2 * SCORE).all()
    # the definition's very own wherever its neighbours are not within the scores' error; equal
    # scores of one beam, of equal rows, and -inf, are told apart by their places alone
    best = at[:, :top]
    gap = want.diff(dim=1).abs()
    if gap.shape[1] < top:
        gap = torch.cat([gap, torch.full((groups, 1), math.inf, dtype=gap.dtype)], 1)
    close = torch.zeros_like(best, dtype=torch.bool)
    near = (gap > 0) & (gap <= 2 * SCORE)
    close |= near[:, :top]
    close[:, 1:] |= near[:, :top - 1]
    assert ((got == best) | close).all()
    return got_s, parent, token


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("groups,beams,vocab,top", [
    (1, 1, 1, 1), (1, 1, 7, 7), (2, 3, 64, 5), (1, 2, 1023, 64), (3, 4, 5000, 4), (1, 1, 100003, 8), (2, 8, 32768, 16),
    (5, 5, 8193, 17), (1, 64, 3001, 64), (40, 2, 4096, 3), (1, 4, 262144, 33), (300, 1, 999, 2)])
def test_select(dtype, groups, beams, vocab, top):
    g = torch.Generator(device="cuda").manual_seed(vocab + top)
    x = (torch.randn(groups, beams, vocab, generator=g, device="cuda") * 3).to(dtype)
    s = -5 * torch.rand(groups, beams, generator=g, device="cuda")
    check(x, s, top)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [500, 40961])
@pytest.mark.parametrize("kind", ["constant", "rising", "falling", "few", "two", "equal rows", "zeros"])
def test_select_orders(dtype, vocab, kind):
    """Values as they lie worst for a threshold, and ties: by place."""
    i = torch.arange(vocab, device="cuda")
    x = {"constant": torch.full((vocab,), 1.25, device="cuda"), "rising": i / 1000.0, "falling": -i / 1000.0,
         "few": (i % 7 == 3).float() * 4, "two": (i >= vocab - 2).float() * 9,
         "equal rows": torch.randn(vocab, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda"),
         "zeros": torch.where(i % 2 == 0, 0.0, -0.0)}[kind]
    x = x.to(dtype).expand(2, 3, vocab).contiguous()
    s = torch.tensor([[-1.0, -1.0, -1.0], [-2.0, -1.0, -3.0]], device="cuda")
    for top in (1, 3, 16, 17, 64):
        got, parent, token = check(x, s, top)
        if kind == "equal rows" and dtype == torch.float32:
            # no two values of the row are equal, the first request's beams are: each token comes with
            # beams 0, 1, 2 (in bf16 a beam's equal values come before the next beam's)
            assert parent[0].tolist() == [j % 3 for j in range(top)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("beams,top", [(16, 16), (32, 32), (64, 17), (64, 64)])
@pytest.mark.parametrize("kind", ["any", "constant", "equal rows", "some finished or dead", "one ahead"])
def test_select_many_lists(dtype, beams, top, kind):
    """As many sampled entries of lists as a request can have, in the orders that are worst for a bound."""
    vocab = 40000
    g = torch.Generator(device="cuda").manual_seed(beams + top)
    x = torch.randn(2, beams, vocab, generator=g, device="cuda") * 2
    s = -9 * torch.rand(2, beams, generator=g, device="cuda")
    fin = None
    if kind == "constant":
        x.fill_(0.75)
        s.fill_(-2.0)
    elif kind == "equal rows":
        x[:] = x[0, 0]
    elif kind == "some finished or dead":
        fin = torch.rand(2, beams, generator=g, device="cuda") < 0.5
        fin[1, 1:] = True
        s[0, 1::5] = -math.inf
        x[0, 2::7, 11] = math.nan
    elif kind == "one ahead":
        s -= 100
        s[:, beams // 2] = 0
    check(x.to(dtype), s, top, finished=fin, pad=7)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_select_nothing_left(dtype):
    """Forbidden tokens, finished and dead beams, rows that are not finite."""
    vocab = 3000
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(6, 4, vocab, generator=g, device="cuda").to(dtype)
    s = -torch.rand(6, 4, generator=g, device="cuda")
    x[0, :, 5:] = -math.inf           # 20 continuations in all
    x[1, 0] = -math.inf               # a beam of nothing
    x[1, 1, 17] = math.nan
    x[1, 2, 2999] = math.inf
    s[2, 0], s[2, 1], s[2, 2] = -math.inf, math.nan, math.inf
    s[3] = -math.inf                  # no beam
    x[5, :, :] = -math.inf
    x[5, 3, 2998] = 0.5               # a single continuation
    fin = torch.zeros(6, 4, dtype=torch.bool, device="cuda")
    fin[4, 1:] = True
    fin[5, 0] = True
    s[5, 0] = -0.25
    for top in (1, 4, 30, 64):
        for pad in (0, 2, 2999):
            check(x, s, top, fin, pad)
    check(x[3:4], s[3:4], 8, torch.ones(1, 4, dtype=torch.bool, device="cuda"), 5)
    for score in (-math.inf, math.nan, math.inf):  # finished, and dead all the same
        check(x[4:5], torch.full((1, 4), score, device="cuda"), 8, torch.ones(1, 4, dtype=torch.bool, device="cuda"), 2999)


def test_select_far_scores():
    """Logits and scores far from 0 that cancel: the comparison in 64 bits decides."""
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(2, 64, 3001, generator=g, device="cuda") * 0.01
    x += torch.linspace(-3e4, 3e4, 64, device="cuda")[None, :, None]
    check(x, -1e3 * torch.rand(2, 64, generator=g, device="cuda"), 33)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("skip", [0, 1, 3, 8])
@pytest.mark.parametrize("pad", [0, 1, 24])
def test_select_strides(dtype, skip, pad):
    """Rows that start anywhere: views of a wider buffer whose other values are NaN."""
    vocab, g = 20011, torch.Generator(device="cuda").manual_seed(3)
    buf = torch.full((3 * 4 * (vocab + pad) + 64,), math.nan, dtype=dtype, device="cuda")
    x = buf[skip:skip + 12 * (vocab + pad)].view(3, 4, vocab + pad)[..., :vocab]
    x.copy_((torch.randn(3, 4, vocab, generator=g, device="cuda") * 2).to(dtype))
    check(x, -torch.rand(3, 4, generator=g, device="cuda"), 9)


def test_select_one_workspace_and_given_outputs():
    ws = gdn.gdn_beam_workspace(8, 8, 70000, 64)
    ws.fill_(255)
    g = torch.Generator(device="cuda").manual_seed(4)
    first = []
    for again in range(2):
        for i, (n, w, v, top) in enumerate([(8, 8, 70000, 8), (1, 3, 4000, 64), (2, 1, 65000, 1)]):
            x = torch.randn(n, w, v, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda")
            s = torch.zeros(n, w, device="cuda")
            out = (torch.empty(n, top, device="cuda"), torch.empty(n, top, dtype=torch.int32, device="cuda"),
                   torch.empty(n, top, dtype=torch.int32, device="cuda"))
            got = gdn.gdn_beam_select(x, s, top, scores_out=out[0], parents=out[1], tokens=out[2], workspace=ws)
            assert all(a is b for a, b in zip(got, out))
            if again:
                assert all(torch.equal(a, b) for a, b in zip(first[i], out))
            else:
                first.append(out)
                check(x, s, top, workspace=ws)


def test_a_level_of_a_tree_and_back():
    """Beam by beam the same as together, captured and replayed."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(3, 4, 9001, generator=g, device="cuda")
    s = -torch.rand(3, 4, generator=g, device="cuda")
    ws = gdn.gdn_beam_workspace(3, 4, 9001, 6)
    want = [t.clone() for t in gdn.gdn_beam_select(x, s, 6, workspace=ws)]
    for i in range(3):
        alone = gdn.gdn_beam_select(x[i:i + 1], s[i:i + 1], 6)
        assert torch.equal(alone[1][0], want[1][i]) and torch.equal(alone[2][0], want[2][i])
    x2, s2 = torch.zeros_like(x), torch.zeros_like(s)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = gdn.gdn_beam_select(x2, s2, 6, workspace=ws)
    x2.copy_(x), s2.copy_(s)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


# ------------------------------------------------------------------ reordering

@pytest.mark.parametrize("dtype,tail", [
    (torch.float32, (4, 128, 128)), (torch.bfloat16, (3, 640)), (torch.int32, (7,)), (torch.int32, (1,)),
    (torch.uint8, (2052,)), (torch.float32, (129,)), (torch.float64, (2, 3))])
@pytest.mark.parametrize("layers,groups,beams", [(1, 1, 1), (1, 3, 2), (2, 2, 8), (3, 1, 64), (2, 5, 33)])
def test_reorder(dtype, tail, layers, groups, beams):
    rng = np.random.default_rng(beams)
    x = torch.randint(0, 250, (layers, groups * beams) + tail, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    for parents in (rng.integers(0, beams, (groups, beams)), np.tile(np.arange(beams), (groups, 1)),
                    np.tile(np.arange(beams)[::-1], (groups, 1)), np.full((groups, beams), beams - 1),
                    np.tile((np.arange(beams) + 1) % beams, (groups, 1))):
        p = torch.tensor(np.ascontiguousarray(parents), dtype=torch.int32).cuda()
        at = (torch.arange(groups)[:, None] * beams + p.cpu()).flatten()
        want = x.cpu()[:, at]
        assert gdn.gdn_beam_reorder(x, p) is x
        assert torch.equal(x.cpu(), want)


def test_reorder_entries_out_of_range_stay():
    x = torch.arange(24, dtype=torch.float32, device="cuda").view(1, 6, 4)
    p = torch.tensor([[2, -1, 7], [1, 1 << 30, -(1 << 31)]], dtype=torch.int32, device="cuda")
    want = x.cpu()[:, [2, 1, 2, 4, 4, 5]]
    assert torch.equal(gdn.gdn_beam_reorder(x, p).cpu(), want)


def test_reorder_unaligned_rows():
    buf = torch.arange(1 + 6 * 36, dtype=torch.float32, device="cuda")
    x = buf[1:].view(1, 6, 36)
    want = x.cpu()[:, [1, 0, 0, 5, 5, 3]]
    got = gdn.gdn_beam_reorder(x, torch.tensor([[1, 0, 0], [2, 2, 0]], dtype=torch.int32, device="cuda"))
    assert torch.equal(got.cpu(), want) and buf[0] == 0


def test_empty_calls():
    e = torch.empty
    out = gdn.gdn_beam_select(e(0, 4, 100, device="cuda"), e(0, 4, device="cuda"), 3)
    assert [tuple(x.shape) for x in out] == [(0, 3)] * 3
    gdn.gdn_beam_reorder(e(0, 4, 8, device="cuda"), torch.zeros(2, 2, dtype=torch.int32, device="cuda"))
    gdn.gdn_beam_reorder(e(2, 4, 0, device="cuda"), torch.zeros(2, 2, dtype=torch.int32, device="cuda"))
