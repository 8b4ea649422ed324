"""The sums of powers of gdn_beam_select: the same for a request whatever the number of requests, and as exact for long rows
as for short ones."""
import pytest
import torch

import gated_deltanet_linear_05_gb300 as gdn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("groups,beams,vocab,top", [
    (64, 8, 150001, 8), (64, 8, 150000, 8), (300, 1, 70000, 3), (40, 48, 33333, 48), (100, 64, 40000, 4)])
def test_a_request_alone_and_in_a_batch(dtype, groups, beams, vocab, top):
    """To the bit, scores too."""
    g = torch.Generator(device="cuda").manual_seed(vocab + top)
    x = (torch.randn(groups, beams, vocab, generator=g, device="cuda") * 3).to(dtype)
    s = -5 * torch.rand(groups, beams, generator=g, device="cuda")
    every = gdn.gdn_beam_select(x, s, top)
    for a, b in ((0, 1), (groups - 1, groups), (3, 5), (1, groups // 2)):
        some = gdn.gdn_beam_select(x[a:b], s[a:b], top)
        for i, j in zip(some, every):
            assert torch.equal(i, j[a:b])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [0, 5, 8])
def test_a_row_alone_and_among_others(dtype, pad):
    """A row's order of sums goes by where it starts, also where its stride has no meaning: of the rows here some or all
    start at multiples of 16 bytes."""
    buf = torch.randn(64, 1, 20011 + pad, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda").to(dtype)
    x, s = buf[..., :20011], torch.zeros(64, 1, device="cuda")
    every = gdn.gdn_beam_select(x, s, 64)
    for i in range(64):
        start = x[i].data_ptr() % 16
        if pad == 5 or start:  # 20016: every row starts at a multiple of 16 bytes
            assert start == 0 or pad != 5
            assert all(torch.equal(a[0], b[i]) for a, b in zip(gdn.gdn_beam_select(x[i:i + 1], s[i:i + 1], 64), every))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("groups,beams,vocab", [(1, 1, 1 << 24), (3, 2, (1 << 22) + 1), (500, 1, 1 << 20), (150, 32, 131072)])
@pytest.mark.parametrize("kind", ["flat", "rising", "falling", "normal"])
def test_long_rows(dtype, groups, beams, vocab, kind):
    """Of a score, relative to the sum of powers: a power 2^-22 (ex2) and its exponent's rounding 2^-25; two factors of 2^-22
    each, from its thread's largest to the step's and from there to the row's; 23 roundings of 2^-24 on its way into the row's
    sum: some 36 of 2^-24, 2^-21 + 34 of them allowed; and 2^-24 of the score."""
    i = torch.arange(vocab, device="cuda", dtype=torch.float32)
    x = {"flat": torch.full_like(i, -0.3), "rising": i * (20.0 / vocab), "falling": i * (-20.0 / vocab),
         "normal": torch.randn(vocab, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")}[kind]
    x[vocab // 3] = 0.0
    x = x.to(dtype)
    want = torch.log_softmax(x.double(), 0)
    rows = x.expand(groups, beams, vocab).contiguous()
    s = -torch.arange(beams, device="cuda", dtype=torch.float32).expand(groups, beams).contiguous()
    score, parent, token = gdn.gdn_beam_select(rows, s, 4)
    exact = s.gather(1, parent.long()).double() + want[token.long()]
    assert ((score.double() - exact).abs() <= 2.0 ** -21 + 34 * 2.0 ** -24 + 2.0 ** -24 * exact.abs()).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_kept_workspace_serves_a_shrinking_batch(dtype):
    """As requests end; what lies behind the workspace stays as it was."""
    size = gdn.gdn_beam_workspace(40, 8, 151936, 8).numel()
    room = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
    x = torch.randn(40, 8, 151936, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(dtype)
    s = torch.zeros(40, 8, device="cuda")
    want = gdn.gdn_beam_select(x, s, 8)
    for n in (40, 39, 17, 5, 4, 3, 2, 1):
        got = gdn.gdn_beam_select(x[:n], s[:n], 8, workspace=room[:size])
        assert all(torch.equal(a, b[:n]) for a, b in zip(got, want))
    assert (room[size:] == 255).all()
