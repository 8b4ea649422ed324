"""GPU parity of the append with rotary positions and of the residual + RMS norm, against their
definitions in 64 bits.  Bounds count the roundings: bf16 outputs half a step (2^-8 relative)
on top of the float32 arithmetic; e4m3 codes half a step (2^-4 relative, or half of the
smallest step) of the value over the stored scale."""
import math

import numpy as np
import pytest
import torch

from attn_testlib import BF16_HALF

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_deltanet_linear_05_gb300 import build
    build.build()


def _bf16(*shape, g, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)


def _append_case(t, lens, hq, hkv, d, page, rot, axes=0, norm=False, fused=False, seed=0,
                 first=0, prefix=0, contiguous=False):
    """Runs the call; returns what it gave and what it should have given with the bound."""
    import gated_deltanet_linear_05_gb300 as gdn
    g = torch.Generator().manual_seed(seed)
    n, tokens = len(t), sum(t)
    pages = sum(-(-x // page) for x in lens) + 3
    table = torch.full((n, max([1] + [-(-x // page) for x in lens])), -1, dtype=torch.int32)
    order = torch.randperm(pages, generator=g).tolist()
    for i, x in enumerate(lens):
        m = -(-x // page)
        table[i, :m] = torch.tensor(order[:m], dtype=torch.int32)
        order = order[m:]
    if fused:
        row = _bf16(tokens, (hq + 2 * hkv) * d, g=g, std=2.0)
        q, k, v = (x.unflatten(1, (-1, d)) for x in row.split([hq * d, hkv * d, hkv * d], 1))
    else:
        q, k, v = (_bf16(tokens, h, d, g=g, std=2.0) for h in (hq, hkv, hkv))
    kc, vc = (_bf16(pages, hkv, page, d, g=g) for _ in range(2))
    freq = np.array([1e6 ** (-2.0 * i / max(rot, 1)) for i in range(rot // 2)])
    if rot >= 32:
        freq[1] = 2.75  # more than one radian, and a slow one
        freq[2] = 1e-12
    qn, kn = ((1 + 0.2 * torch.randn(d, generator=g)) if norm else None for _ in range(2))
    place = np.concatenate([np.arange(l - c, l) for c, l in zip(t, lens)]) if tokens else np.zeros(0, int)
    seq = np.repeat(np.arange(n), t)
    pos = axis = None
    if axes:
        pos = torch.randint(0, 2 ** 31 - 1, (axes, tokens), generator=g, dtype=torch.int32)
        pos[0, :min(3, tokens)] = torch.tensor([0, -5, 2 ** 31 - 1], dtype=torch.int32)[:min(3, tokens)]
        axis = torch.randint(0, axes, (rot // 2,), generator=g, dtype=torch.int32)
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    if fused:
        row = row.cuda()
        dq, dk, dv = (x.unflatten(1, (-1, d)) for x in row.split([hq * d, hkv * d, hkv * d], 1))
    else:
        dq, dk, dv = q.cuda(), k.cuda(), v.cuda()
    dkc, dvc = kc.cuda(), vc.cuda()
    out = gdn.gdn_kv_append(
        dq, dk, dv, dkc, dvc, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
        torch.tensor(freq, dtype=torch.float64).cuda() if rot else None,
        cu_seqlens=None if contiguous else torch.tensor([0] + list(np.cumsum(t)), dtype=torch.int32).cuda(),
        positions=dev(pos), rope_axis=dev(axis), q_norm=dev(qn), k_norm=dev(kn), eps=1e-5,
        prefix_len=prefix)
    torch.cuda.synchronize()
    # the definition; angles modulo a turn in long double (64 bits lose 2^-22 rad at 2^31)
    if pos is None:
        p = (place + prefix)[:, None].repeat(max(rot // 2, 1), 1)
    else:
        p = pos.numpy()[axis.numpy()].T
    ang = p[:, :rot // 2].astype(np.longdouble) * freq.astype(np.longdouble)[None]
    c, s = (torch.from_numpy(f(ang).astype(np.float64)) for f in (np.cos, np.sin))

    def want(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-5) * w.double()
        m = rot // 2
        a, b = x[..., :m], x[..., m:rot]
        y = torch.cat([a * c[:, None] - b * s[:, None], b * c[:, None] + a * s[:, None], x[..., rot:]], -1)
        size = torch.cat([torch.hypot(a, b), torch.hypot(a, b), x[..., rot:].abs()], -1)
        # half a bf16 step of the result; cosine, sine and the norm in float32
        return y, BF16_HALF * y.abs() + 2.0 ** -19 * size

    kc2, vc2 = kc.double(), vc.double()
    kb = torch.zeros_like(kc2)
    yk, ek = want(k, kn)
    for i in range(tokens):
        if place[i] < 0:
            continue
        pg, r = int(table[seq[i], place[i] // page]), place[i] % page
        kc2[pg, :, r], kb[pg, :, r], vc2[pg, :, r] = yk[i], ek[i], v[i].double()
    yq, eq = want(q, qn)
    return (out, dkc, dvc), (yq, kc2, vc2), (eq, kb, torch.zeros_like(vc2))


def _within(case):
    for got, ref, bound in zip(*case):
        x = got.cpu().double()
        excess = (x - ref).abs() - bound
        assert excess.numel() == 0 or excess.max().item() <= 1e-30, excess.max().item()


@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (128, 16), (128, 0), (128, 96), (256, 256),
                                   (256, 64), (256, 160)])
@pytest.mark.parametrize("axes", [0, 1, 3])
@pytest.mark.parametrize("norm", [False, True])
def test_append_rotation(d, rot, axes, norm):
    if rot == 0 and axes:
        pytest.skip("no rotation, no axes")
    _within(_append_case([5, 1, 0, 40], [5, 17, 3, 90], 6, 2, d, 16, rot, axes, norm, seed=rot + axes))


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 1), (16, 4), (3, 3)])
def test_append_heads_and_pages(page, hq, hkv):
    _within(_append_case([page + 3, 1, 2 * page], [page + 3, page, 2 * page + 1], hq, hkv, 128, page, 64,
                         fused=True, seed=page + hq))


@pytest.mark.parametrize("n", [1, 3, 200])
def test_append_step(n):
    lens = [(7 * i) % 50 + 1 for i in range(n)]
    _within(_append_case([1] * n, lens, 4, 2, 256, 16, 64, norm=True, fused=True, seed=n, prefix=777,
                         contiguous=True))


@pytest.mark.parametrize("d", [128, 256])
def test_append_head_major(d):
    """Token strides below the head strides give the bits of contiguous rows."""
    import gated_deltanet_linear_05_gb300 as gdn
    g = torch.Generator().manual_seed(81)
    q, k, v = (_bf16(46, h, d, g=g).cuda() for h in (6, 2, 2))
    table = torch.arange(24, dtype=torch.int32).view(4, 6).cuda()
    lens, cu = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([5, 17, 3, 90], [0, 5, 6, 6, 46]))
    freq, w = torch.linspace(1e-4, 1, 32, dtype=torch.float64).cuda(), 1 + 0.1 * torch.arange(d).cuda() / d
    got = []
    for rows in ((q, k, v), [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]):
        kc, vc = (torch.zeros(24, 2, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        got.append((gdn.gdn_kv_append(*rows, kc, vc, table, lens, freq, cu, q_norm=w, k_norm=w), kc, vc))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*got)) and got[0][1].any()


@pytest.mark.parametrize("axes", [0, 3])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("step", [False, True])
def test_append_of_seen_sizes(step, norm, axes):
    """Other values of the same sizes each time: the way through the marshalling module."""
    t, lens = ([1] * 4, [5, 17, 3, 90]) if step else ([5, 1, 3, 40], [5, 17, 3, 90])
    for seed in (82, 83, 84):
        _within(_append_case(t, lens, 6, 2, 128, 16, 64, axes, norm, fused=True, seed=seed, prefix=9,
                             contiguous=step))


def test_append_rows_without_a_place():
    """More tokens than keys: the first tokens are rotated for q but not stored; a sequence of
    no keys stores nothing."""
    _within(_append_case([9, 4, 2], [5, 0, 30], 4, 2, 128, 16, 128, seed=3))


def test_append_many_sequences():
    t = [(i * 5) % 4 for i in range(1500)]
    _within(_append_case(t, [x + i % 9 for i, x in enumerate(t)], 2, 1, 128, 16, 32, seed=4))


def test_append_bad_pages_and_in_place():
    """Entries out of range drop their rows and touch nothing else; q_out may be q."""
    import gated_deltanet_linear_05_gb300 as gdn
    g = torch.Generator().manual_seed(5)
    q, k, v = (_bf16(40, h, 128, g=g).cuda() for h in (4, 2, 2))
    kc, vc = (torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.tensor([[2, 4, -1]], dtype=torch.int32).cuda()
    cu, lens = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([0, 40], [40]))
    want = gdn.gdn_kv_append(q, k, v, kc.clone(), vc.clone(), table, lens, cu_seqlens=cu)
    out = gdn.gdn_kv_append(q, k, v, kc, vc, table, lens, cu_seqlens=cu, q_out=q)
    torch.cuda.synchronize()
    assert out is q and torch.equal(out, want)
    assert torch.equal(kc[2].transpose(0, 1), k[:16]) and torch.equal(vc[2].transpose(0, 1), v[:16])
    for c in (kc, vc):
        assert not c[[0, 1, 3]].any()


# ------------------------------------------------------------------ residual + RMS norm

def _norm_case(rows, cols, dtype, out, group, residual=True, seed=0, mode="plain"):
    import gated_deltanet_linear_05_gb300 as gdn
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(cols, generator=g))).to(dtype)
    r = torch.randn(rows, cols, generator=g).to(dtype) if residual else None
    w = 1 + 0.3 * torch.randn(cols, generator=g)
    dx, dr = x.cuda(), None if r is None else r.cuda()
    kw = {}
    if mode == "in place":
        kw["residual_out"] = dr
    elif mode == "over x":
        kw["residual_out"] = dx
    got = gdn.gdn_add_rmsnorm(dx, dr, w.cuda(), 1e-6, out=out, group=group, **kw)
    torch.cuda.synchronize()
    h = x if r is None else (x.float() + r.float()).to(dtype)
    assert torch.equal(got[-1].cpu(), h)  # one float32 addition and one rounding: exact
    f = h.double()
    y = f / torch.sqrt(f.square().mean(-1, keepdim=True) + 1e-6) * w.double()
    tiny = 2.0 ** -20 * y.abs()  # the sum of squares, root, reciprocal and products in float32
    if out == "same":
        half = BF16_HALF if dtype == torch.bfloat16 else 2.0 ** -24
        assert ((got[0].cpu().double() - y).abs() <= half * y.abs() + tiny).all()
        return
    assert got[0].dtype == torch.float8_e4m3fn
    width = group or cols
    scale = y.abs().unflatten(-1, (-1, width)).amax(-1).clamp(min=1e-12) / 448
    sc = got[1].cpu().double()
    assert sc.shape == scale.shape and ((sc - scale).abs() <= 2.0 ** -20 * scale).all()
    v = y / sc.repeat_interleave(width, -1)
    code = got[0].cpu().float().double()
    # half a step: 2^-4 relative for normal codes, 2^-10 absolute below 2^-6; 2^-19 of the
    # value for the float32 arithmetic, which may move it across a border
    assert ((code - v).abs() <= torch.clamp(v.abs() * 2.0 ** -4, min=2.0 ** -10) + 2.0 ** -19 * v.abs()).all()
    assert (code.abs() <= 448).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out,group", [("same", 0), ("e4m3", 0), ("e4m3", 128)])
@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 1024), (5, 4096), (2, 5120), (400, 2048),
                                       (2, 16384), (1, 65536), (310, 8320)])
def test_norm(rows, cols, dtype, out, group):
    _norm_case(rows, cols, dtype, out, group, seed=rows + cols)


@pytest.mark.parametrize("cols", [8, 24, 136, 4104])
@pytest.mark.parametrize("out", ["same", "e4m3"])
def test_norm_odd_widths(cols, out):
    _norm_case(7, cols, torch.bfloat16, out, 0, seed=cols)


@pytest.mark.parametrize("mode", ["in place", "over x"])
def test_norm_in_place(mode):
    _norm_case(33, 4096, torch.bfloat16, "e4m3", 128, mode=mode)


def test_norm_without_residual():
    _norm_case(9, 2048, torch.bfloat16, "same", 0, residual=False)
    _norm_case(9, 2048, torch.float32, "e4m3", 128, residual=False)


@pytest.mark.parametrize("group", [0, 128])
def test_norm_zero_rows_and_nan(group):
    """A row of zeros has the smallest scale and zero codes; NaN and infinities reach the
    scale and the codes of their row (a NaN its own group's), and no other row."""
    import gated_deltanet_linear_05_gb300 as gdn
    x = torch.ones(4, 512, dtype=torch.bfloat16)
    x[0] = 0
    x[1, 200] = math.nan
    x[2, 300] = math.inf
    y8, scale, h = gdn.gdn_add_rmsnorm(x.cuda(), torch.zeros_like(x).cuda(), torch.ones(512).cuda(), 1e-6,
                                       out="e4m3", group=group)
    torch.cuda.synchronize()
    y, sc = y8.cpu().float(), scale.cpu()
    assert (y[0] == 0).all() and torch.allclose(sc[0], torch.full_like(sc[0], 1e-12 / 448))
    assert y[1].isnan().all() and sc[1].isnan().all()  # the row's norm is NaN
    at = 2 if group else 0
    assert sc[2, at].isnan() and y[2, 300].isnan()  # inf / inf
    assert torch.isfinite(y[3]).all() and (y[3] == 448).all()


@pytest.mark.parametrize("group", [0, 128])
def test_norm_codes_at_ties(group):
    """y = the weights exactly (a row of ones, eps 0), over a scale of 3, 5 and 7: quotients that lie on a
    tie between two codes go to the even one, and every other to the nearest."""
    import gated_deltanet_linear_05_gb300 as gdn
    ties = [17.0, 19.0, 21.0, 27.0, 34.0, 38.0, 46.0, 68.0, 92.0, 232.0, 424.0, 1.0625, 0.5625 + 2.0 ** -5]
    for s in (3.0, 5.0, 7.0):
        w = torch.zeros(512)
        for at in range(0, 512, 128):
            w[at] = 448 * s
            w[at + 1:at + 14] = torch.tensor(ties) * s
            w[at + 14:at + 27] = -torch.tensor(ties) * s
            w[at + 27:at + 100] = torch.linspace(-400, 400, 73) * s
        x = torch.ones(5, 512, dtype=torch.float32, device="cuda")
        y8, scale, _ = gdn.gdn_add_rmsnorm(x, None, w.cuda(), 0.0, out="e4m3", group=group)
        torch.cuda.synchronize()
        assert (scale == s).all()
        want = (w / s).to(torch.float8_e4m3fn).float()  # one float32 quotient, exact where it is a tie
        assert torch.equal(y8.cpu().float(), want.expand(5, -1))


def test_norm_rows_past_32_bits():
    """Rows whose elements lie past 2^31."""
    import gated_deltanet_linear_05_gb300 as gdn
    rows, cols = 33000, 65536
    x = torch.full((rows, cols), 2.0, dtype=torch.bfloat16, device="cuda")
    x[-1] = 3.0
    y, h = gdn.gdn_add_rmsnorm(x, None, torch.ones(cols, device="cuda"), 0.0)
    torch.cuda.synchronize()
    assert h is x and (y[-1] == 1.0).all() and (y[0] == 1.0).all()
