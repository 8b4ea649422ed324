"""Trees of drafts on the GPU: attention and the delta rule against their definitions in 64 bits."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_05_gb300 as gdn
from attn_testlib import Batch
from tree_testlib import DeltaBatch, attention, delta_rule, packed, paths, trees

pytestmark = pytest.mark.gpu

# what the layer is held to in float32, relative to the rms (dot products of 128 terms and sums over at most
# 64 nodes: some 200 roundings of 2^-24 of terms that are at most a few times the rms)
LAYER_F32 = 1e-4


def attend(b, parents, **kw):
    lse = torch.full(b.q.shape[:2], float("nan"), device="cuda")
    if b.prefix:
        kw.update(prefix_table=b.prefix_table, prefix_len=b.prefix)
    o = gdn.gdn_tree_attention(b.q, b.k_cache, b.v_cache, b.page_table, b.kv_lens, b.cu, packed(parents),
                               gate=b.gate, lse=lse, **kw)
    return o, lse


def check_attention(b, parents, scale=None, **kw):
    o, lse = attend(b, parents, scale=scale, **kw)
    want, bound, want_lse = attention(b, parents, scale)
    err = (o.cpu().double() - want).abs()
    assert (err <= bound + 1e-6).all(), float((err - bound).max())
    lse = lse.cpu().double()
    none = torch.isinf(want_lse)
    assert (lse[none] == -float("inf")).all() and (o.cpu()[none] == 0).all()
    # scores: products of 128 or 256 terms in float32; the exponential and the logarithm a few 2^-22
    assert ((lse - want_lse)[~none].abs() <= 2.0 ** -16 * (1 + want_lse[~none].abs())).all()
    assert gdn.gdn_device_status() == 0
    return o


ATTENTION = [
    # t, lens, hq, hkv, d, page, prefix, gate
    ([1], [1], 1, 1, 128, 16, 0, False),
    ([64], [64], 4, 2, 128, 16, 0, False),
    ([64], [64], 4, 2, 256, 64, 0, True),
    ([5, 0, 17, 1, 33], [5, 40, 140, 128, 161], 4, 1, 128, 16, 0, True),
    ([16, 63, 2, 64], [127, 200, 129, 1000], 6, 2, 128, 32, 0, False),
    ([16, 63, 2, 64], [127, 200, 129, 1000], 6, 2, 256, 32, 0, True),
    ([64, 64, 64], [192, 256, 191], 16, 1, 128, 128, 0, False),
    ([40, 7], [3000, 2222], 32, 2, 128, 64, 0, False),       # parts joined
    ([50, 64], [2500, 4001], 16, 2, 256, 64, 0, True),
    ([33] * 40, [33 + 13 * i for i in range(40)], 8, 8, 128, 16, 0, False),
    ([9, 30, 1], [9, 77, 300], 8, 2, 128, 16, 200, False),   # behind a prefix
    ([9, 30, 1], [9, 77, 300], 8, 2, 256, 64, 129, True),
    ([3, 64], [3, 64], 5, 1, 128, 32, 5, True),
    ([30, 12, 64], [20, 0, 63], 4, 2, 128, 16, 0, False),    # fewer keys than nodes
    ([64, 20], [64, 300], 128, 1, 128, 16, 0, False),        # one token to a row tile
]


@pytest.mark.parametrize("case", range(len(ATTENTION)))
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_attention(case, seed):
    t, lens, hq, hkv, d, page, prefix, gate = ATTENTION[case]
    b = Batch(t, lens, hq, hkv, d, page, prefix, gate, seed=seed + 10 * case)
    check_attention(b, trees(t, seed))


@pytest.mark.parametrize("scale", [0.0, -0.07, 0.3])
def test_attention_scales(scale):
    b = Batch([20, 45], [100, 260], 4, 2, 128, 16, seed=3)
    check_attention(b, trees(b.t, 3), scale)


def test_attention_strides():
    b = Batch([20, 45], [100, 260], 4, 2, 128, 16, gate=True, seed=4, q_pad=8, page_pad=64)
    check_attention(b, trees(b.t, 4))


def test_attention_chain_is_causal():
    """A chain is the causal order of the drafts' call, to the bit where the same keys are cut alike."""
    b = Batch([16, 33, 64], [400, 33, 900], 8, 2, 128, 16, seed=5)
    got, _ = attend(b, trees(b.t, 0, ("chain",)))
    want = gdn.gdn_paged_attention(b.q, b.k_cache, b.v_cache, b.page_table, b.kv_lens, b.cu)
    assert ((got.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 2.0 ** -8 * 0.2).all()


@pytest.mark.parametrize("prefix", [0, 100])
def test_attention_leaves_other_rows(prefix):
    """Rows behind the last sequence stay as they were; hidden nodes do not matter, whatever they hold."""
    b = Batch([20, 30], [100, 30], 4, 2, 128, 16, prefix=prefix, seed=6)
    parents = trees(b.t, 6, ("bushy",))
    cu = b.cu.clone()
    q = torch.cat([b.q, torch.full_like(b.q[:7], float("nan"))])
    kw = dict(prefix_table=b.prefix_table, prefix_len=prefix) if prefix else {}
    o = torch.full_like(q, 7.0)
    gdn.gdn_tree_attention(q, b.k_cache, b.v_cache, b.page_table, b.kv_lens, cu, packed(parents + [[0] * 7]), o=o, **kw)
    assert (o[50:] == 7).all()
    want, bound, _ = attention(b, parents)
    assert ((o[:50].cpu().double() - want).abs() <= bound + 1e-6).all()


def test_attention_one_large_workspace():
    """Calls of several shapes with one workspace, and again: the same bits."""
    ws = gdn.gdn_attn_workspace(40, 1500, 16, 16, 256, prefix_len=512)
    first = []
    for again in range(2):
        for i, (t, lens, hq, hkv, d, page, prefix, gate) in enumerate(ATTENTION[3:12]):
            b = Batch(t, lens, hq, hkv, d, page, prefix, gate, seed=i)
            o, lse = attend(b, trees(t, i), workspace=ws)
            if again:
                assert torch.equal(o, first[i][0]) and torch.equal(lse, first[i][1])
            else:
                first.append((o, lse))


def test_attention_captured():
    """Captured, then replayed with other lengths, trees and queries in place."""
    a, b = (Batch([20, 9, 40], lens, 8, 2, 128, 16, gate=True, seed=s) for s, lens in ((7, [90, 500, 41]), (8, [300, 10, 200])))
    most = max(a.page_table.shape[1], b.page_table.shape[1])
    pages = max(a.k_cache.shape[0], b.k_cache.shape[0])
    pa, pb = trees(a.t, 7), trees(a.t, 8)
    s = dict(q=a.q.clone(), gate=a.gate.clone(), up=packed(pa), lens=a.kv_lens.clone(),
             table=torch.zeros(3, most, dtype=torch.int32, device="cuda"))
    cache = [torch.full((pages,) + a.k_cache.shape[1:], float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ws = gdn.gdn_attn_workspace(3, 69, 8, 2, 128)

    def put(x, p):
        s["q"].copy_(x.q), s["gate"].copy_(x.gate), s["up"].copy_(packed(p)), s["lens"].copy_(x.kv_lens)
        s["table"][:, :x.page_table.shape[1]].copy_(x.page_table)
        for c, y in zip(cache, (x.k_cache, x.v_cache)):
            c[:y.shape[0]].copy_(y)

    def call():
        return gdn.gdn_tree_attention(s["q"], *cache, s["table"], s["lens"], a.cu, s["up"], gate=s["gate"], workspace=ws)

    put(a, pa)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = call()
    for x, p in ((b, pb), (a, pa)):
        put(x, p)
        graph.replay()
        want, bound, _ = attention(x, p)
        assert ((o.cpu().double() - want).abs() <= bound + 1e-6).all()


# ------------------------------------------------------------------ the delta rule

def relative(got, want):
    return float((got.cpu().double() - want).abs().max() / want.square().mean().sqrt())


DELTA = [
    # t, chunk, hk, hv
    ([1], 16, 1, 1), ([16], 16, 1, 2), ([3, 0, 16, 7], 16, 2, 2), ([9, 1], 32, 1, 4), ([32, 17, 0, 31], 32, 2, 4),
    ([64], 64, 1, 1), ([64, 33, 5, 0, 49], 64, 2, 6), ([2, 60], 64, 3, 3), ([16] * 30, 16, 4, 8),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(DELTA)))
@pytest.mark.parametrize("state", [True, False])
def test_delta_rule(case, dtype, state):
    t, chunk, hk, hv = DELTA[case]
    b = DeltaBatch(t, hk, hv, dtype, seed=case, state=state)
    before = None if b.state is None else b.state.clone()
    o = torch.empty(b.v.shape, device="cuda")
    _, delta = gdn.gdn_verify_tree(*b.args(), o=o, chunk=chunk)
    want_o, want_d, _ = delta_rule(b)
    assert relative(o, want_o) <= LAYER_F32 and relative(delta, want_d) <= LAYER_F32
    if state:
        assert torch.equal(before, b.state)
    if dtype == "bf16":  # its own type: the same, rounded once
        o16, delta16 = gdn.gdn_verify_tree(*b.args(), chunk=chunk)
        assert torch.equal(o16, o.bfloat16()) and torch.equal(delta16, delta)
    assert gdn.gdn_device_status() == 0


@pytest.mark.parametrize("kind", ["chain", "star", "bushy", "wild"])
@pytest.mark.parametrize("decay", [0.01, 40.0])
def test_delta_rule_decays(kind, decay):
    """States carried far, and decays that underflow along a path."""
    b = DeltaBatch([64, 40, 64], 2, 4, "bf16", seed=11, decay=decay, kinds=(kind,))
    o, delta = gdn.gdn_verify_tree(*b.args(), o=torch.empty(b.v.shape, device="cuda"))
    want_o, want_d, _ = delta_rule(b)
    assert relative(o, want_o) <= LAYER_F32 and relative(delta, want_d) <= LAYER_F32


@pytest.mark.parametrize("scale", [1e-3, 1e3])
def test_delta_rule_large_and_small_states(scale):
    """The state's 24 bits count at any magnitude."""
    b = DeltaBatch([30, 32], 1, 2, "bf16", seed=12)
    b.state *= scale
    b.v = (b.v.float() * scale).bfloat16()
    o, delta = gdn.gdn_verify_tree(*b.args(), o=torch.empty(b.v.shape, device="cuda"), chunk=32)
    want_o, want_d, _ = delta_rule(b)
    assert relative(o, want_o) <= LAYER_F32 and relative(delta, want_d) <= LAYER_F32


def test_delta_rule_leaves_other_rows():
    b = DeltaBatch([5, 20], 1, 2, "bf16", seed=13, extra=6)
    for x in (b.q, b.k, b.v, b.g, b.beta):
        x[25:] = float("nan")
    o, delta = torch.full_like(b.v, 7.0), torch.full(b.v.shape, 7.0, device="cuda")
    gdn.gdn_verify_tree(*b.args(), o=o, delta=delta, chunk=32)
    assert (o[25:] == 7).all() and (delta[25:] == 7).all()
    assert torch.isfinite(o[:25]).all()


def test_delta_rule_chain_is_the_drafts_block():
    """A chain gives the linear block's outputs and deltas, to the bound of that call's fp16 products."""
    b = DeltaBatch([16, 9, 12], 2, 4, "bf16", seed=14, kinds=("chain",))
    o, delta = gdn.gdn_verify_tree(*b.args(), o=torch.empty(b.v.shape, device="cuda"), chunk=16)
    o2, _, delta2 = gdn.gdn_verify_block_capture(b.q, b.k, b.v, b.g, b.beta, b.state, torch.empty_like(b.state), b.cu,
                                                 o=torch.empty(b.v.shape, device="cuda"))
    for x, y in ((o, o2), (delta, delta2)):
        assert float((x - y).abs().max() / x.square().mean().sqrt()) <= 2e-2


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_accepted_path(dtype):
    """The state after an accepted path: gdn_state_rollback on the path's rows."""
    b = DeltaBatch([20, 33, 7, 64], 2, 4, dtype, seed=15, kinds=("bushy", "narrow"))
    _, delta = gdn.gdn_verify_tree(*b.args())
    _, _, states = delta_rule(b)
    leaves = [19, 30, 0, 63]
    rows, first = [], np.cumsum([0] + b.t)
    taken = [paths(up)[leaf] for up, leaf in zip(b.parents, leaves)]
    for at, path in zip(first, taken):
        rows += [int(at) + i for i in path]
    rows = torch.tensor(rows, device="cuda")
    lens = torch.tensor([len(p) for p in taken], dtype=torch.int32, device="cuda")
    cu = torch.cat([lens.new_zeros(1), lens.cumsum(0).to(torch.int32)])
    out = gdn.gdn_state_rollback(b.k[rows], b.g[rows], delta[rows], b.state, lens, torch.empty_like(b.state), cu)
    want = torch.stack([s[leaf] for s, leaf in zip(states, leaves)])
    assert relative(out, want) <= LAYER_F32


def test_delta_rule_captured():
    a, b = (DeltaBatch([30, 12], 1, 2, "bf16", seed=s) for s in (16, 17))
    st = [x.clone() for x in a.args()]
    o = torch.empty(a.v.shape, device="cuda")
    delta = torch.empty_like(o)
    gdn.gdn_verify_tree(*st, o=o, delta=delta, chunk=32)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_verify_tree(*st, o=o, delta=delta, chunk=32)
    for x in (b, a):
        for y, z in zip(st, x.args()):
            y.copy_(z)
        graph.replay()
        want_o, want_d, _ = delta_rule(x)
        assert relative(o, want_o) <= LAYER_F32 and relative(delta, want_d) <= LAYER_F32
