"""Calls for trees and beams that the contract allows at its borders: rows that are not finite, masks of the
type's lowest value, offsets past 32 bits, two streams at once, sequences beside a malformed one."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_05_gb300 as gdn
from attn_testlib import Batch
from tree_testlib import DeltaBatch, attention, delta_rule, packed, trees

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,page", [(128, 16), (256, 64)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("context", [0, 70, 3000])
def test_attention_of_rows_that_are_not_finite(d, page, value, context):
    """A query that is not finite makes its own row NaN and no other; hidden nodes' keys are not looked at by
    rows that do not see them."""
    t = [40, 9]
    b = Batch(t, [x + context for x in t], 4, 2, d, page, seed=21)
    parents = trees(t, 21, ("bushy",))
    b.q[7, 1, 3] = value
    b.q[45, 0] = value
    lse = torch.zeros(b.q.shape[:2], device="cuda")
    o = gdn.gdn_tree_attention(b.q, b.k_cache, b.v_cache, b.page_table, b.kv_lens, b.cu, packed(parents), lse=lse)
    bad = torch.zeros(b.q.shape[:2], dtype=torch.bool)
    bad[7, 1] = bad[45, 0] = True
    b.q[7, 1, 3] = 0
    b.q[45, 0] = 0
    want, bound, _ = attention(b, parents)
    o = o.cpu().double()
    assert ((o - want).abs() <= bound + 1e-6)[~bad].all()
    # scores of +-inf in every sign or NaN: the row has one of +inf or NaN but for luck with a few keys
    assert torch.isnan(o[45, 0]).all() and torch.isnan(lse.cpu()[45, 0])
    assert torch.isnan(o[7, 1]).all() or context == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_select_with_masks_of_the_lowest_value(dtype):
    """Tokens masked by the type's lowest finite value rank after all others and before -inf."""
    low = torch.finfo(dtype).min
    x = torch.randn(2, 3, 700, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(dtype)
    x[0, :, 4:] = low
    x[1, :, 2:] = -float("inf")
    x[1, 0, 9] = low
    s = torch.tensor([[-1.0, -2.0, -3.0]] * 2, device="cuda")
    score, parent, token = gdn.gdn_beam_select(x, s, 20)
    every = s[..., None].double() + torch.log_softmax(x.double(), -1)
    assert sorted((parent[0, :12] * 700 + token[0, :12]).tolist()) == sorted(
        w * 700 + t for w in range(3) for t in range(4))
    # Of a score: its beam's sum of powers (exact to 2^-22, some 85 roundings of 2^-24 relative to the sum, which the
    # logarithm makes absolute) and its own rounding to float32, half a step, 2^-24 of it.
    best, at = torch.sort(every.flatten(1), dim=1, descending=True, stable=True)
    tol = 2.0 ** -22 + 85 * 2.0 ** -24 + 2.0 ** -24 * best[0, :20].abs()
    assert ((score[0].double() - best[0, :20]).abs() <= tol).all()
    # the masked ones' scores, equal in 64 bits (a step there is 2^74), come in order of place
    assert torch.equal((parent * 700 + token)[0, 12:].long(), torch.arange(4, 12, device="cuda"))
    assert torch.equal((parent * 700 + token)[1, :7].long(), at[1, :7])
    assert (score[1, 7:] == -float("inf")).all()
    assert torch.equal((parent * 700 + token)[1, 7:].long(), at[1, 7:20])


def test_select_far_rows():
    """Logits of more than 2^32 bytes, the largest vocabulary."""
    vocab = 1 << 24
    x = torch.zeros(65, 2, vocab, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(3)
    where = rng.integers(0, vocab, (65, 2, 3))
    for g in (0, 31, 64):
        for w in range(2):
            for i, t in enumerate(where[g, w]):
                x[g, w, int(t)] = 30 + 2 * i + w
    score, parent, token = gdn.gdn_beam_select(x, torch.zeros(65, 2, device="cuda"), 6)
    for g in (0, 31, 64):
        every = torch.log_softmax(x[g].double(), -1).flatten()
        at = torch.topk(every, 6).indices
        assert torch.equal(parent[g] * vocab + token[g], at.int())
    for g in (1, 63):  # equal everywhere: by place
        assert parent[g].tolist() == [0] * 6 and token[g].tolist() == list(range(6))


def test_reorder_far_rows():
    x = torch.empty(1, 4, (1 << 28) + 4, dtype=torch.float32, device="cuda")
    for w in range(4):
        x[0, w].fill_(w)
        x[0, w, -1] = 10 + w
    gdn.gdn_beam_reorder(x, torch.tensor([[3, 1, 1, 0]], dtype=torch.int32, device="cuda"))
    for w, p in enumerate((3, 1, 1, 0)):
        assert x[0, w, -1] == 10 + p and (x[0, w, :-1] == p).all()


def test_two_streams_at_once():
    """Calls on two streams, each with a workspace of its own: what they give one after another."""
    tree = [Batch([30, 12], [400, 50], 8, 2, 128, 16, seed=s) for s in (31, 32)]
    delta = [DeltaBatch([30, 12], 2, 4, "bf16", seed=s) for s in (31, 32)]
    up = [packed(trees([30, 12], s, ("bushy",))) for s in (31, 32)]
    logits = [torch.randn(2, 4, 50001, device="cuda") for _ in range(2)]
    scores = torch.zeros(2, 4, device="cuda")
    ws = [(gdn.gdn_attn_workspace(2, 42, 8, 2, 128), gdn.gdn_beam_workspace(2, 4, 50001, 8)) for _ in range(2)]

    def calls(i, stream=None):
        b = tree[i]
        kw = {} if stream is None else dict(stream=stream)
        return (gdn.gdn_tree_attention(b.q, b.k_cache, b.v_cache, b.page_table, b.kv_lens, b.cu, up[i], workspace=ws[i][0], **kw),
                *gdn.gdn_verify_tree(*delta[i].args(), chunk=32, **kw),
                *gdn.gdn_beam_select(logits[i], scores, 8, workspace=ws[i][1], **kw))

    want = [calls(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        got = [None, None]
        for i in range(2):
            got[i] = calls(i, streams[i])
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))


def test_sequences_beside_a_tree_of_too_many_nodes():
    """More nodes than a tree may have, or than `chunk`: unspecified for that sequence, the others as ever."""
    t = [20, 90, 33]
    b = Batch(t, [100, 90, 300], 4, 2, 128, 16, seed=41)
    parents = trees(t, 41, ("bushy",))
    o = gdn.gdn_tree_attention(b.q, b.k_cache, b.v_cache, b.page_table, b.kv_lens, b.cu, packed(parents)).cpu().double()
    want, bound, _ = attention(b, parents)
    for rows in (slice(0, 20), slice(110, 143)):
        assert ((o - want).abs() <= bound + 1e-6)[rows].all()
    d = DeltaBatch(t, 1, 2, "bf16", seed=42)
    o, delta = gdn.gdn_verify_tree(*d.args(), o=torch.empty(d.v.shape, device="cuda"))
    want_o, want_d, _ = delta_rule(d)
    for rows in (slice(0, 20), slice(110, 143)):
        for x, y in ((o, want_o), (delta, want_d)):
            assert ((x.cpu().double() - y)[rows].abs().max() / y[rows].square().mean().sqrt()) <= 1e-4


def test_malformed_cu_seqlens_stays_inside():
    """Decreasing or too large: other rows may hold anything, nothing outside the outputs is touched."""
    d = DeltaBatch([20, 20], 1, 2, "bf16", seed=43)
    b = Batch([20, 20], [60, 60], 4, 2, 128, 16, seed=43)
    up = packed(d.parents)
    for bad in ([0, 30, 10], [0, 500, 40], [-7, 20, 1 << 30], [40, 40, 0]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        room = torch.full((44, 2, 128), 7.0, device="cuda")
        wide = torch.full((44, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        gdn.gdn_verify_tree(d.q, d.k, d.v, d.g, d.beta, d.state, cu, up, o=room[2:42].bfloat16().contiguous(), delta=room[2:42])
        gdn.gdn_tree_attention(b.q, b.k_cache, b.v_cache, b.page_table, b.kv_lens, cu, up, o=wide[2:42])
        assert (room[:2] == 7).all() and (room[42:] == 7).all() and (wide[:2] == 7).all() and (wide[42:] == 7).all()
    assert gdn.gdn_device_status() == 0


def test_a_bad_value_stays_in_its_sequence():
    d = DeltaBatch([20, 30, 9], 1, 2, "f32", seed=44)
    d.v[25, 0, 5] = float("nan")
    d.k[30] = float("inf")
    o, delta = gdn.gdn_verify_tree(*d.args())
    ok = [slice(0, 20), slice(50, 59)]
    want_o, want_d, _ = delta_rule(d)
    for rows in ok:
        for x, y in ((o, want_o), (delta, want_d)):
            assert ((x.cpu().double() - y)[rows].abs().max() / y[rows].square().mean().sqrt()) <= 1e-4
