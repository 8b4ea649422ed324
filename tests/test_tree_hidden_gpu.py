"""Trees of drafts: what a node does not see does not matter."""
import pytest
import torch

import gated_deltanet_linear_05_gb300 as gdn
from attn_testlib import Batch
from tree_testlib import DeltaBatch, attention, packed, paths, trees

pytestmark = pytest.mark.gpu


def hidden_from(parents, changed):
    """Nodes that see none of `changed`."""
    return [i for i, path in enumerate(paths(parents)) if not set(path) & set(changed)]


@pytest.mark.parametrize("d,page", [(128, 16), (256, 64)])
@pytest.mark.parametrize("t,context", [(40, 0), (40, 70), (64, 3000), (5, 12)])
def test_attention_does_not_see_hidden_nodes(d, page, t, context):
    """Whatever finite keys and values the nodes have that a row does not see: it is what the definition says without them,
    to the bound that counts the probabilities' rounding to bf16 and the output's.  (Not to the bit: the power that a row's
    probabilities are relative to moves with those of its warp's other rows, and their rounding with it; the row's result
    is relative to the same power throughout.)  Their weights are 0 and not small: the least of bf16, 2^-133, of 3e38 would show."""
    b = Batch([t, 9], [t + context, 30], 4, 2, d, page, seed=51)
    parents = trees(b.t, 51, ("bushy",))
    changed = [t - 1, t // 2, t // 3]
    for j in changed:
        at = context + j
        where = b.pages[0][at // page], slice(None), at % page
        b.k_cache[where] = 90 * torch.randn(2, d, generator=torch.Generator().manual_seed(j)).to(b.k_cache)
        b.v_cache[where] = 3e38
    o = gdn.gdn_tree_attention(b.q, b.k_cache, b.v_cache, b.page_table, b.kv_lens, b.cu, packed(parents)).cpu().double()
    want, bound, _ = attention(b, parents)
    same = hidden_from(parents[0], changed) + list(range(t, t + 9))
    assert len(same) > 10 and ((o - want).abs() <= bound + 1e-6)[same].all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,chunk", [(16, 16), (30, 32), (64, 64)])
def test_the_delta_rule_does_not_see_hidden_nodes(dtype, t, chunk):
    b = DeltaBatch([t, 9], 1, 2, dtype, seed=52, kinds=("bushy",))
    before = gdn.gdn_verify_tree(*b.args(), chunk=chunk)
    changed = [t - 1, t // 2, t // 3]
    for x, scale in ((b.q, 9), (b.k, 9), (b.v, 1e6)):
        x[changed] = (scale * torch.randn(x[changed].shape, generator=torch.Generator().manual_seed(1))).to(x)
    b.g[changed] = -3.0
    b.beta[changed] = 0.75
    after = gdn.gdn_verify_tree(*b.args(), chunk=chunk)
    same = hidden_from(b.parents[0], changed) + list(range(t, t + 9))
    for x, y in zip(before, after):
        assert torch.equal(x[same], y[same]) and not torch.equal(x[changed], y[changed])
