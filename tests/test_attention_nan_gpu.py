"""Queries that are not finite.  softmax of scores that are NaN, or of which one is +inf or all are
-inf, is NaN: such a row has to come out as NaN however the call was cut into parts (a row of
zeros is one that sees no key), and every other row as without it."""
import math

import pytest
import torch

from attn_testlib import Batch, reference
from test_attention_gpu import _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_deltanet_linear_05_gb300 import build
    build.build()


CASES = {  # tokens, contexts, prefix
    "step, whole": ([1] * 400, [60] * 400, 0),
    "step, split": ([1], [20000], 0),
    "step, split in two levels, one short": ([1, 1, 1], [9000, 30, 15000], 0),
    "rows, whole": ([3, 300, 5], [3, 300, 90], 0),
    "rows, split": ([20, 2], [12000, 30], 0),
    "prefix, step": ([1] * 5, [0, 1, 90, 200, 7], 300),
    "prefix, step, long": ([1, 1], [6000, 10], 3000),
    "prefix, rows": ([16, 3, 40], [16, 50, 40], 200),
}


def _rows(b):
    """A few (token, head) rows, the first and last of the call among them."""
    n = b.q.shape[0]
    return sorted({(0, 0), (n - 1, b.hq - 1), (n // 2, 1), (n // 3, b.hq // 2)})


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("value", ["nan", "one nan", "inf", "-inf"])
@pytest.mark.parametrize("case", CASES)
def test_rows_that_are_not_finite(case, value, d):
    t, lens, prefix = CASES[case]
    b = Batch(t, lens, 8, 2, d, 64, prefix=prefix, gate=True, seed=71)
    ref, bound, ref_lse = reference(b)
    bad = torch.zeros(b.q.shape[:2], dtype=torch.bool, device="cuda")
    for tok, head in _rows(b):
        if value == "one nan":
            b.q[tok, head, d // 3] = math.nan
        else:
            b.q[tok, head] = float(value)
        bad[tok, head] = True
    out, lse = (x.cpu().double() for x in _run(b))
    bad = bad.cpu()
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    assert ((out - ref).abs() <= bound + 1e-30)[~bad].all()
    assert ((lse - ref_lse).abs() <= 2.0 ** -15 * (1 + ref_lse.abs()))[~bad].all()


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("step,prefix", [(True, 0), (False, 0), (True, 40), (False, 40)])
def test_scores_that_are_all_minus_infinity(step, prefix, d):
    """Keys of ones and a query with one -inf: every score is -inf, the row's softmax 0 / 0 and the
    sum of exponentials 0; the other rows' softmax is the plain mean."""
    t, lens = ([1, 1, 1], [1, 70, 9000]) if step else ([2, 30, 1], [2, 90, 9000])
    b = Batch(t, lens, 4, 2, d, 64, prefix=prefix, seed=72)
    b.k_cache[~b.k_cache.isnan()] = 1.0
    b.q.fill_(1.0)
    bad = torch.zeros(b.q.shape[:2], dtype=torch.bool, device="cuda")
    for tok, head in _rows(b):
        b.q[tok, head, 5] = -math.inf
        bad[tok, head] = True
    out, lse = _run(b, step=step)
    torch.cuda.synchronize()
    assert out[bad].isnan().all() and (lse[bad] == -math.inf).all()
    assert torch.isfinite(out[~bad]).all() and torch.isfinite(lse[~bad]).all()


@pytest.mark.parametrize("d", [128, 256])
def test_part_of_a_row_minus_infinity(d):
    """Scores of -inf over the first 8000 of 9000 keys: those parts count for nothing."""
    b = Batch([1, 20], [9000, 9000], 4, 2, d, 64, seed=73)
    far = [p for s in b.pages for p in s[:8000 // 64]]
    near = [p for s in b.pages for p in s[8000 // 64:]]
    b.k_cache[far] = 0.0
    b.k_cache[far, :, :, 5] = 3.0e38
    b.k_cache[near, :, :, 5] = 0.0
    b.q[..., 5] = -3.0e38
    for step in (True, False):
        c = Batch([1], [9000], 4, 2, d, 64, seed=73) if step else b
        if step:
            c.k_cache, c.v_cache, c.q = b.k_cache, b.v_cache, b.q[:1]
            c.pages, c.page_table = b.pages[:1], b.page_table[:1].contiguous()
        out, lse = _run(c, step=step)
        torch.cuda.synchronize()
        # the same row over the last 1000 keys alone
        ks, vs = (torch.cat([x[p] for p in c.pages[-1]], 1)[:, 8000:9000].double()
                  for x in (c.k_cache, c.v_cache))
        q = c.q[-1].double()
        for h in range(4):
            s = ks[h // 2] @ q[h] * d ** -0.5
            p = torch.softmax(s, 0)
            want, mean = p @ vs[h // 2], p @ vs[h // 2].abs()
            assert ((out[-1, h].double() - want).abs() <= 2.0 ** -8 * (mean + want.abs()) + 2.0 ** -14 * mean).all()
            e = torch.logsumexp(s, 0)
            assert abs(lse[-1, h].item() - e.item()) <= 2.0 ** -15 * (1 + abs(e.item()))


@pytest.mark.parametrize("step,prefix", [(True, 0), (False, 0), (True, 40), (False, 40)])
def test_nothing_to_see_is_still_zero(step, prefix):
    """A NaN query that sees no key gives the zeros and -inf of every such row; behind a prefix it
    sees the prefix."""
    t, lens = ([1, 1], [0, 3]) if step else ([4, 9], [0, 3])
    b = Batch(t, lens, 4, 2, 128, 16, prefix=prefix, seed=74)
    b.q[0] = math.nan
    out, lse = _run(b, step=step)
    torch.cuda.synchronize()
    if prefix:
        assert out[0].isnan().all() and lse[0].isnan().all()
    else:
        assert (out[0] == 0).all() and (lse[0] == -math.inf).all()
