"""GPU parity of the attention over the paged cache, with and without a shared prefix, against
the definition in 64 bits.  The bound of every element counts the kernel's roundings
(attn_testlib.reference); the log-sum-exp is float32 throughout: 2^-15 (1 + |lse|)."""
import pytest
import torch

from attn_testlib import Batch, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_deltanet_linear_05_gb300 import build
    build.build()


def _workspace(b):
    import gated_deltanet_linear_05_gb300 as gdn
    return gdn.gdn_attn_workspace(len(b.t), sum(b.t), b.hq, b.hkv, b.d, prefix_len=b.prefix)


def _run(b, step=None, scale=None, workspace=None, lse=True, **kw):
    import gated_deltanet_linear_05_gb300 as gdn
    step = all(x == 1 for x in b.t) if step is None else step
    ws = _workspace(b) if workspace is None else workspace
    out = torch.full(b.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    l = torch.full(b.q.shape[:2], float("nan"), device="cuda") if lse else None
    args = (b.page_table, b.kv_lens, None if step else b.cu, b.gate, scale, out, l, ws)
    if b.prefix:
        gdn.gdn_shared_prefix_attention(b.q, b.k_cache, b.v_cache, b.prefix_table, b.prefix, *args, **kw)
    else:
        gdn.gdn_paged_attention(b.q, b.k_cache, b.v_cache, *args, **kw)
    return out, l


def _check(b, out, l=None, scale=None):
    torch.cuda.synchronize()
    ref, bound, lse = reference(b, scale)
    got = out.cpu().double()
    assert torch.isfinite(got).all()
    excess = (got - ref).abs() - bound
    assert excess.max().item() <= 1e-30, "worst excess %.3g, at row %s" % (
        excess.max().item(), divmod(int(excess.argmax()), b.hq * b.d))
    if l is not None:
        x = l.cpu().double()
        assert torch.equal(torch.isinf(x), torch.isinf(lse))
        fine = torch.isfinite(lse)
        assert ((x - lse)[fine].abs() <= 2.0 ** -15 * (1 + lse[fine].abs())).all()


HEADS = [(1, 1), (4, 4), (4, 1), (6, 2), (10, 2), (16, 1), (24, 1), (40, 2)]


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_step_heads(hq, hkv, d):
    b = Batch([1] * 5, [1, 63, 64, 200, 333], hq, hkv, d, 16, seed=1)
    _check(b, *_run(b))


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("gate", [False, True])
def test_step_pages(page, d, gate):
    lens = [0, 1, page - 1, page, page + 1, 2 * page, 127, 128, 129, 257, 1000]
    b = Batch([1] * len(lens), lens, 8, 2, d, page, gate=gate, seed=2)
    _check(b, *_run(b))


@pytest.mark.parametrize("d", [128, 256])
def test_step_long_split(d):
    """Few rows over long contexts: many parts joined."""
    b = Batch([1, 1], [9001, 20000], 4, 1, d, 64, seed=3)
    _check(b, *_run(b))


@pytest.mark.parametrize("lens", [[20000], [3100], [1300], [900, 15000, 5], [7000, 7000]])
@pytest.mark.parametrize("hq,d", [(4, 128), (16, 128), (5, 256)])
def test_step_joins_of_many_parts(hq, d, lens):
    """One kv-head: a context lies in up to all runs; the second call finds the counters ready."""
    b = Batch([1] * len(lens), lens, hq, 1, d, 64, gate=True, seed=41)
    ws = _workspace(b)
    out, l = _run(b, workspace=ws)
    _check(b, out, l)
    again, l2 = _run(b, workspace=ws)
    assert torch.equal(out, again) and torch.equal(l, l2)


def test_step_many_sequences():
    """More sequences than CTAs, empty ones among them."""
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 90, (700,), generator=g).tolist()
    b = Batch([1] * 700, lens, 4, 2, 128, 16, seed=4)
    _check(b, *_run(b))


@pytest.mark.parametrize("lens", [[0], [0, 0, 0], [1]])
def test_step_tiny(lens):
    b = Batch([1] * len(lens), lens, 4, 2, 128, 16, seed=5)
    _check(b, *_run(b))


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_rows_heads(hq, hkv, d):
    b = Batch([1, 16, 7, 130, 0, 40], [1, 16, 200, 130, 5, 333], hq, hkv, d, 32, seed=6)
    _check(b, *_run(b))


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("gate", [False, True])
def test_rows_pages(page, d, gate):
    """Tiles that end inside a page, at it and past it; rows before the first key (kv_len
    below the number of tokens) see nothing."""
    t = [1, 3, page, 127, 128, 129, 64, 5]
    lens = [page, page + 1, page, 127, 128, 200, 20, 0]
    b = Batch(t, lens, 4, 2, d, page, gate=gate, seed=7)
    _check(b, *_run(b))


@pytest.mark.parametrize("d", [128, 256])
def test_rows_prompt(d):
    """A prompt of several tiles in both directions, and one that continues a context."""
    b = Batch([700, 300], [700, 1500], 4, 2, d, 64, seed=8)
    _check(b, *_run(b))


@pytest.mark.parametrize("d", [128, 256])
def test_rows_long_context_split(d):
    """Few query rows on a long context: the keys are split and joined."""
    b = Batch([20, 2], [12000, 3], 4, 2, d, 64, seed=9)
    _check(b, *_run(b))


def test_rows_many_sequences():
    g = torch.Generator().manual_seed(10)
    t = torch.randint(0, 6, (400,), generator=g).tolist()
    lens = [max(0, x + int(torch.randint(-2, 70, (1,), generator=g))) for x in t]
    b = Batch(t, lens, 4, 2, 128, 16, seed=10)
    _check(b, *_run(b, step=False))


def _check_many(b, out, l):
    """_check with the caches brought over once, not once a sequence."""
    b.k_cache, b.v_cache = (c.cpu().double() for c in (b.k_cache, b.v_cache))
    _check(b, out, l)


@pytest.mark.parametrize("prefix", [0, 20])
def test_rows_more_tiles_than_the_plan_keeps(prefix):
    """Several chunks of sequences in the plan and tiles past those whose lengths it keeps at hand;
    long sequences, whose tiles all threads write, in the first chunk and after it."""
    g = torch.Generator().manual_seed(35)
    t = torch.randint(0, 4, (4600,), generator=g).tolist()
    t[7], t[1300], t[4599] = 700, 400, 333
    lens = [x + int(torch.randint(0, 9, (1,), generator=g)) for x in t]
    b = Batch(t, lens, 4, 2, 128, 16, prefix=prefix, seed=35)
    _check_many(b, *_run(b, step=False))


@pytest.mark.parametrize("d,n", [(128, 5000), (256, 2700)])
def test_prefix_more_row_tiles_than_units(d, n):
    """One query head a kv-head: more (row tile, kv-head) pairs of the prefix than units, so one part each."""
    b = Batch([1] * n, [i % 5 for i in range(n)], 8, 8, d, 16, prefix=130, gate=True, seed=36)
    _check_many(b, *_run(b))


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (6, 2), (16, 1), (24, 1)])
@pytest.mark.parametrize("prefix", [1, 64, 300])
def test_prefix_step(prefix, hq, hkv, d):
    b = Batch([1] * 6, [0, 1, 16, 17, 100, 257], hq, hkv, d, 16, prefix=prefix, gate=True, seed=11)
    _check(b, *_run(b))


@pytest.mark.parametrize("d", [128, 256])
def test_prefix_long(d):
    b = Batch([1] * 40, list(range(0, 80, 2)), 8, 2, d, 64, prefix=7000, seed=12)
    _check(b, *_run(b))


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("prefix", [5, 500])
def test_prefix_rows(prefix, d):
    b = Batch([16, 1, 70, 0, 9], [16, 40, 90, 3, 4], 6, 2, d, 32, prefix=prefix, seed=13)
    _check(b, *_run(b))


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("lens,prefix", [([6000, 3500], 17), ([0, 0, 0], 9000), ([5000], 5000),
                                         ([i * 7 % 401 for i in range(300)], 130), ([1], 1)])
def test_prefix_divisions(lens, prefix, d):
    """One kind of work far larger than the other, both alike, more sequences than CTAs."""
    b = Batch([1] * len(lens), lens, 4, 2, d, 64, prefix=prefix, seed=24)
    _check(b, *_run(b))


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("hq,hkv", [(128, 1), (64, 1), (34, 2)])
@pytest.mark.parametrize("prefix", [0, 70])
def test_wide_groups(hq, hkv, prefix, d):
    """More query heads a kv-head than the decode kernel takes, up to a tile of one token."""
    for t, lens in (([1, 1, 1], [5, 130, 300]), ([3, 1, 20], [3, 130, 300])):
        b = Batch(t, lens, hq, hkv, d, 32, prefix=prefix, gate=True, seed=25)
        _check(b, *_run(b))


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("lens", [[5, 17, 128, 129, 700], [1024, 90], [1025, 90, 300]])
@pytest.mark.parametrize("d", [128, 256])
def test_drafts_around_the_narrow_bound(d, lens, gate):
    """A few rows a sequence, contexts to both sides of what chooses the tiles' width."""
    b = Batch([3, 5, 1, 8, 2][:len(lens)], lens, 12, 4, d, 16, gate=gate, seed=51)
    _check(b, *_run(b))


@pytest.mark.parametrize("t", [31, 32, 33, 65])
@pytest.mark.parametrize("d", [128, 256])
def test_rows_around_a_narrow_tile(t, d):
    """Rows of one, and just more than one, sub-tile: mean rows a sequence of 124 to 260."""
    b = Batch([t, t, t], [t, t + 1, t + 200], 8, 2, d, 32, gate=True, seed=52)
    _check(b, *_run(b))


@pytest.mark.parametrize("d,length", [(128, 9000), (256, 1000), (256, 9000)])
def test_one_draft_split(d, length):
    b = Batch([6], [length], 8, 2, d, 64, seed=53)
    _check(b, *_run(b))


@pytest.mark.parametrize("prefix", [70, 1500])
@pytest.mark.parametrize("d", [128, 256])
def test_prefix_drafts(prefix, d):
    b = Batch([2, 9, 1, 4], [2, 40, 333, 129], 12, 4, d, 16, prefix=prefix, gate=True, seed=54)
    _check(b, *_run(b))


@pytest.mark.parametrize("d", [128, 256])
def test_prompt_of_uneven_tiles(d):
    """One prompt whose tiles would fill the machine unevenly, split or not."""
    b = Batch([700], [703], 12, 4, d, 128, gate=True, seed=55)
    _check(b, *_run(b))


@pytest.mark.parametrize("seed", range(12))
def test_drawn_shapes(seed):
    """Sizes drawn over the whole range of heads, pages, lengths and kinds of call."""
    import random
    r = random.Random(100 + seed)
    hkv, group = r.choice([1, 2, 3]), r.choice([1, 2, 3, 5, 7, 8, 13, 16])
    n = r.randint(1, 9)
    step = r.random() < 0.4
    t = [1] * n if step else [r.choice([0, 1, 2, 17, r.randint(1, 200)]) for _ in range(n)]
    lens = [max(0, a + r.choice([-1, 0, 0, 1, r.randint(0, 700)])) for a in t]
    b = Batch(t, lens, hkv * group, hkv, r.choice([128, 256]), r.choice([16, 32, 64, 128]),
              prefix=r.choice([0, 0, 1, 63, 200]), gate=r.random() < 0.5, seed=seed, q_pad=r.choice([0, 8]),
              page_pad=r.choice([0, 128]))
    if sum(t):
        _check(b, *_run(b, step=step))


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("prefix", [0, 100])
def test_strides(step, prefix):
    """Padded heads and tokens in q and gate, padding between pages; NaN in the padding."""
    t = [1] * 4 if step else [3, 20, 1, 8]
    b = Batch(t, [30, 64, 1, 99], 6, 2, 128, 16, prefix=prefix, gate=True, seed=14, q_pad=24,
              page_pad=64)
    _check(b, *_run(b, step=step))


def _head_major(x):
    return None if x is None else x.transpose(0, 1).contiguous().transpose(0, 1)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("prefix", [0, 100])
def test_head_major(prefix, step, d):
    """A token stride below the head stride, in q and gate together or in one of them."""
    t = [1] * 5 if step else [3, 20, 1, 140]
    b = Batch(t, [30, 64, 1, 299, 7][:len(t)], 6, 2, d, 16, prefix=prefix, gate=True, seed=31)
    q, gate = b.q, b.gate
    for both in ((_head_major(q), gate), (q, _head_major(gate)), (_head_major(q), _head_major(gate))):
        b.q, b.gate = both
        _check(b, *_run(b, step=step))


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("prefix", [0, 70])
@pytest.mark.parametrize("kind", ["step", "drafts", "prompts"])
@pytest.mark.parametrize("gate", [False, True])
def test_calls_as_users_make_them(gate, kind, prefix, d):
    """No log-sum-exp, a new output, sizes that have been seen: the way through the marshalling module,
    with other values of the same sizes each time."""
    import gated_deltanet_linear_05_gb300 as gdn
    t = {"step": [1] * 4, "drafts": [3, 7, 1, 5], "prompts": [200, 1, 90]}[kind]
    lens = [200, 64, 99, 300][:len(t)]
    ws = None
    for seed in (32, 33, 34):
        b = Batch(t, lens, 8, 2, d, 32, prefix=prefix, gate=gate, seed=seed)
        ws = _workspace(b) if ws is None else ws
        args = (b.page_table, b.kv_lens, None if kind == "step" else b.cu)
        if prefix:
            out = gdn.gdn_shared_prefix_attention(b.q, b.k_cache, b.v_cache, b.prefix_table, prefix, *args,
                                                  gate=b.gate, workspace=ws)
        else:
            out = gdn.gdn_paged_attention(b.q, b.k_cache, b.v_cache, *args, gate=b.gate, workspace=ws)
        _check(b, out)


@pytest.mark.parametrize("step", [False, True])
def test_scale_and_extreme_scores(step):
    """Scores of +-1000: the running maximum carries them; a negative and a zero scale."""
    b = Batch([1] * 3 if step else [4, 1, 30], [50, 300, 130], 4, 2, 128, 16, seed=15, std=30.0)
    for scale in (3.0, -3.0, 0.0):
        ref, bound, lse = reference(b, scale)
        out, l = _run(b, step=step, scale=scale)
        torch.cuda.synchronize()
        # a score's own error, D 2^-24 sum|q k| scale, is no longer small beside the exponent's
        # argument: it moves a probability by that much, and the mean of |v| with it
        err = 128 * 2.0 ** -24 * abs(scale) * 128 * 30.0 * 1.0
        got = out.cpu().double()
        assert torch.isfinite(got).all()
        vmax = 6.0
        assert ((got - ref).abs() <= bound + 2 * err * vmax).all()
        assert ((l.cpu().double() - lse).abs() <= 2.0 ** -15 * (1 + lse.abs()) + err).all()


@pytest.mark.parametrize("scale", [1e-39, -1e-39, 1e-44, 2.0 ** -126, -2.0 ** -126])
@pytest.mark.parametrize("kind", ["step", "rows", "prefix"])
def test_scales_at_the_end_of_float32(kind, scale):
    """At and below the smallest normal number: the mean of the visible values."""
    t = [7, 30, 1] if kind == "rows" else [1, 1, 1]
    b = Batch(t, [9, 300, 130], 4, 2, 128, 16, prefix=50 if kind == "prefix" else 0, seed=26)
    _check(b, *_run(b, step=kind != "rows", scale=scale), scale)


@pytest.mark.parametrize("kind", ["step", "rows", "prefix step", "prefix rows"])
def test_more_than_2_to_the_30_keys(kind):
    """One page over and over, its scores 0, and at the end of the context 40 times one whose scores
    are 60: the mean of that page's values."""
    import gated_deltanet_linear_05_gb300 as gdn
    g = torch.Generator().manual_seed(29)
    keys = (1 << 30) + 128 * 50
    k, v = torch.zeros(2, 1, 128, 128), torch.randn(2, 1, 128, 128, generator=g)
    k[1] = 60 / 128 ** 0.5
    k, v = k.bfloat16().cuda(), v.bfloat16().cuda()
    far = torch.zeros(1, keys // 128, dtype=torch.int32, device="cuda")
    far[:, -40:] = 1
    q = torch.ones(1, 1, 128, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda") if "rows" in kind else None
    lens = torch.tensor([0 if "prefix" in kind else keys], dtype=torch.int32, device="cuda")
    if "prefix" in kind:
        o = gdn.gdn_shared_prefix_attention(q, k, v, far[0], keys, far[:, :1].contiguous(), lens, cu)
    else:
        o = gdn.gdn_paged_attention(q, k, v, far, lens, cu)
    torch.cuda.synchronize()
    x = v[1, 0].double()
    want, mean = x.mean(0), x.abs().mean(0)
    assert ((o[0, 0].double() - want).abs() <= 2.0 ** -8 * (mean + want.abs()) + 2.0 ** -14 * mean).all()
    assert gdn.gdn_device_status() == 0


def test_far_pages():
    """A cache whose pages lie past 2^31 elements."""
    import gated_deltanet_linear_05_gb300 as gdn
    b = Batch([1, 9], [40, 33], 4, 2, 128, 16, seed=16)
    pages = b.k_cache.shape[0]
    stride = 1 << 29
    ws = _workspace(b)
    big = [torch.empty((pages - 1) * stride + b.k_cache[0].numel(), dtype=torch.bfloat16, device="cuda")
           .as_strided(b.k_cache.shape, (stride,) + b.k_cache.stride()[1:]) for _ in range(2)]
    assert (pages - 1) * stride > 1 << 31
    big[0].copy_(b.k_cache)
    big[1].copy_(b.v_cache)
    out = gdn.gdn_paged_attention(b.q, big[0], big[1], b.page_table, b.kv_lens, b.cu, workspace=ws)
    one = gdn.gdn_paged_attention(b.q[:2], big[0], big[1], b.page_table, b.kv_lens, workspace=ws)
    _check(b, out)
    c = Batch([1, 1], [40, 33], 4, 2, 128, 16, seed=16)
    c.k_cache, c.v_cache, c.q, c.pages = b.k_cache, b.v_cache, b.q[:2], b.pages
    _check(c, one)


def test_workspace_is_left_ready_and_results_repeat():
    """One workspace for calls of several kinds in turn; every call gives the bits of its first."""
    import gated_deltanet_linear_05_gb300 as gdn
    kinds = [Batch([1] * 3, [5000, 70, 0], 8, 2, 128, 64, seed=17),
             Batch([20, 3, 1], [6000, 70, 9], 8, 2, 128, 64, seed=18),
             Batch([1] * 3, [50, 7, 900], 8, 2, 128, 64, prefix=2000, seed=19),
             Batch([1] * 2, [4000, 9000], 8, 2, 256, 64, seed=20)]
    ws = gdn.gdn_attn_workspace(3, 24, 8, 2, 256, prefix_len=2000)
    first = [_run(b, workspace=ws) for b in kinds]
    for b, (o, l) in zip(kinds, first):
        _check(b, o, l)
    for _ in range(3):
        for b, (o, l) in zip(kinds, first):
            o2, l2 = _run(b, workspace=ws)
            assert torch.equal(o, o2) and torch.equal(l, l2)


@pytest.mark.parametrize("t,lens,prefix", [([1, 1, 1], [9000, 70, 0], 0), ([20, 3, 1], [6000, 70, 9], 0),
                                           ([1, 1, 1], [50, 7, 900], 2000), ([20, 3, 1], [60, 7, 900], 2000)])
@pytest.mark.parametrize("d", [128, 256])
def test_workspace_beyond_its_counters_may_hold_anything(d, t, lens, prefix):
    b = Batch(t, lens, 8, 2, d, 64, prefix=prefix, gate=True, seed=30)
    ws = _workspace(b)
    for poison in (0, 255, 127):
        ws[2048:] = poison
        _check(b, *_run(b, workspace=ws))


@pytest.mark.parametrize("kind", ["step", "rows", "prefix"])
def test_graph_and_stream(kind):
    """Captured on a side stream and replayed on new values of the same tensors."""
    prefix = 200 if kind == "prefix" else 0
    t = [6, 30] if kind == "rows" else [1, 1]
    b = Batch(t, [600, 90], 8, 2, 128, 64, prefix=prefix, seed=21)
    ws = _workspace(b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _run(b, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out, l = _run(b, workspace=ws)
    b.q.mul_(-0.5)
    b.lens = [300, 64]
    b.kv_lens.copy_(torch.tensor(b.lens, dtype=torch.int32))
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    _check(b, out, l)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("t", [[1, 1, 1], [4, 130, 1], [2, 2, 2]])
def test_cache_without_pages(t, d):
    """No page, so no key, whatever the lengths say: zeros and -inf; the append stores nothing."""
    import gated_deltanet_linear_05_gb300 as gdn
    b = Batch(t, [5, 200, 3], 4, 2, d, 16, gate=True, seed=28)
    b.k_cache, b.v_cache = (torch.empty(0, 2, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = (torch.ones(sum(t), 2, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = gdn.gdn_kv_append(b.q, k, v, b.k_cache, b.v_cache, b.page_table, b.kv_lens, cu_seqlens=b.cu)
    for step in ([True, False] if t == [1, 1, 1] else [False]):
        out, l = _run(b, step=step)
        torch.cuda.synchronize()
        assert torch.equal(q, b.q) and (out == 0).all() and (l == -float("inf")).all()
    assert gdn.gdn_device_status() == 0


def test_bad_pages_stay_with_their_sequence():
    """A table entry out of range spoils its own sequence only."""
    import gated_deltanet_linear_05_gb300 as gdn
    for step in (True, False):
        b = Batch([1, 1, 1] if step else [5, 5, 5], [100, 90, 300], 4, 2, 128, 16, seed=22)
        b.page_table[1, 2] = 1 << 30
        b.page_table[1, 3] = -1
        out, _ = _run(b, step=step)
        torch.cuda.synchronize()
        ref, bound, _ = reference(b)
        t = b.t[0]
        keep = torch.cat([torch.arange(0, t), torch.arange(2 * t, 3 * t)])
        assert ((out.cpu().double() - ref).abs() <= bound + 1e-30)[keep].all()
    assert gdn.gdn_device_status() == 0


def test_malformed_cu_seqlens_stays_in_bounds():
    """Decreasing and too large entries: no access out of range, no lost wait."""
    import gated_deltanet_linear_05_gb300 as gdn
    b = Batch([5, 5, 5], [100, 90, 300], 4, 2, 128, 16, seed=23)
    for cu in ([0, 12, 3, 15], [0, 100, 200, 300], [-5, 5, 5, 15], [0, 0, 0, 0]):
        b.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        _run(b, step=False)
        torch.cuda.synchronize()
    assert gdn.gdn_device_status() == 0
