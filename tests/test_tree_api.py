"""What the calls for trees of drafts and for beams refuse, on the host and before anything is launched.
The calls pass made-up device addresses, so the module runs only where no GPU is visible."""
import ctypes

import pytest
import torch

import gated_deltanet_linear_05_gb300 as gdn
from gated_deltanet_linear_05_gb300 import build as gdn_build

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses: CPU-only checks")

OK, INVALID, UNSUPPORTED, ALIAS, WORKSPACE = (gdn.GDN_OK, gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED,
                                              gdn.GDN_ERR_ALIAS, gdn.GDN_ERR_WORKSPACE)
A = 1 << 24  # made-up buffers lie A bytes apart


@pytest.fixture(scope="module")
def L():
    gdn_build.build()
    return gdn.lib()


# ------------------------------------------------------------------ gdn_tree_attention

def _attend(L, n=2, tokens=0, prefix_len=0, **kw):
    s = gdn.make_attn_shape(n, tokens, 4, 2, 128, page_size=16, num_pages=8, max_pages=4, prefix_len=prefix_len,
                            **{k: kw.pop(k) for k in ("scale", "dtype") if k in kw})
    a = dict(q=A, gate=None, k=2 * A, v=3 * A, prefix=None, table=4 * A, lens=5 * A, cu=6 * A, up=7 * A, o=8 * A, lse=None,
             ws=64 * A, nbytes=1 << 40)
    a.update(kw)
    return L.gdn_tree_attention(ctypes.byref(s), *[a[x] for x in ("q", "gate", "k", "v", "prefix", "table", "lens", "cu", "up",
                                                                  "o", "lse", "ws", "nbytes")], None)


@pytest.mark.parametrize("kw,status", [
    ({}, OK), (dict(cu=None), INVALID), (dict(cu=None, n=0), INVALID), (dict(up=7 * A + 2), INVALID), (dict(tokens=3, up=None), INVALID),
    (dict(n=-1), INVALID), (dict(dtype=gdn.GDN_F32), UNSUPPORTED), (dict(scale=float("nan")), INVALID),
    (dict(prefix_len=20), INVALID), (dict(prefix_len=20, prefix=9 * A), OK), (dict(prefix_len=20, prefix=9 * A + 1), INVALID),
    (dict(tokens=3, ws=None), WORKSPACE), (dict(tokens=3, nbytes=100), WORKSPACE), (dict(tokens=3, ws=64 * A + 16), WORKSPACE),
    (dict(tokens=3, o=A + 64), ALIAS), (dict(tokens=3, gate=8 * A), ALIAS), (dict(tokens=3, q=None), INVALID),
    (dict(tokens=3, lens=None), INVALID), (dict(tokens=3, q=A + 8), INVALID)])
def test_attention_refuses(L, kw, status):
    assert _attend(L, **kw) == status


def test_attention_workspace_holds_the_trees():
    """Room for 64 bits a token, monotonous in the tokens."""
    gdn_build.build()
    size = [gdn.gdn_attn_workspace_size(gdn.make_attn_shape(2, t, 4, 2, 128)) for t in (0, 1, 33, 100, 1000)]
    assert size == sorted(size) and size[-1] - size[0] >= 8000


# ------------------------------------------------------------------ gdn_verify_tree

def _verify(L, n=2, tokens=0, hk=2, hv=4, chunk=32, dtype=gdn.GDN_BF16, o_fp32=0, algo=0, dk=128, **kw):
    s = gdn.make_shape(n, tokens, hk, hv, dk, 128, chunk, dtype, o_fp32, algo)
    a = dict(q=A, k=2 * A, v=3 * A, g=4 * A, beta=5 * A, state=16 * A, cu=6 * A, up=7 * A, o=8 * A, delta=9 * A)
    a.update(kw)
    return L.gdn_verify_tree(ctypes.byref(s), *[a[x] for x in ("q", "k", "v", "g", "beta", "state", "cu", "up", "o", "delta")], None)


@pytest.mark.parametrize("kw,status", [
    ({}, OK), (dict(state=None), OK), (dict(n=0, cu=None), OK), (dict(n=-1), INVALID), (dict(hv=3), INVALID), (dict(hk=0), INVALID),
    (dict(dk=64), UNSUPPORTED), (dict(chunk=48), UNSUPPORTED), (dict(chunk=128), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED),
    (dict(o_fp32=2), INVALID), (dict(algo=gdn.GDN_ALGO_TWO_PASS), UNSUPPORTED), (dict(algo=gdn.GDN_ALGO_RECURRENT), UNSUPPORTED),
    (dict(cu=None), INVALID), (dict(cu=6 * A + 2), INVALID), (dict(up=7 * A + 1), INVALID), (dict(state=16 * A + 8), INVALID),
    *[({"tokens": 3, x: None}, INVALID) for x in ("q", "k", "v", "g", "beta", "up", "o", "delta")],
    *[({"tokens": 3, x: 20 * A + 4}, INVALID) for x in ("q", "k", "v", "g", "beta", "o", "delta")],
    *[({"tokens": 3, "o": x * A}, ALIAS) for x in (1, 2, 3, 4, 5, 16, 6, 7, 9)],
    *[({"tokens": 3, "delta": x * A}, ALIAS) for x in (1, 2, 3, 4, 5, 16, 6, 7, 8)],
    (dict(tokens=3, delta=8 * A + 3 * 4 * 128 * 2 - 16), ALIAS), (dict(tokens=3, o_fp32=1, delta=8 * A + 3 * 4 * 128 * 2), ALIAS)])
def test_verify_refuses(L, kw, status):
    assert _verify(L, **kw) == status


# ------------------------------------------------------------------ gdn_beam_select

def _select(L, groups=2, beams=3, vocab=100, top=4, dtype=gdn.GDN_BF16, pad=0, stride=0, **kw):
    s = gdn.make_beam_shape(groups, beams, vocab, top, dtype, pad, stride)
    a = dict(logits=A, scores=2 * A, fin=None, out=3 * A, up=4 * A, tok=5 * A, ws=6 * A, nbytes=A)
    a.update(kw)
    return L.gdn_beam_select(ctypes.byref(s), *[a[x] for x in ("logits", "scores", "fin", "out", "up", "tok", "ws", "nbytes")], None)


BAD_BEAMS = [
    (dict(groups=-1), INVALID), (dict(beams=0), INVALID), (dict(beams=65), UNSUPPORTED), (dict(vocab=0), INVALID), (dict(top=0), INVALID),
    (dict(top=65, vocab=100), UNSUPPORTED), (dict(top=9, vocab=8), INVALID), (dict(vocab=(1 << 24) + 1), UNSUPPORTED),
    (dict(dtype=2), UNSUPPORTED), (dict(pad=-1), INVALID), (dict(pad=100), INVALID), (dict(stride=99), INVALID), (dict(stride=-200), INVALID),
    (dict(stride=1 << 40), UNSUPPORTED), (dict(groups=1 << 20), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", BAD_BEAMS + [
    (dict(groups=0, logits=None), OK),
    *[({x: None}, INVALID) for x in ("logits", "scores", "out", "up", "tok")],
    *[({x: 20 * A + 2}, INVALID) for x in ("scores", "out", "up", "tok")],
    (dict(logits=A + 1), INVALID), (dict(logits=A + 2, dtype=gdn.GDN_F32), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=6 * A + 128), WORKSPACE), (dict(nbytes=8), WORKSPACE),
    (dict(out=4 * A), ALIAS), (dict(up=5 * A + 8), ALIAS), (dict(out=2 * A), ALIAS), (dict(tok=A + 2 * 3 * 200 - 4), ALIAS),
    (dict(fin=3 * A + 4), ALIAS), (dict(tok=6 * A), ALIAS), (dict(scores=6 * A), ALIAS), (dict(stride=400, up=A + 4000), ALIAS)])
def test_select_refuses(L, kw, status):
    assert _select(L, **kw) == status


@pytest.mark.parametrize("kw,status", BAD_BEAMS)
def test_beam_workspace_size_refuses(L, kw, status):
    args = dict(groups=2, beams=3, vocab=100, top=4, dtype=gdn.GDN_BF16, pad=0, stride=0)
    args.update(kw)
    s = gdn.make_beam_shape(*[args[x] for x in ("groups", "beams", "vocab", "top", "dtype", "pad", "stride")])
    with pytest.raises(gdn.GdnError):
        gdn.gdn_beam_workspace_size(s)


# ------------------------------------------------------------------ gdn_beam_reorder

@pytest.mark.parametrize("args,status", [
    ((0, 2, 4, 64, A, 2 * A), OK), ((1, 0, 4, 64, A, 2 * A), OK), ((1, 2, 4, 0, None, None), OK), ((-1, 2, 4, 64, A, 2 * A), INVALID),
    ((1, -2, 4, 64, A, 2 * A), INVALID), ((1, 2, 0, 64, A, 2 * A), INVALID), ((1, 2, 65, 64, A, 2 * A), UNSUPPORTED),
    ((1, 2, 4, -64, A, 2 * A), INVALID), ((1, 2, 4, 66, A, 2 * A), INVALID), ((1, 2, 4, 64, None, 2 * A), INVALID),
    ((1, 2, 4, 64, A, None), INVALID), ((1, 2, 4, 64, A + 2, 2 * A), INVALID), ((1, 2, 4, 64, A, 2 * A + 1), INVALID),
    ((1, 2, 4, 64, 2 * A + 508, 2 * A), ALIAS), ((1, 2, 4, 1 << 40, A, 2 * A), UNSUPPORTED), ((1 << 20, 1 << 20, 4, 64, A, 2 * A), UNSUPPORTED),
    ((1 << 12, 1 << 12, 4, 1 << 20, A, 2 * A), UNSUPPORTED)])
def test_reorder_refuses(L, args, status):
    assert L.gdn_beam_reorder(*args, None) == status


# ------------------------------------------------------------------ the binding

def test_binding_refuses_before_the_library():
    """Tensors that are not on a GPU, of the wrong type or shape."""
    q = torch.zeros(4, 4, 128, dtype=torch.bfloat16)
    cache = torch.zeros(2, 2, 16, 128, dtype=torch.bfloat16)
    idx = torch.zeros(1, dtype=torch.int32)
    table, cu, up = torch.zeros(1, 2, dtype=torch.int32), torch.tensor([0, 4], dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    for kw in (dict(), dict(parents=up[:3]), dict(cu_seqlens=None), dict(parents=up.long())):
        a = dict(q=q, k_cache=cache, v_cache=cache, page_table=table, kv_lens=idx, cu_seqlens=cu, parents=up, workspace=idx)
        a.update(kw)
        with pytest.raises((ValueError, TypeError)):
            gdn.gdn_tree_attention(**a)
    with pytest.raises(ValueError):
        gdn.gdn_verify_tree(q, q, q, *[torch.zeros(4, 4)] * 2, None, cu, up)
    logits, scores = torch.zeros(1, 2, 8), torch.zeros(1, 2)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        gdn.gdn_beam_select(logits, scores, 2)
    for bad in (logits[0], logits.double(), logits.transpose(1, 2)):
        with pytest.raises(ValueError):
            gdn.gdn_beam_select(bad, scores, 2)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        gdn.gdn_beam_reorder(torch.zeros(1, 2, 4), torch.zeros(1, 2, dtype=torch.int32))
