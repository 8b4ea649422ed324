"""What the attention-layer calls refuse, on the host and before anything is launched.  The calls
pass made-up device addresses, so the module runs only where no GPU is visible."""
import ctypes

import pytest

import gated_deltanet_linear_05_gb300 as gdn
from gated_deltanet_linear_05_gb300 import build as gdn_build


def _gpu_visible():
    try:
        import torch
        return torch.cuda.is_available()
    except Exception:
        return False


pytestmark = pytest.mark.skipif(_gpu_visible(), reason="fake device addresses: CPU-only checks")

OK, INVALID, UNSUPPORTED, ALIAS, WORKSPACE = (gdn.GDN_OK, gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED,
                                              gdn.GDN_ERR_ALIAS, gdn.GDN_ERR_WORKSPACE)
A = 1 << 20  # made-up buffers lie A bytes apart


@pytest.fixture(scope="module")
def L():
    gdn_build.build()
    return gdn.lib()


def _shape(n=2, tokens=0, hq=4, hkv=2, d=128, **kw):
    base = dict(page_size=16, num_pages=8, max_pages=4)
    fields = {k: kw.pop(k) for k in list(kw) if k in ("q_stride", "k_stride", "v_stride", "gate_stride", "page_stride")}
    s = gdn.make_attn_shape(n, tokens, hq, hkv, d, **{**base, **kw})
    for k, v in fields.items():
        if k == "page_stride":
            s.page_stride = v
        else:
            getattr(s, k)[:] = v
    return s


def _attend(L, s, prefix=None, **kw):
    a = dict(q=A, gate=None, k=2 * A, v=3 * A, table=4 * A, lens=5 * A, cu=6 * A, o=7 * A, lse=None, ws=64 * A,
             nbytes=1 << 40)
    a.update(kw)
    head = [ctypes.byref(s), a["q"], a["gate"], a["k"], a["v"]]
    tail = [a["table"], a["lens"], a["cu"], a["o"], a["lse"], a["ws"], a["nbytes"], None]
    if prefix is None:
        return L.gdn_paged_attention(*head, *tail)
    return L.gdn_shared_prefix_attention(*head, prefix, *tail)


def _append(L, s, eps=1e-6, **kw):
    a = dict(q=A, k=2 * A, v=3 * A, qn=None, kn=None, freq=None, axis=None, pos=None, table=4 * A, lens=5 * A,
             cu=6 * A, out=7 * A, kc=8 * A, vc=9 * A)
    a.update(kw)
    return L.gdn_kv_append(ctypes.byref(s), a["q"], a["k"], a["v"], a["qn"], a["kn"], eps, a["freq"], a["axis"],
                           a["pos"], a["table"], a["lens"], a["cu"], a["out"], a["kc"], a["vc"], None)


SHAPES = [
    (dict(n=-1), INVALID), (dict(tokens=-1), INVALID), (dict(hq=0), INVALID), (dict(hq=5), INVALID),
    (dict(hkv=0), INVALID), (dict(d=64), UNSUPPORTED), (dict(d=96), UNSUPPORTED),
    (dict(dtype=gdn.GDN_F32), UNSUPPORTED), (dict(hq=258, hkv=2), UNSUPPORTED),
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED),
    (dict(num_pages=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(max_pages=1 << 28), UNSUPPORTED),
    (dict(page_stride=2 * 16 * 128 - 8), INVALID), (dict(page_stride=2 * 16 * 128 + 4), INVALID),
    (dict(page_stride=1 << 40), UNSUPPORTED), (dict(tokens=1 << 30), UNSUPPORTED),
    (dict(n=0, tokens=5), INVALID), (dict(q_stride=(512, 64)), INVALID), (dict(q_stride=(-512, 128)), INVALID),
    (dict(q_stride=(516, 128)), INVALID), (dict(q_stride=(1 << 40, 128)), UNSUPPORTED),
]


@pytest.mark.parametrize("change,status", SHAPES)
def test_shapes_refused_by_every_call(L, change, status):
    assert _attend(L, _shape(**change)) == status
    assert _append(L, _shape(**change)) == status
    assert _attend(L, _shape(**{"prefix_len": 20, **change}), prefix=10 * A) == status


def test_null_shape(L):
    assert L.gdn_paged_attention(*[None] * 11, 0, None) == INVALID
    assert L.gdn_shared_prefix_attention(*[None] * 12, 0, None) == INVALID
    assert L.gdn_kv_append(*[None] * 6, 0.0, *[None] * 10) == INVALID
    assert L.gdn_attn_workspace_size(None) == ctypes.c_size_t(-1).value


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(cu=None), INVALID),
    (dict(q=A + 8), INVALID), (dict(o=A * 7 + 8), INVALID), (dict(k=2 * A + 4), INVALID),
    (dict(gate=A * 20 + 2), INVALID), (dict(lens=5 * A + 2), INVALID), (dict(cu=6 * A + 1), INVALID),
    (dict(table=4 * A + 2), INVALID), (dict(lse=30 * A + 2), INVALID),
    (dict(o=A), ALIAS), (dict(o=A + 1024), ALIAS), (dict(gate=7 * A + 16), ALIAS),
    (dict(ws=None), WORKSPACE), (dict(ws=64 * A + 128), WORKSPACE), (dict(nbytes=16), WORKSPACE),
])
def test_attention_arguments(L, change, status):
    assert _attend(L, _shape(n=3, tokens=7), **change) == status
    assert _attend(L, _shape(n=3, tokens=7, prefix_len=40), prefix=10 * A, **change) == status


def test_attention_other_refusals(L):
    assert _attend(L, _shape(prefix_len=16)) == INVALID  # a prefix goes with the other call
    assert _attend(L, _shape(), prefix=10 * A) == INVALID
    assert _attend(L, _shape(prefix_len=16), prefix=None) == INVALID
    assert _attend(L, _shape(n=2, tokens=2, prefix_len=16), prefix=10 * A + 2) == INVALID
    for scale in (float("nan"), float("inf")):
        assert _attend(L, _shape(scale=scale)) == INVALID
    assert _attend(L, _shape(n=3, tokens=7, gate_stride=(512, 100)), gate=30 * A) == INVALID
    assert _attend(L, _shape(n=3, tokens=7, gate_stride=(512, 100)), o=A) == ALIAS  # no gate: not read
    assert _attend(L, _shape(n=3, tokens=2), cu=None) == INVALID  # one token per sequence
    assert _attend(L, _shape(n=0, tokens=0)) == OK  # nothing to do
    assert _attend(L, _shape(n=2, tokens=0)) == OK


def test_no_tokens_behind_a_prefix(L):
    """Nothing to do, and a size all the same (tiles of the prefix's pass are divided by their number)."""
    for n in (0, 2):
        for d in (128, 256):
            shape = _shape(n=n, tokens=0, d=d, prefix_len=40)
            assert 0 < gdn.gdn_attn_workspace_size(shape) <= gdn.gdn_attn_workspace_size(
                _shape(n=max(n, 1), tokens=1, d=d, prefix_len=40))
            assert _attend(L, shape, prefix=10 * A) == OK


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_contexts_next_to_the_end_of_32_bits(L, page):
    """Key tiles are counted in whole tiles past the last key: the last few thousand are refused."""
    most, room = 0x7fffffff // page, 0x7fffe000 // page
    assert _attend(L, _shape(page_size=page, max_pages=most)) == UNSUPPORTED
    assert _attend(L, _shape(page_size=page, max_pages=room + 1)) == UNSUPPORTED
    assert _attend(L, _shape(page_size=page, max_pages=room)) == OK
    assert _attend(L, _shape(page_size=page, max_pages=room // 2, prefix_len=0x7fffe000 - room // 2 * page),
                   prefix=10 * A) == OK
    assert _attend(L, _shape(page_size=page, max_pages=room // 2, prefix_len=0x7fffe001 - room // 2 * page),
                   prefix=10 * A) == UNSUPPORTED
    assert _append(L, _shape(page_size=page, max_pages=most)) == OK


def test_scale_past_float32(L):
    """The kernels take scale * log2(e) in float32: its overflow is refused, not turned into NaN."""
    for scale in (3e38, -3e38, 2.4e38):
        assert _attend(L, _shape(scale=scale)) == INVALID
        assert _attend(L, _shape(scale=scale, prefix_len=16), prefix=10 * A) == INVALID
    for scale in (2.3e38, -2.3e38, 1e-44, 0.0):
        assert _attend(L, _shape(scale=scale)) == OK


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(out=None), INVALID),
    (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(freq=None), INVALID), (dict(freq=20 * A + 4), INVALID),
    (dict(qn=20 * A + 4), INVALID), (dict(kn=20 * A + 8), INVALID), (dict(pos=20 * A + 2), INVALID),
    (dict(axis=20 * A + 1), INVALID), (dict(v=3 * A + 8), INVALID), (dict(vc=9 * A + 8), INVALID),
    (dict(out=A + 16), ALIAS), (dict(out=2 * A), ALIAS), (dict(out=3 * A + 32), ALIAS),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
])
def test_append_arguments(L, change, status):
    assert _append(L, _shape(n=3, tokens=7, rotary_dim=64), **{"freq": 20 * A, **change}) == status


def test_append_other_refusals(L):
    for rot in (-16, 8, 24, 144):
        assert _append(L, _shape(rotary_dim=rot)) == INVALID
    for axes in (0, 9):
        assert _append(L, _shape(num_axes=axes)) == INVALID
    for f in ("k_stride", "v_stride"):
        assert _append(L, _shape(**{f: (256, 120)})) == INVALID
    assert _append(L, _shape(n=3, tokens=7, q_stride=(1024, 128)), out=A) == ALIAS  # q itself only when contiguous
    assert _append(L, _shape(n=3, tokens=0)) == OK


def _norm(L, rows=4, cols=256, dtype=gdn.GDN_BF16, x=A, r=2 * A, w=3 * A, eps=1e-6, h=4 * A, y=5 * A, scale=None,
          group=0):
    return L.gdn_add_rmsnorm(rows, cols, dtype, x, r, w, eps, h, y, scale, group, None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(cols=12), UNSUPPORTED), (dict(cols=65544), UNSUPPORTED),
    (dict(dtype=2), UNSUPPORTED), (dict(group=64, scale=6 * A), UNSUPPORTED), (dict(group=128), INVALID),
    (dict(cols=136, group=128, scale=6 * A), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(h=None), INVALID),
    (dict(x=A + 8), INVALID), (dict(w=3 * A + 4), INVALID), (dict(y=5 * A + 8), INVALID), (dict(scale=6 * A + 2), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(h=A + 16), ALIAS), (dict(h=2 * A + 16), ALIAS), (dict(y=2 * A), ALIAS), (dict(y=4 * A), ALIAS),
    (dict(y=A + 16), ALIAS), (dict(y=A, scale=6 * A), ALIAS), (dict(scale=5 * A + 16), ALIAS), (dict(scale=A), ALIAS),
    (dict(h=A, y=A), ALIAS),
])
def test_norm_refusals(L, change, status):
    assert _norm(L, **change) == status


def test_norm_of_nothing(L):
    assert _norm(L, rows=0) == OK


def test_workspace_size(L):
    """Grows with what decides it and never shrinks with the batch."""
    last = 0
    for n in (1, 8, 64, 512):
        size = gdn.gdn_attn_workspace_size(_shape(n=n, tokens=n))
        assert size >= last
        last = size
    with pytest.raises(gdn.GdnError):
        gdn.gdn_attn_workspace_size(_shape(d=64))


@pytest.mark.parametrize("n,tokens", [(0x7fffffff, 0), (0x7fffffff - 600, 0), (0x7ffffff0, 0x7ffffff0), (1 << 30, 1 << 30)])
@pytest.mark.parametrize("prefix", [0, 5])
def test_tables_past_32_bits(L, n, tokens, prefix):
    """Tiles are counted in 32 bits: more sequences and tokens are refused, not given a short workspace."""
    shape = _shape(n=n, tokens=tokens, hq=1, hkv=1, prefix_len=prefix)
    assert L.gdn_attn_workspace_size(ctypes.byref(shape)) == ctypes.c_size_t(-1).value
    assert _attend(L, shape, prefix=10 * A if prefix else None) == UNSUPPORTED
    assert gdn.gdn_attn_workspace_size(_shape(n=1 << 30, tokens=0, hq=1, hkv=1, prefix_len=prefix)) > 36 << 30


# ------------------------------------------------------------------ the binding's own checks

def test_binding_refuses_before_the_library():
    import torch
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    c = torch.zeros(3, 2, 16, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.gdn_paged_attention(q, c, c, i[:, None], i)  # CPU tensors
    with pytest.raises(ValueError):
        gdn.gdn_kv_append(q, q[:, :2], q[:, :2], c, c, i[:, None], i)
    with pytest.raises(TypeError):
        gdn.gdn_add_rmsnorm(q.half(), None, torch.ones(128))
    with pytest.raises(ValueError):
        gdn.gdn_add_rmsnorm(q, None, torch.ones(128))
