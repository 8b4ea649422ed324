"""The attention calls' marshalling module (csrc/marshal.c): what it hands back to the Python side,
that both sides give the same, that errors keep their kinds, and that no reference is lost."""
import gc
import sys

import pytest

import gated_deltanet_linear_05_gb300 as gdn
from gated_deltanet_linear_05_gb300 import build as gdn_build


@pytest.fixture(scope="module", autouse=True)
def _built():
    gdn_build.build()


def _attention():
    from gated_deltanet_linear_05_gb300 import attention
    return attention


def test_module_hands_back_what_it_does_not_know():
    import torch
    quick = _attention()._fast()
    t = torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    c = torch.zeros(1, 2, 16, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    assert quick.attend({}, t, c, c, None, 0, i[:, None], i, None, None, None, None, t) is None  # CPU tensors
    assert quick.append({}, t, t, t, c, c, i[:, None], i, None, None, None, None, None, None, 1e-6, None, 0) is None
    assert quick.norm({}, t, None, torch.ones(128), 1e-6, "same", 0) is None
    with pytest.raises(TypeError):
        quick.attend({}, t)
    with pytest.raises(AttributeError):
        quick.norm({}, 1, None, t, 1e-6, "same", 0)


def _batch():
    from attn_testlib import Batch
    b = Batch([1, 1], [40, 70], 4, 2, 128, 16, gate=True, seed=1)
    return b, gdn.gdn_attn_workspace(2, 2, 4, 2, 128)


@pytest.mark.gpu
def test_seen_and_unseen_calls_agree():
    import torch
    A = _attention()
    b, ws = _batch()
    args = (b.q, b.k_cache, b.v_cache, b.page_table, b.kv_lens)
    A._made.clear()
    first = gdn.gdn_paged_attention(*args, gate=b.gate, workspace=ws)  # not seen: the Python side
    again = gdn.gdn_paged_attention(*args, gate=b.gate, workspace=ws)  # seen
    given = torch.empty_like(first)
    assert gdn.gdn_paged_attention(*args, gate=b.gate, workspace=ws, o=given) is given
    side = torch.cuda.Stream()  # a stream of its own: the Python side
    side.wait_stream(torch.cuda.current_stream())
    other = gdn.gdn_paged_attention(*args, gate=b.gate, workspace=ws, stream=side)
    torch.cuda.synchronize()
    for o in (again, given, other):
        assert torch.equal(first, o)
    x, r, w = torch.randn(5, 256, device="cuda"), torch.randn(5, 256, device="cuda"), torch.ones(256, device="cuda")
    for kw in (dict(), dict(out="e4m3"), dict(out="e4m3", group=128)):
        one, two = (gdn.gdn_add_rmsnorm(x, r, w, **kw) for _ in range(2))
        assert len(one) == len(two) and all(torch.equal(p.float(), q.float()) for p, q in zip(one, two))
    y, h = gdn.gdn_add_rmsnorm(x, None, w)
    y, h = gdn.gdn_add_rmsnorm(x, None, w)
    assert h is x
    q, k, v = (torch.randn(2, n, 128, device="cuda").bfloat16() for n in (4, 2, 2))
    f = torch.ones(16, dtype=torch.float64, device="cuda")
    outs = [gdn.gdn_kv_append(q, k, v, b.k_cache, b.v_cache, b.page_table, b.kv_lens, f) for _ in range(2)]
    torch.cuda.synchronize()
    assert torch.equal(*outs)


@pytest.mark.gpu
def test_errors_of_seen_calls():
    """After a call has been seen, a wrong tensor of the same sizes still meets its error."""
    import torch
    b, ws = _batch()
    args = [b.q, b.k_cache, b.v_cache, b.page_table, b.kv_lens]
    for _ in range(2):
        gdn.gdn_paged_attention(*args, workspace=ws)
    for at, wrong, error in ((0, b.q.half(), TypeError), (1, b.k_cache.half(), TypeError), (3, b.page_table.long(), ValueError),
                             (4, b.kv_lens.cpu(), ValueError), (3, b.page_table.t().contiguous().t(), ValueError)):
        bad = list(args)
        bad[at] = wrong
        with pytest.raises(error):
            gdn.gdn_paged_attention(*bad, workspace=ws)
    with pytest.raises(gdn.GdnError):
        gdn.gdn_paged_attention(*args, workspace=ws[:1000])  # too small
    with pytest.raises(ValueError):
        gdn.gdn_paged_attention(*args, workspace=ws, o=torch.empty_like(b.q)[:1])
    with pytest.raises(gdn.GdnError):
        gdn.gdn_paged_attention(b.q, *args[1:], workspace=ws, o=b.q)  # over q itself
    x = torch.ones(3, 128, device="cuda")
    for _ in range(2):
        gdn.gdn_add_rmsnorm(x, x, torch.ones(128, device="cuda"))
    with pytest.raises(ValueError):
        gdn.gdn_add_rmsnorm(x, x.t().contiguous().t(), torch.ones(128, device="cuda"))
    with pytest.raises(ValueError):
        gdn.gdn_add_rmsnorm(x, x, torch.ones(64, device="cuda"))
    with pytest.raises(gdn.GdnError):
        gdn.gdn_add_rmsnorm(x, x, torch.ones(128, device="cuda"), eps=-1.0)


@pytest.mark.gpu
def test_references_stay():
    import torch
    b, ws = _batch()
    x, r, w = torch.randn(5, 256, device="cuda"), torch.randn(5, 256, device="cuda"), torch.ones(256, device="cuda")
    q, k, v = (torch.randn(2, n, 128, device="cuda").bfloat16() for n in (4, 2, 2))

    def calls():
        gdn.gdn_paged_attention(b.q, b.k_cache, b.v_cache, b.page_table, b.kv_lens, gate=b.gate, workspace=ws)
        gdn.gdn_add_rmsnorm(x, r, w, out="e4m3", group=128)
        gdn.gdn_kv_append(q, k, v, b.k_cache, b.v_cache, b.page_table, b.kv_lens)
        try:
            gdn.gdn_paged_attention(b.q, b.k_cache, b.v_cache, b.page_table, b.kv_lens, gate=b.gate, workspace=ws[:256])
        except gdn.GdnError:
            pass

    held = (b.q, b.k_cache, b.page_table, b.kv_lens, b.gate, ws, x, r, w, q, k, torch.bfloat16, torch.float32,
            torch.float8_e4m3fn)
    for _ in range(3):
        calls()
    torch.cuda.synchronize()
    gc.collect()
    before, memory = [sys.getrefcount(t) for t in held], torch.cuda.memory_allocated()
    for _ in range(200):
        calls()
    torch.cuda.synchronize()
    gc.collect()
    after = [sys.getrefcount(t) for t in held]
    assert all(abs(a - c) <= 2 for a, c in zip(before, after)), (before, after)
    assert torch.cuda.memory_allocated() <= memory + (1 << 16)


# ------------------------------------------------------------------ without the module

def test_calls_without_the_module(monkeypatch):
    """The Python side does all that the module does: without it the calls work, a little slower."""
    import ctypes
    import torch
    from pretend import Library, World, on
    A = _attention()
    world = World(monkeypatch, ctypes.sizeof(gdn.GdnAttnShape))
    library = Library(world, gdn.lib())
    for name, value in (("lib", lambda: library), ("_raw_stream", lambda d: world.handle), ("_current_device", lambda: 0),
                        ("_quick", None)):
        monkeypatch.setattr(A, name, value)
    monkeypatch.setitem(sys.modules, "gated_deltanet_linear_05_gb300._marshal", None)
    monkeypatch.delattr(gdn, "_marshal", raising=False)
    x, w = on(torch.ones(3, 256)), on(torch.ones(256))
    for _ in range(2):
        y, scale, h = A.gdn_add_rmsnorm(x, x, w, out="e4m3")
        assert world.calls[-1][1][7:10] == [h.data_ptr(), y.data_ptr(), scale.data_ptr()]
    q = on(torch.zeros(2, 2, 128, dtype=torch.bfloat16))
    c = on(torch.zeros(1, 2, 16, 128, dtype=torch.bfloat16))
    i = on(torch.zeros(2, 1, dtype=torch.int32))
    for _ in range(2):
        assert A.gdn_kv_append(q, q, q, c, c, i, i[:, 0].contiguous()).data_ptr() == world.calls[-1][1][-4]
        assert A.gdn_paged_attention(q, c, c, i, i[:, 0].contiguous()).data_ptr() == world.calls[-1][1][-5]
    assert len(world.calls) == 6
    A._made.clear()


def test_build_without_python_headers(monkeypatch, tmp_path):
    """The library is what a build has to make; the module is left out where Python.h is not there."""
    monkeypatch.setattr(gdn_build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    monkeypatch.setattr(gdn_build, "MARSHAL", str(tmp_path / "_marshal.so"))
    assert gdn_build.build() == gdn_build.LIB
    assert not (tmp_path / "_marshal.so").exists()


# ------------------------------------------------------------------ both ways make the same C call

@pytest.fixture
def ways(monkeypatch):
    """call(f, outputs) -> the C call's arguments from the Python side and from the module, with the
    addresses of the outputs that the call made replaced by their places in what it returned."""
    import ctypes
    from pretend import Library, World
    A = _attention()
    world = World(monkeypatch, ctypes.sizeof(gdn.GdnAttnShape))
    library = Library(world, gdn.lib())
    for name, value in (("lib", lambda: library), ("_raw_stream", lambda d: world.handle), ("_current_device", lambda: 0),
                        ("_quick", None)):
        monkeypatch.setattr(A, name, value)
    A._made.clear()

    def once(f):
        world.made.clear()
        out = f(A)
        out = out if isinstance(out, tuple) else (out,)
        name, args = world.calls.pop()
        assert not world.calls
        where = {t.data_ptr(): i for i, t in enumerate(out)}
        new = {a for _, a, _, _ in world.made}
        shapes = [(t.shape, t.dtype, t.is_contiguous()) for t in out]
        return name, [("output", where[a]) if type(a) is int and a in where and a in new else a for a in args], shapes

    def both(f):
        A._made.clear()
        first = once(f)

        def refuse(*args):
            raise AssertionError("the module handed the call back")

        with monkeypatch.context() as m:
            for name in ("_check", "_norm_plan", "_alike"):
                m.setattr(A, name, refuse)
            second = once(f)
        return first, second

    yield both
    A._made.clear()


def _rows(tokens, heads, d, pad):
    """[tokens, heads, d] bf16 with padded strides, or head-major."""
    import torch
    from pretend import on
    if pad == "head-major":
        return on(torch.zeros(heads, tokens, d, dtype=torch.bfloat16)).transpose(0, 1)
    return on(torch.zeros(tokens, heads * (d + pad) + pad, dtype=torch.bfloat16)).as_strided(
        (tokens, heads, d), (heads * (d + pad) + pad, d + pad, 1))


def _cache(hkv=2, d=128):
    import torch
    from pretend import on
    kc, vc = (on(torch.zeros(8, hkv, 16, d, dtype=torch.bfloat16)) for _ in range(2))
    ints = lambda *shape: on(torch.zeros(*shape, dtype=torch.int32))  # noqa: E731
    return kc, vc, ints(3, 2), ints(3), ints(4), ints(2)


@pytest.mark.parametrize("prefix", [False, True])
@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("gate", [None, 0, 8, "head-major"])
@pytest.mark.parametrize("given", [False, True])
def test_both_ways_attention(ways, prefix, rows, gate, given):
    import torch
    from pretend import on
    kc, vc, table, lens, cu, ptable = _cache()
    tokens = 7 if rows else 3
    for pad in (0, 8, "head-major"):
        q = _rows(tokens, 4, 128, pad)
        g = None if gate is None else _rows(tokens, 4, 128, gate)
        o = on(torch.zeros(tokens, 4, 128, dtype=torch.bfloat16)) if given else None
        ws = on(torch.zeros(1 << 27, dtype=torch.uint8))
        kw = dict(cu_seqlens=cu if rows else None, gate=g, o=o, workspace=ws, scale=0.25 if given else None)

        def f(A):
            if prefix:
                return A.gdn_shared_prefix_attention(q, kc, vc, ptable, 20, table, lens, **kw)
            return A.gdn_paged_attention(q, kc, vc, table, lens, **kw)

        first, second = ways(f)
        assert first == second
        assert first[1][-5] == (o.data_ptr() if given else ("output", 0))
        assert first[1][1] == q.data_ptr() and first[1][2] == (g.data_ptr() if gate is not None else 0)


@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("rope", ["none", "places", "positions", "axes", "axes without a choice"])
@pytest.mark.parametrize("norms", ["none", "q", "k", "both"])
@pytest.mark.parametrize("given", [False, True])
def test_both_ways_append(ways, rows, rope, norms, given):
    import torch
    from pretend import on
    kc, vc, table, lens, cu, _ = _cache()
    tokens = 7 if rows else 3
    q, k, v = _rows(tokens, 4, 128, 8), _rows(tokens, 2, 128, 0), _rows(tokens, 2, 128, "head-major")
    w = on(torch.ones(128)), on(torch.ones(128))
    kw = dict(cu_seqlens=cu if rows else None, q_norm=w[0] if norms in ("q", "both") else None,
              k_norm=w[1] if norms in ("k", "both") else None, eps=1e-5, prefix_len=40 if given else 0,
              q_out=on(torch.zeros(tokens, 4, 128, dtype=torch.bfloat16)) if given else None)
    if rope != "none":
        kw["inv_freq"] = on(torch.ones(16, dtype=torch.float64))
    if rope == "positions":
        kw["positions"] = on(torch.zeros(tokens, dtype=torch.int32))
    if rope.startswith("axes"):
        kw["positions"] = on(torch.zeros(3, tokens, dtype=torch.int32))
    if rope == "axes":
        kw["rope_axis"] = on(torch.zeros(16, dtype=torch.int32))
    first, second = ways(lambda A: A.gdn_kv_append(q, k, v, kc, vc, table, lens, **kw))
    assert first == second
    shape = gdn.GdnAttnShape.from_buffer_copy(first[1][0])
    assert (shape.num_seqs, shape.total_tokens, shape.num_q_heads, shape.num_kv_heads) == (3, tokens, 4, 2)
    assert shape.rotary_dim == (0 if rope == "none" else 32) and shape.num_axes == (3 if rope.startswith("axes") else 1)
    assert shape.prefix_len == kw["prefix_len"] and list(shape.v_stride) == [128, tokens * 128]
    assert first[1][4:7] == [kw[n].data_ptr() if kw[n] is not None else 0 for n in ("q_norm", "k_norm")] + [
        pytest.approx(1e-5, rel=2 ** -23)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("out,group", [("same", 0), ("e4m3", 0), ("e4m3", 128)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("shape", [(3, 256), (2, 5, 128), (256,), (0, 128)])
def test_both_ways_norm(ways, residual, out, group, dtype, shape):
    import torch
    from pretend import on
    x, r = (on(torch.zeros(shape, dtype=getattr(torch, dtype))) for _ in range(2))
    w = on(torch.ones(shape[-1]))
    first, second = ways(lambda A: A.gdn_add_rmsnorm(x, r if residual else None, w, 1e-5, out=out, group=group))
    if 0 not in shape:  # (empty tensors have no addresses to tell them apart)
        assert first == second
    assert first[1][:3] == second[1][:3] and first[2] == second[2]
    assert len(first[2]) == (2 if out == "same" else 3)
