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
