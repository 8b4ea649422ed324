"""The two ways of marshalling of the calls for trees and beams: both make the same C call, errors keep their
kinds, streams and devices are the call's, and no reference is lost."""
import gc
import sys

import pytest
import torch

import gated_deltanet_linear_05_gb300 as gdn
import pretend
from gated_deltanet_linear_05_gb300 import build as gdn_build
from pretend import I32, I64, P, S, Library, Stream, World, on

NEW = dict(gdn_tree_attention=[P] * 13 + [S, P], gdn_verify_tree=[P] * 12, gdn_beam_select=[P] * 8 + [S, P],
           gdn_beam_reorder=[I32, I32, I32, I64, P, P, P])


@pytest.fixture(scope="module", autouse=True)
def _built():
    gdn_build.build()


@pytest.fixture
def world(monkeypatch):
    from gated_deltanet_linear_05_gb300 import attention as A
    from gated_deltanet_linear_05_gb300 import branching as B
    monkeypatch.setattr(pretend, "SIGNATURES", {**pretend.SIGNATURES, **NEW})
    w = World(monkeypatch, 32)  # (no struct is shorter)
    library = Library(w, gdn.lib())
    for m in (A, B):
        for name, value in (("lib", lambda: library), ("_raw_stream", lambda d: w.handle), ("_current_device", lambda: w.device)):
            monkeypatch.setattr(m, name, value)
    monkeypatch.setattr(A, "_quick", None)
    A._made.clear(), B._made.clear()
    w.A, w.B, w.monkeypatch = A, B, monkeypatch
    yield w
    A._made.clear(), B._made.clear()


def once(world, f):
    world.made.clear()
    out = f()
    name, args = world.calls.pop()
    assert not world.calls
    where = {t.data_ptr(): i for i, t in enumerate(out if isinstance(out, tuple) else (out,))}
    new = {a for _, a, _, _ in world.made}
    return name, [("output", where[a]) if type(a) is int and a in where and a in new else a for a in args]


def both(world, f):
    """The C call from the Python side and from the module."""
    first = once(world, f)

    def refuse(*args):
        raise AssertionError("the module handed the call back")

    with world.monkeypatch.context() as m:
        for module, name in ((world.A, "_check"), (world.B, "_check_tensors"), (world.B, "_kind"), (world.B, "_on_current")):
            m.setattr(module, name, refuse)
        assert once(world, f) == first
    return first


def zeros(*shape, dtype=torch.float32):
    return on(torch.zeros(*shape, dtype=dtype))


@pytest.mark.parametrize("prefix", [False, True])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("given", [False, True])
def test_tree_attention(world, prefix, gate, given):
    q, g, o = (zeros(7, 4, 128, dtype=torch.bfloat16) for _ in range(3))
    kc, vc = (zeros(8, 2, 16, 128, dtype=torch.bfloat16) for _ in range(2))
    ints = lambda *shape: zeros(*shape, dtype=torch.int32)  # noqa: E731
    table, lens, cu, up, ptable = ints(3, 2), ints(3), ints(4), ints(7), ints(2)
    kw = dict(gate=g if gate else None, o=o if given else None, workspace=zeros(1 << 27, dtype=torch.uint8))
    if prefix:
        kw.update(prefix_table=ptable, prefix_len=20)
    name, args = both(world, lambda: gdn.gdn_tree_attention(q, kc, vc, table, lens, cu, up, **kw))
    assert name == "gdn_tree_attention"
    assert args[1:11] == [q.data_ptr(), g.data_ptr() if gate else 0, kc.data_ptr(), vc.data_ptr(), ptable.data_ptr() if prefix else 0,
                          table.data_ptr(), lens.data_ptr(), cu.data_ptr(), up.data_ptr(), o.data_ptr() if given else ("output", 0)]
    for bad in (up[:6], up.long(), up.float(), ints(7, 1), ints(14)[::2], on(torch.ones(7, dtype=torch.int32), 1)):
        with pytest.raises((ValueError, TypeError)):  # also where the rest has been seen
            gdn.gdn_tree_attention(q, kc, vc, table, lens, cu, bad, **kw)
    with pytest.raises(ValueError):
        gdn.gdn_tree_attention(q, kc, vc, table, lens, None, up, **kw)
    assert not world.calls


def _tree(dtype=torch.bfloat16):
    return dict(q=zeros(5, 2, 128, dtype=dtype), k=zeros(5, 2, 128, dtype=dtype), v=zeros(5, 4, 128, dtype=dtype), g=zeros(5, 4),
                beta=zeros(5, 4), state_in=zeros(2, 4, 128, 128), cu_seqlens=zeros(3, dtype=torch.int32),
                parents=zeros(5, dtype=torch.int32))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("given", ["none", "o", "fp32 o", "delta", "both"])
def test_verify(world, dtype, state, given):
    t = _tree(dtype)
    if not state:
        t["state_in"] = None
    o = zeros(5, 4, 128, dtype=torch.float32 if given == "fp32 o" else dtype) if given in ("o", "fp32 o", "both") else None
    delta = zeros(5, 4, 128) if given in ("delta", "both") else None
    name, args = both(world, lambda: gdn.gdn_verify_tree(**t, o=o, delta=delta, chunk=16))
    assert name == "gdn_verify_tree"
    assert args[1:9] == [0 if x is None else x.data_ptr() for x in t.values()]
    assert args[9:11] == [("output", 0) if o is None else o.data_ptr(), ("output", 1) if delta is None else delta.data_ptr()]
    assert args[11] == world.handle


def test_verify_refuses(world):
    t = _tree()
    gdn.gdn_verify_tree(**t)  # seen
    world.calls.clear()
    for name, bad in [("k", zeros(5, 2, 128)), ("k", zeros(4, 2, 128, dtype=torch.bfloat16)), ("v", zeros(5, 4, 64, dtype=torch.bfloat16)),
                      ("g", zeros(5, 2)), ("beta", zeros(5, 4, dtype=torch.float64)), ("state_in", zeros(3, 4, 128, 128)),
                      ("state_in", zeros(2, 4, 128, 128, dtype=torch.bfloat16)), ("cu_seqlens", zeros(3)), ("parents", zeros(4, dtype=torch.int32)),
                      ("q", zeros(5, 2, 256, dtype=torch.bfloat16)[..., :128]), ("parents", on(torch.ones(5, dtype=torch.int32), 1)),
                      ("q", torch.ones(5, 2, 128, dtype=torch.bfloat16)), ("v", zeros(5, 512, dtype=torch.bfloat16))]:
        with pytest.raises((ValueError, TypeError)):
            gdn.gdn_verify_tree(**{**t, name: bad})
    for kw in (dict(o=zeros(5, 4, 128, dtype=torch.float16)), dict(o=zeros(5, 2, 128, dtype=torch.bfloat16)),
               dict(delta=zeros(5, 4, 128, dtype=torch.bfloat16))):
        with pytest.raises((ValueError, TypeError)):
            gdn.gdn_verify_tree(**t, **kw)
    assert not world.calls


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("finished", [False, True])
@pytest.mark.parametrize("pad", [0, 3])
def test_select(world, dtype, finished, pad):
    x = zeros(2, 3, 40 + pad, dtype=dtype)[..., :40]
    s, f, ws = zeros(2, 3), zeros(2, 3, dtype=torch.bool), zeros(1 << 20, dtype=torch.uint8)
    name, args = both(world, lambda: gdn.gdn_beam_select(x, s, 4, finished=f if finished else None, pad_token=pad, workspace=ws))
    assert name == "gdn_beam_select"
    assert args[1:4] == [x.data_ptr(), s.data_ptr(), f.data_ptr() if finished else 0]
    assert args[4:9] == [("output", 0), ("output", 1), ("output", 2), ws.data_ptr(), ws.nbytes]
    shape = gdn.GdnBeamShape.from_buffer_copy(args[0])
    assert (shape.num_groups, shape.beams, shape.vocab, shape.top, shape.pad_token, shape.row_stride) == (2, 3, 40, 4, pad, 40 + pad)
    for kw in (dict(scores=zeros(2, 4)), dict(scores=zeros(2, 3, dtype=torch.float64)), dict(scores=zeros(2, 6)[:, ::2]),
               dict(finished=zeros(2, 3)), dict(finished=zeros(3, 2, dtype=torch.bool)), dict(logits=torch.ones(2, 3, 40)),
               dict(scores=on(torch.ones(2, 3), 1)), dict(workspace=on(torch.ones(8, dtype=torch.uint8), 1))):
        a = dict(logits=x, scores=s, top=4, finished=f if finished else None, pad_token=pad, workspace=ws)
        with pytest.raises((ValueError, TypeError)):
            gdn.gdn_beam_select(**{**a, **kw})
    assert not world.calls


def test_reorder(world):
    up = zeros(2, 3, dtype=torch.int32)
    for x in (zeros(2, 6, 4, 128), zeros(1, 6, 7, dtype=torch.int32), zeros(3, 6, dtype=torch.float32)):
        name, args = both(world, lambda: gdn.gdn_beam_reorder(x, up))
        assert (name, args) == ("gdn_beam_reorder", [x.shape[0], 2, 3, x[0, 0].nbytes, up.data_ptr(), x.data_ptr(), world.handle])
    for rows, p in ((zeros(2, 5, 4), up), (zeros(6), up), (zeros(2, 6, 8)[..., ::2], up), (zeros(2, 6, 4), up.long()),
                    (zeros(2, 6, 4), up[0]), (zeros(2, 6, 4), on(torch.ones(2, 3, dtype=torch.int32), 1)), (torch.ones(2, 6, 4), up)):
        with pytest.raises((ValueError, TypeError)):
            gdn.gdn_beam_reorder(rows, p)
    assert not world.calls


def test_given_stream(world):
    """What a call allocates belongs to the stream that it is given."""
    side = Stream(900)
    x, s = zeros(2, 3, 40), zeros(2, 3)
    t = _tree()
    q = zeros(5, 2, 128, dtype=torch.bfloat16)
    kc = zeros(2, 2, 16, 128, dtype=torch.bfloat16)
    table, lens = zeros(2, 1, dtype=torch.int32), zeros(2, dtype=torch.int32)
    for f in (lambda: gdn.gdn_beam_select(x, s, 4, stream=side), lambda: gdn.gdn_verify_tree(**t, stream=side),
              lambda: gdn.gdn_tree_attention(q, kc, kc, table, lens, t["cu_seqlens"], t["parents"], stream=side),
              lambda: gdn.gdn_beam_reorder(zeros(1, 6, 4), zeros(2, 3, dtype=torch.int32), stream=side)):
        for _ in range(2):
            world.made.clear()
            f()
            name, args = world.calls.pop()
            assert args[-1] == 900, name
            assert all(handle == 900 for fn, _, size, handle in world.made if fn != "zeros"), name
    assert world.handle == 100


@pytest.mark.gpu
def test_references_stay():
    from tree_testlib import DeltaBatch
    b = DeltaBatch([5, 9], 1, 2, "bf16", seed=1)
    x, s = torch.randn(2, 3, 500, device="cuda"), torch.zeros(2, 3, device="cuda")
    f, ws = torch.zeros(2, 3, dtype=torch.bool, device="cuda"), gdn.gdn_beam_workspace(2, 3, 500, 4)
    rows = torch.zeros(2, 6, 64, device="cuda")

    def calls():
        gdn.gdn_verify_tree(*b.args(), chunk=16)
        _, up, _ = gdn.gdn_beam_select(x, s, 3, finished=f, workspace=ws)
        gdn.gdn_beam_reorder(rows, up)
        try:
            gdn.gdn_beam_select(x, s, 3, finished=f, workspace=ws[:256])
        except gdn.GdnError:
            pass

    held = (*b.args(), x, s, f, ws, rows, torch.float32, torch.int32, torch.bool, torch.bfloat16)
    for _ in range(3):
        calls()
    torch.cuda.synchronize()
    gc.collect()
    before, memory = [sys.getrefcount(t) for t in held], torch.cuda.memory_allocated()
    for _ in range(200):
        calls()
    torch.cuda.synchronize()
    gc.collect()
    assert all(abs(a - c) <= 2 for a, c in zip(before, [sys.getrefcount(t) for t in held]))
    assert torch.cuda.memory_allocated() <= memory + (1 << 16)
