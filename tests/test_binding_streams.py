"""Streams and devices of the torch binding's calls, without a GPU.  What a call allocates when it is
given a stream of its own has to belong to that stream, or the allocator hands it to work that is
not ordered with it, and the zeroes of a fresh workspace race the kernels.  Tensors of another
device than the current one are refused: the library launches on the current one."""
import pytest
import torch

import gated_deltanet_linear_05_gb300 as gdn
from gated_deltanet_linear_05_gb300 import build as gdn_build
from pretend import Library, Stream, World, on

SIDE = 777


@pytest.fixture(scope="module", autouse=True)
def _built():
    gdn_build.build()


@pytest.fixture
def attention(monkeypatch):
    """(attention.py over a recording library, the pretended machine)."""
    import ctypes
    from gated_deltanet_linear_05_gb300 import attention as A
    real = gdn.lib()
    world = World(monkeypatch, ctypes.sizeof(gdn.GdnAttnShape))
    library = Library(world, real)
    monkeypatch.setattr(A, "lib", lambda: library)
    monkeypatch.setattr(A, "_raw_stream", lambda device: world.handle)
    monkeypatch.setattr(A, "_current_device", lambda: world.device, raising=False)
    monkeypatch.setattr(A, "_quick", None)  # bound anew to the recording entry points
    A._made.clear()
    yield A, world
    A._made.clear()


def _batch(n=3, hq=4, hkv=2, d=128):
    q = on(torch.zeros(n, hq, d, dtype=torch.bfloat16))
    k, v = (on(torch.zeros(n, hkv, d, dtype=torch.bfloat16)) for _ in range(2))
    kc, vc = (on(torch.zeros(8, hkv, 16, d, dtype=torch.bfloat16)) for _ in range(2))
    table, lens = on(torch.zeros(n, 2, dtype=torch.int32)), on(torch.ones(n, dtype=torch.int32))
    return q, k, v, kc, vc, table, lens


@pytest.mark.parametrize("turn", [1, 2])  # unseen sizes, then seen ones
@pytest.mark.parametrize("prefix", [False, True])
def test_attention_on_a_stream(attention, prefix, turn):
    A, world = attention
    q, _, _, kc, vc, table, lens = _batch()
    for _ in range(turn):
        if prefix:
            o = A.gdn_shared_prefix_attention(q, kc, vc, table[0].contiguous(), 20, table, lens, stream=Stream(SIDE))
        else:
            o = A.gdn_paged_attention(q, kc, vc, table, lens, stream=Stream(SIDE))
    name, args = world.calls[-1]
    assert args[-1] == SIDE and args[-5] == o.data_ptr()
    assert world.made_at(o.data_ptr())[2] == SIDE
    assert world.made_at(args[-3])[2] == SIDE  # the workspace


@pytest.mark.parametrize("turn", [1, 2])
def test_append_on_a_stream(attention, turn):
    A, world = attention
    q, k, v, kc, vc, table, lens = _batch()
    for _ in range(turn):
        out = A.gdn_kv_append(q, k, v, kc, vc, table, lens, stream=Stream(SIDE))
    assert world.calls[-1][1][-1] == SIDE
    assert world.made_at(out.data_ptr())[2] == SIDE


@pytest.mark.parametrize("turn", [1, 2])
@pytest.mark.parametrize("out,group", [("same", 0), ("e4m3", 128)])
def test_norm_on_a_stream(attention, out, group, turn):
    A, world = attention
    x, w = on(torch.ones(3, 256)), on(torch.ones(256))
    for _ in range(turn):
        outputs = A.gdn_add_rmsnorm(x, x, w, out=out, group=group, stream=Stream(SIDE))
    assert world.calls[-1][1][-1] == SIDE
    for t in outputs:
        assert world.made_at(t.data_ptr())[2] == SIDE


def test_given_tensors_are_used(attention):
    """With everything given nothing is allocated, on a stream of its own or not."""
    A, world = attention
    q, _, _, kc, vc, table, lens = _batch()
    ws = A.gdn_attn_workspace(3, 3, 4, 2, 128)
    o = on(torch.empty_like(q))
    world.made.clear()
    for stream in (Stream(SIDE), None):
        assert A.gdn_paged_attention(q, kc, vc, table, lens, o=o, workspace=ws, stream=stream) is o
        assert world.calls[-1][1][-1] == (SIDE if stream else 100)
        assert world.calls[-1][1][-3] == ws.data_ptr()
    assert not world.made


@pytest.mark.parametrize("prefix", [False, True])
def test_fresh_workspaces_zero_their_counters_alone(attention, prefix):
    """A gigabyte of partial results need not be zeroed at every call that brings no workspace."""
    A, world = attention
    n = 1024
    q = on(torch.zeros(n, 32, 128, dtype=torch.bfloat16))
    kc, vc = (on(torch.zeros(2, 8, 16, 128, dtype=torch.bfloat16)) for _ in range(2))
    table, lens = on(torch.zeros(n, 1, dtype=torch.int32)), on(torch.ones(n, dtype=torch.int32))
    world.made.clear()
    if prefix:
        A.gdn_shared_prefix_attention(q, kc, vc, table[0].contiguous(), 5, table, lens)
    else:
        A.gdn_paged_attention(q, kc, vc, table, lens)
    ws = A.gdn_attn_workspace(n, n, 32, 8, 128, prefix_len=5 if prefix else 0)
    assert (ws[:2048] == 0).all()
    name, size, _ = world.made_at(world.calls[-1][1][-3])
    assert size == ws.nbytes
    assert all(name != "zeros" or size <= 2048 for name, _, size, _ in world.made)


# ------------------------------------------------------------------ the delta-rule calls

class Recorder:
    """Entry points that record (name, arguments); the size queries are the real library's."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if "size" in name:
            return getattr(self.real, name)
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def layer(monkeypatch):
    """(the recorder in the library's place, the pretended machine)."""
    rec = Recorder(gdn.lib())
    world = World(monkeypatch, 0)
    monkeypatch.setattr(gdn, "lib", lambda: rec)
    return rec, world


def _layer_tensors(n=2, t=2, hk=2, hv=4):
    bf, f = torch.bfloat16, torch.float32
    z = lambda dtype, *shape: on(torch.zeros(*shape, dtype=dtype))  # noqa: E731
    c = 128 * (2 * hk + hv)
    return dict(q=z(bf, t, hk, 128), k=z(bf, t, hk, 128), v=z(bf, t, hv, 128), g=z(f, t, hv), beta=z(f, t, hv),
                s=z(f, n, hv, 128, 128), cu=z(torch.int32, n + 1), conv_w=z(f, c, 4), A=z(f, hv), dt=z(f, hv),
                conv=z(bf, n, 3, c), w=z(f, 128))


LAYER = {
    "prefill": lambda x, st: gdn.gdn_prefill_chunked(x["q"], x["k"], x["v"], x["g"], x["beta"], None, x["s"], x["cu"], stream=st),
    "prefill, by position": lambda x, st: gdn.gdn_prefill_chunked(x["q"], x["k"], x["v"], x["g"], x["beta"], None, x["s"],
                                                                  x["cu"], None, 64, None, st),
    "split": lambda x, st: gdn.gdn_prefill_split(x["q"], x["k"], x["v"], x["g"], x["beta"], None, x["s"], x["cu"],
                                                 segment_len=64, stream=st),
    "verify": lambda x, st: gdn.gdn_verify_block(x["q"], x["k"], x["v"], x["g"], x["beta"], None, x["s"], x["cu"], stream=st),
    "decode": lambda x, st: gdn.gdn_decode_step(x["q"], x["k"], x["v"], x["g"], x["beta"], None, x["s"], stream=st),
    "prologue": lambda x, st: gdn.gdn_input_prologue(x["q"], x["k"], x["v"], x["g"], x["beta"], x["conv_w"], x["A"], x["dt"],
                                                     None, x["conv"], stream=st),
    "norm": lambda x, st: gdn.gdn_gated_rmsnorm(x["v"], x["v"], x["w"], stream=st),
    "block step": lambda x, st: gdn.gdn_decode_block_step(x["q"], x["k"], x["v"], x["g"], x["beta"], x["conv_w"], x["A"],
                                                          x["dt"], x["conv"], x["conv"], x["s"], x["s"], x["v"], x["w"], stream=st),
    "capture": lambda x, st: gdn.gdn_verify_block_capture(x["q"], x["k"], x["v"], x["g"], x["beta"], None, x["s"], x["cu"], stream=st),
}


@pytest.mark.parametrize("call", LAYER)
def test_delta_rule_calls_on_a_stream(layer, call):
    rec, world = layer
    x = _layer_tensors()
    world.made.clear()
    LAYER[call](x, Stream(SIDE))
    assert rec.calls[-1][1][-1] == SIDE
    assert world.made and all(handle == SIDE for _, _, _, handle in world.made), world.made
    LAYER[call](x, None)
    assert rec.calls[-1][1][-1] == 100


# ------------------------------------------------------------------ devices

def _moved(tensors, index):
    return [on(t, index) for t in tensors]


def _calls(A, q, k, v, kc, vc, table, lens, x, w):
    ws = on(torch.zeros(1 << 22, dtype=torch.uint8), q.get_device())
    prefix = table[0].contiguous()
    return {
        "attention": lambda st: A.gdn_paged_attention(q, kc, vc, table, lens, workspace=ws, stream=st),
        "prefix": lambda st: A.gdn_shared_prefix_attention(q, kc, vc, prefix, 20, table, lens, workspace=ws, stream=st),
        "append": lambda st: A.gdn_kv_append(q, k, v, kc, vc, table, lens, stream=st),
        "norm": lambda st: A.gdn_add_rmsnorm(x, x, w, out="e4m3", stream=st),
    }


@pytest.mark.parametrize("seen", [False, True])
@pytest.mark.parametrize("call", ["attention", "prefix", "append", "norm"])
def test_tensors_of_another_device(attention, call, seen):
    """Refused, whether or not their sizes have been seen; a stream of their device makes it current."""
    A, world = attention
    tensors = _batch() + (on(torch.ones(3, 256)), on(torch.ones(256)))
    here, there = _calls(A, *tensors), _calls(A, *_moved(tensors, 1))
    if seen:
        for _ in range(2):
            here[call](None)
    before = len(world.calls)
    with pytest.raises(ValueError):
        there[call](None)
    with pytest.raises(ValueError):
        here[call](Stream(SIDE, 1))
    assert len(world.calls) == before
    there[call](Stream(SIDE, 1))
    assert len(world.calls) == before + 1 and world.calls[-1][1][-1] == SIDE
    world.device = 1
    there[call](None)
    with pytest.raises(ValueError):
        here[call](None)
    assert len(world.calls) == before + 2


@pytest.mark.parametrize("call", LAYER)
def test_delta_rule_tensors_of_another_device(layer, call):
    rec, world = layer
    x = _layer_tensors()
    there = {k: on(t, 1) for k, t in x.items()}
    with pytest.raises(ValueError):
        LAYER[call](there, None)
    with pytest.raises(ValueError):
        LAYER[call]({**x, "v": there["v"]}, None)
    with pytest.raises(ValueError):
        LAYER[call](x, Stream(SIDE, 1))
    assert not rec.calls
    LAYER[call](there, Stream(SIDE, 1))
    assert rec.calls[-1][1][-1] == SIDE


# ------------------------------------------------------------------ the interpreter lock

@pytest.mark.parametrize("call", ["attention", "append", "norm"])
def test_other_threads_run_while_a_launch_waits(attention, call):
    """A launch blocks while the stream's queue is full: the interpreter lock is not held meanwhile (a
    host function on the stream may need it).  The launch here is 0.4 s of sleep."""
    import threading
    import time
    A, world = attention
    tensors = _batch() + (on(torch.ones(3, 256)), on(torch.ones(256)))
    calls = _calls(A, *tensors)
    calls[call](None)  # sizes seen
    # as the entry point: a C function that sleeps, whatever its arguments
    sleep = _sleeper()
    library = A.lib()
    for name in ("gdn_paged_attention", "gdn_kv_append", "gdn_add_rmsnorm"):
        setattr(library, name, getattr(sleep, name))
    A._quick = None
    count, stop = [0], threading.Event()

    def work():
        while not stop.is_set():
            count[0] += 1
            time.sleep(0.01)

    t = threading.Thread(target=work)
    t.start()
    try:
        time.sleep(0.05)
        before = count[0]
        calls[call](None)
        after = count[0]
    finally:
        stop.set()
        t.join()
    assert after - before >= 5  # of about 40


def _sleeper():
    """A library whose entry points sleep 0.4 s and return GDN_OK."""
    import ctypes
    import os
    import subprocess
    import tempfile
    with tempfile.TemporaryDirectory() as d:
        src, so = os.path.join(d, "s.c"), os.path.join(d, "s.so")
        with open(src, "w") as f:
            f.write("#include <unistd.h>\n" + "".join(
                "int %s() { usleep(400000); return 0; }\n" % n
                for n in ("gdn_paged_attention", "gdn_kv_append", "gdn_add_rmsnorm")))
        subprocess.run(["gcc", "-std=gnu11", "-shared", "-fPIC", src, "-o", so], check=True)
        return ctypes.CDLL(so)
