"""Calls that are given a stream of their own, without a workspace or outputs, while the current
stream is busy and fills whatever memory the allocator hands it: the results are those of a quiet
call, bit for bit (no result depends on the order of execution)."""
import pytest
import torch

from attn_testlib import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_deltanet_linear_05_gb300 import build
    build.build()


def _beside_a_busy_stream(call, sizes):
    """call(stream) with a side stream, its outputs; the current stream is some ms behind and then
    fills new buffers of these sizes."""
    side, a = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        a = a @ a * 1e-3
    out = call(side)
    for size in sizes:
        for _ in range(3):
            torch.empty(size, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("prefix", [0, 500])
@pytest.mark.parametrize("t,lens", [([1, 1], [9001, 20000]), ([20, 2], [12000, 3])])
def test_attention_beside_a_busy_stream(t, lens, prefix):
    import gated_deltanet_linear_05_gb300 as gdn
    b = Batch(t, lens, 4, 1, 128, 64, prefix=prefix, gate=True, seed=61)
    cu = None if t == [1, 1] else b.cu

    def call(stream, ws=None):
        args = (b.page_table, b.kv_lens, cu, b.gate)
        if prefix:
            return gdn.gdn_shared_prefix_attention(b.q, b.k_cache, b.v_cache, b.prefix_table, prefix, *args,
                                                   workspace=ws, stream=stream)
        return gdn.gdn_paged_attention(b.q, b.k_cache, b.v_cache, *args, workspace=ws, stream=stream)

    ws = gdn.gdn_attn_workspace(len(t), sum(t), 4, 1, 128, prefix_len=prefix)
    want = call(None, ws)
    for _ in range(3):
        got = _beside_a_busy_stream(call, [ws.numel(), b.q.nbytes])
        assert torch.equal(got, want)


def test_append_and_norm_beside_a_busy_stream():
    import gated_deltanet_linear_05_gb300 as gdn
    b = Batch([30, 9], [40, 9], 4, 2, 128, 16, seed=62)
    k, v = (torch.randn(39, 2, 128, device="cuda").bfloat16() for _ in range(2))
    freq = torch.ones(16, dtype=torch.float64, device="cuda")
    append = lambda stream: gdn.gdn_kv_append(  # noqa: E731
        b.q, k, v, b.k_cache, b.v_cache, b.page_table, b.kv_lens, freq, b.cu, stream=stream)
    x, w = torch.randn(300, 4096, device="cuda"), torch.ones(4096, device="cuda")
    norm = lambda stream: gdn.gdn_add_rmsnorm(x, x, w, out="e4m3", group=128, stream=stream)  # noqa: E731
    q, (y, scale, h) = append(None), norm(None)
    for _ in range(3):
        assert torch.equal(_beside_a_busy_stream(append, [b.q.nbytes]), q)
        y2, scale2, h2 = _beside_a_busy_stream(norm, [x.nbytes, y.nbytes, scale.nbytes])
        assert torch.equal(y2.float(), y.float()) and torch.equal(scale2, scale) and torch.equal(h2, h)


def test_decode_block_step_beside_a_busy_stream():
    """The fused decode step without a workspace: its counters are zeroed on the call's own stream."""
    import gated_deltanet_linear_05_gb300 as gdn
    g = torch.Generator().manual_seed(63)
    n, hk, hv = 6, 4, 8
    c = 128 * (2 * hk + hv)
    r = lambda dtype, *shape: torch.randn(*shape, generator=g).to(dtype).cuda()  # noqa: E731
    bf, f = torch.bfloat16, torch.float32
    q, k, v, z = (r(bf, n, h, 128) for h in (hk, hk, hv, hv))
    a, b, w, conv = r(f, n, hv), r(f, n, hv), r(f, c, 4), r(bf, n, 3, c)
    A, dt, state, norm = r(f, hv), r(f, hv), r(f, n, hv, 128, 128), r(f, 128)
    conv_out, state_out = torch.empty_like(conv), torch.empty_like(state)
    step = lambda stream: gdn.gdn_decode_block_step(  # noqa: E731
        q, k, v, a, b, w, A, dt, conv, conv_out, state, state_out, z, norm, stream=stream)[0]
    want = step(None).clone()
    want_state = state_out.clone()
    size = gdn.gdn_workspace_size(gdn.make_shape(n, n, hk, hv), gdn.GDN_OP_DECODE_BLOCK) + 256
    for _ in range(3):
        assert torch.equal(_beside_a_busy_stream(step, [size, z.nbytes]), want)
        assert torch.equal(state_out, want_state)
