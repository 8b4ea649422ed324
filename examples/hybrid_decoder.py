"""A small hybrid decoder served through libgdn: gated delta-rule layers and, every fourth layer,
a gated softmax-attention layer over a paged cache.  Random weights, random "tokens".

    python examples/hybrid_decoder.py

A system prompt is read once; several requests continue from it: their delta-rule layers start
from a copy of its state, their attention layers share its pages of the cache.  Each request's own
prompt is read in one packed call, then all of them go token by token.  At the end the same
sequences are read in one piece, without the shared prefix, and the outputs compared.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_linear_05_gb300 as gdn  # noqa: E402

BF16 = torch.bfloat16


class Layer:
    """Weights of one layer: projections in and out, norms, and what its kind needs."""

    def __init__(self, kind, hidden, g, device):
        def normal(*shape, std=None):
            std = 1 / math.sqrt(shape[-1]) if std is None else std
            return (torch.randn(*shape, generator=g) * std).to(device)

        self.kind = kind
        self.norm = 1 + normal(hidden, std=0.1)
        if kind == "delta":
            self.hk, self.hv, d = 2, 4, 128
            self.width = (2 * self.hk + self.hv) * d
            self.w_in = normal(self.width + self.hv * d, hidden).to(BF16)  # q, k, v, z
            self.w_gates = normal(2 * self.hv, hidden).to(BF16)            # a, b
            self.conv = normal(self.width, gdn.GDN_CONV_WIDTH, std=0.5)
            self.A_log, self.dt_bias = normal(self.hv, std=0.5), normal(self.hv, std=0.5)
            self.out_norm = 1 + normal(d, std=0.1)
            self.w_out = normal(hidden, self.hv * d).to(BF16)
        else:
            self.hq, self.hkv, self.d, rot = 8, 2, 256, 64
            self.w_in = normal((2 * self.hq + 2 * self.hkv) * self.d, hidden).to(BF16)  # q, gate, k, v
            self.q_norm, self.k_norm = 1 + normal(self.d, std=0.1), 1 + normal(self.d, std=0.1)
            self.inv_freq = torch.tensor([1e7 ** (-2 * i / rot) for i in range(rot // 2)],
                                         dtype=torch.float64, device=device)
            self.w_out = normal(hidden, self.hq * self.d).to(BF16)


class Cache:
    """Pages of one attention layer."""

    def __init__(self, layer, pages, page, device):
        shape = (pages, layer.hkv, page, layer.d)
        self.k, self.v = (torch.empty(shape, dtype=BF16, device=device) for _ in range(2))


class Batch:
    """Sequences that are served together: their delta states, pages and lengths."""

    def __init__(self, model, count, most, prefix=None):
        n, dev = count, model.device
        self.prefix = prefix
        self.tables = model.take_pages(n * -(-most // model.page)).view(n, -1)
        self.lens = torch.zeros(n, dtype=torch.int32, device=dev)
        self.state, self.conv = {}, {}
        for i, l in enumerate(model.layers):
            if l.kind != "delta":
                continue
            if prefix is None:
                self.state[i] = torch.zeros(n, l.hv, 128, 128, device=dev)
                self.conv[i] = torch.zeros(n, gdn.GDN_CONV_WIDTH - 1, l.width, dtype=BF16, device=dev)
            else:  # start from the prefix's state
                self.state[i] = prefix.state[i].expand(n, -1, -1, -1).contiguous()
                self.conv[i] = prefix.conv[i].expand(n, -1, -1).contiguous()

    @property
    def shared(self):
        return 0 if self.prefix is None else self.prefix.length


class Model:
    def __init__(self, hidden=512, layers=4, pages=256, page=16, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.hidden, self.page, self.device = hidden, page, device
        self.layers = [Layer("attention" if i % 4 == 3 else "delta", hidden, g, device)
                       for i in range(layers)]
        self.caches = [Cache(l, pages, page, device) if l.kind == "attention" else None
                       for l in self.layers]
        self.final = torch.ones(hidden, device=device)
        self.free = torch.randperm(pages, generator=g).to(torch.int32).to(device)
        self.workspaces = {}

    def take_pages(self, count):
        taken, self.free = self.free[:count], self.free[count:]
        assert taken.numel() == count, "out of pages"
        return taken.clone()

    def workspace(self, kind, batch, tokens, layer):
        """Kept from call to call; zeroed once, as the calls ask for."""
        n = batch.lens.numel()
        # what decides the size; a batch behind a prefix needs more than a plain one
        key = (kind, n, tokens) + ((layer.hq, layer.hkv, layer.d, batch.shared > 0) if kind == "attention"
                                   else (layer.hk, layer.hv))
        if key not in self.workspaces:
            if kind == "attention":
                self.workspaces[key] = gdn.gdn_attn_workspace(n, tokens, layer.hq, layer.hkv, layer.d,
                                                              prefix_len=batch.shared)
            else:
                shape = gdn.make_shape(n, n, layer.hk, layer.hv)
                size = gdn.gdn_workspace_size(shape, gdn.GDN_OP_DECODE_BLOCK) + 256
                self.workspaces[key] = torch.zeros(size, dtype=torch.uint8, device=self.device)
        return self.workspaces[key]

    def delta(self, i, l, x, batch, cu):
        d = 128
        q, k, v, z = (x @ l.w_in.T).split([l.hk * d, l.hk * d, l.hv * d, l.hv * d], 1)
        q, k, v, z = (t.contiguous().view(x.shape[0], -1, d) for t in (q, k, v, z))
        a, b = (t.float().contiguous() for t in (x @ l.w_gates.T).split(l.hv, 1))
        conv, state = batch.conv[i], batch.state[i]
        if cu is None:
            y, _ = gdn.gdn_decode_block_step(q, k, v, a, b, l.conv, l.A_log, l.dt_bias, conv, conv, state,
                                             state, z, l.out_norm,
                                             workspace=self.workspace("delta", batch, x.shape[0], l))
        else:
            q, k, v, gl, beta = gdn.gdn_input_prologue(q, k, v, a, b, l.conv, l.A_log, l.dt_bias, conv,
                                                       conv, cu)
            o = torch.empty(v.shape, dtype=torch.float32, device=v.device)
            gdn.gdn_prefill_chunked(q, k, v, gl, beta, state, state, cu, o)
            y = gdn.gdn_gated_rmsnorm(o, z, l.out_norm)
        return y.flatten(1) @ l.w_out.T

    def attention(self, i, l, codes, scale, batch, cu):
        # the projection of the norm's 8-bit output: the scales of its rows come after the product
        row = ((codes.to(BF16) @ l.w_in.T).float() * scale).to(BF16)
        q, gate, k, v = (t.unflatten(1, (-1, l.d)) for t in
                         row.split([l.hq * l.d, l.hq * l.d, l.hkv * l.d, l.hkv * l.d], 1))
        c, ws = self.caches[i], self.workspace("attention", batch, row.shape[0], l)
        q = gdn.gdn_kv_append(q, k, v, c.k, c.v, batch.tables, batch.lens, l.inv_freq, cu_seqlens=cu,
                              q_norm=l.q_norm, k_norm=l.k_norm, prefix_len=batch.shared)
        if batch.prefix is None:
            o = gdn.gdn_paged_attention(q, c.k, c.v, batch.tables, batch.lens, cu, gate=gate, workspace=ws)
        else:
            o = gdn.gdn_shared_prefix_attention(q, c.k, c.v, batch.prefix.tables[0], batch.shared,
                                                batch.tables, batch.lens, cu, gate=gate, workspace=ws)
        return o.flatten(1) @ l.w_out.T

    def forward(self, x, batch, counts=None):
        """Hidden states x [tokens, hidden] of the batch's next tokens: `counts` of each sequence,
        or one each.  Returns the normed hidden states."""
        cu = None
        if counts is not None:
            cu = torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).to(self.device)
        batch.lens += 1 if counts is None else torch.tensor(counts, dtype=torch.int32, device=self.device)
        residual = None
        for i, l in enumerate(self.layers):
            if l.kind == "delta":
                y, residual = gdn.gdn_add_rmsnorm(x, residual, l.norm)
                x = self.delta(i, l, y, batch, cu)
            else:
                y8, scale, residual = gdn.gdn_add_rmsnorm(x, residual, l.norm, out="e4m3")
                x = self.attention(i, l, y8, scale, batch, cu)
        return gdn.gdn_add_rmsnorm(x, residual, self.final)[0]


def main(requests=5, system=100, prompts=(7, 40, 1, 23, 64), steps=6, seed=1):
    g = torch.Generator().manual_seed(seed)
    model = Model()
    most = max(prompts) + steps

    def tokens(n):
        return torch.randn(n, model.hidden, generator=g).to(BF16).to(model.device)

    head = tokens(system)
    own = [tokens(n) for n in prompts]
    then = [tokens(requests) for _ in range(steps)]

    prefix = Batch(model, 1, system)
    model.forward(head, prefix, [system])
    prefix.length = system
    served = Batch(model, requests, most, prefix)
    out = [list(model.forward(torch.cat(own), served, list(prompts)).split(list(prompts)))]
    for x in then:
        out.append(list(model.forward(x, served).split(1)))
    got = [torch.cat([o[i] for o in out]) for i in range(requests)]

    # the same sequences in one piece
    whole = Batch(model, requests, system + most)
    counts = [system + n + steps for n in prompts]
    x = torch.cat([t for i in range(requests) for t in [head, own[i]] + [s[i:i + 1] for s in then]])
    want = model.forward(x, whole, counts).split(counts)
    worst = 0.0
    for i in range(requests):
        a, b = got[i].float(), want[i][system:].float()
        worst = max(worst, ((a - b).norm() / b.norm()).item())
    return worst


if __name__ == "__main__":
    error = main()
    torch.cuda.synchronize()
    print("served behind a shared prefix against read in one piece: relative difference %.2e" % error)
