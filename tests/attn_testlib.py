"""Inputs and the 64-bit definition of the attention-layer operators, for the tests."""
import numpy as np
import torch

BF16_HALF = 2.0 ** -8  # half a step of bf16, relative


class Batch:
    """A paged cache and the queries of one call.  `lens`: own keys of each sequence, `t`: its
    query tokens.  Every cache row that no sequence owns holds NaN, and table entries past a
    sequence's last page are out of range."""

    def __init__(self, t, lens, hq, hkv, d, page, prefix=0, gate=False, seed=0, std=1.5,
                 q_pad=0, page_pad=0, spare=2, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.t, self.lens, self.hq, self.hkv, self.d = list(t), list(lens), hq, hkv, d
        self.page, self.prefix = page, prefix
        n, tokens = len(t), sum(t)
        own = [-(-x // page) for x in lens]
        first = -(-prefix // page)
        pages = first + sum(own) + spare
        order = torch.randperm(pages, generator=g).tolist()
        self.prefix_pages = order[:first]
        at, self.pages = first, []
        for m in own:
            self.pages.append(order[at:at + m])
            at += m
        most = max([1] + own)
        table = torch.full((n, most), -7, dtype=torch.int32)
        for i, p in enumerate(self.pages):
            table[i, :len(p)] = torch.tensor(p, dtype=torch.int32)
            if len(p) < most:
                table[i, len(p)] = 1 << 30
        self.page_table = table.to(device)
        self.prefix_table = torch.tensor(self.prefix_pages or [0], dtype=torch.int32).to(device)
        self.kv_lens = torch.tensor(lens, dtype=torch.int32).to(device)
        self.cu = torch.tensor([0] + list(np.cumsum(t)), dtype=torch.int32).to(device)
        row = hkv * page * d + page_pad

        def cache():
            flat = torch.full((pages, row), float("nan"), dtype=torch.bfloat16)
            c = flat[:, :hkv * page * d].view(pages, hkv, page, d) if not page_pad else \
                flat.as_strided((pages, hkv, page, d), (row, page * d, d, 1))
            for used, m in [(self.prefix_pages, prefix)] + list(zip(self.pages, lens)):
                for j, pg in enumerate(used):
                    live = min(page, m - j * page)
                    c[pg, :, :live] = torch.randn(hkv, live, d, generator=g).to(torch.bfloat16)
            dev = flat.to(device)
            return dev.as_strided((pages, hkv, page, d), (row, page * d, d, 1))

        self.k_cache, self.v_cache = cache(), cache()
        self.q = self._rows(tokens, hq, g, std, q_pad, device)
        self.gate = self._rows(tokens, hq, g, 2.0, q_pad, device) if gate else None

    def _rows(self, tokens, heads, g, std, pad, device):
        flat = torch.full((tokens, heads * (self.d + pad) + pad), float("nan"), dtype=torch.bfloat16)
        view = flat.as_strided((tokens, heads, self.d), (flat.shape[1], self.d + pad, 1))
        view.copy_((torch.randn(tokens, heads, self.d, generator=g) * std).to(torch.bfloat16))
        return flat.to(device).as_strided(view.shape, view.stride())


def gather(cache, pages, count):
    """Keys of a page list as [hkv, count, d] float64 on the CPU."""
    c = cache.cpu().double()
    if not pages or count <= 0:
        return c.new_zeros(c.shape[1], 0, c.shape[3])
    return torch.cat([c[p] for p in pages], 1)[:, :count]


def reference(b, scale=None):
    """(o, bound on |o_kernel - o|, lse) by the definition in 64 bits.

    The bound counts the kernel's roundings: the probabilities to bf16 (half a step of
    each, so 2^-8 of the softmax-weighted mean of |v|), the output to bf16, and 2^-15 of that
    mean for everything in float32 (a score's error of at most D 2^-24 sum|q k| scale and the
    exponential's argument)."""
    scale = b.d ** -0.5 if scale is None else scale
    group = b.hq // b.hkv
    q = b.q.cpu().double()
    gate = None if b.gate is None else torch.sigmoid(b.gate.cpu().double())
    o = torch.zeros(q.shape, dtype=torch.float64)
    mean = torch.zeros_like(o)
    lse = torch.full(q.shape[:2], -float("inf"), dtype=torch.float64)
    pk, pv = (gather(c, b.prefix_pages, b.prefix) for c in (b.k_cache, b.v_cache))
    at = 0
    for t, l, pages in zip(b.t, b.lens, b.pages):
        k = torch.cat([pk, gather(b.k_cache, pages, l)], 1)
        v = torch.cat([pv, gather(b.v_cache, pages, l)], 1)
        for h in range(b.hq):
            kk, vv = k[h // group], v[h // group]
            s = q[at:at + t, h] @ kk.T * scale
            place = torch.arange(l - t, l)[:, None]
            s = s.masked_fill(torch.arange(-b.prefix, l)[None] > torch.clamp(place, min=-1), -float("inf"))
            if s.shape[1] == 0:
                continue
            e = torch.logsumexp(s, 1, keepdim=True)
            p = torch.where(torch.isinf(e), torch.zeros_like(s), torch.exp(s - e))
            o[at:at + t, h], mean[at:at + t, h] = p @ vv, p @ vv.abs()
            lse[at:at + t, h] = e[:, 0]
        at += t
    if gate is not None:
        o, mean = o * gate, mean * gate
    return o, (BF16_HALF + 2.0 ** -15) * mean + BF16_HALF * (1 + 2.0 ** -7) * o.abs(), lse
