"""Trees of drafts and the 64-bit definitions of the operators on them, for the tests."""
import numpy as np
import torch

from attn_testlib import BF16_HALF, gather


def tree(kind, t, rng):
    """Parents of a tree of t nodes; "wild" holds values that mean -1 as well."""
    if kind == "chain":
        return [i - 1 for i in range(t)]
    if kind == "star":
        return [-1] * t
    if kind == "wild":
        return [int(rng.choice([rng.integers(-1, i) if i else -1, i, i + 3, -5, 1 << 30, -(1 << 31)])) for i in range(t)]
    wide = {"narrow": 2, "bushy": 9}[kind]
    return [max(-1, i - 1 - int(rng.integers(0, wide))) for i in range(t)]


def paths(parents):
    """Each node's ancestors, from the context down, itself last."""
    out = []
    for i, p in enumerate(parents):
        out.append((out[p] if 0 <= p < i else []) + [i])
    return out


def trees(t, seed, kinds=("bushy", "chain", "star", "narrow", "wild")):
    rng = np.random.default_rng(seed)
    return [tree(kinds[(i + seed) % len(kinds)], n, rng) for i, n in enumerate(t)]


def packed(lists, device="cuda"):
    return torch.tensor([p for x in lists for p in x], dtype=torch.int32).to(device)


def attention(b, parents, scale=None):
    """(o, bound, lse) of attn_testlib's batch with its sequences' nodes under `parents`; the bound
    as attn_testlib.reference counts it."""
    scale = b.d ** -0.5 if scale is None else scale
    group = b.hq // b.hkv
    q = b.q.cpu().double()
    o = torch.zeros(q.shape, dtype=torch.float64)
    mean = torch.zeros_like(o)
    lse = torch.full(q.shape[:2], -float("inf"), dtype=torch.float64)
    pk, pv = (gather(c, b.prefix_pages, b.prefix) for c in (b.k_cache, b.v_cache))
    at = 0
    for t, l, pages, up in zip(b.t, b.lens, b.pages, parents):
        k = torch.cat([pk, gather(b.k_cache, pages, l)], 1)
        v = torch.cat([pv, gather(b.v_cache, pages, l)], 1)
        first = b.prefix + l - t  # of the tree's keys
        hide = torch.ones(t, b.prefix + l, dtype=torch.bool)
        hide[:, :max(first, 0)] = False
        for i, path in enumerate(paths(up)):
            hide[i, [first + j for j in path if first + j >= b.prefix]] = False
        for h in range(b.hq):
            s = q[at:at + t, h] @ k[h // group].T * scale
            s = s.masked_fill(hide, -float("inf"))
            if s.shape[1] == 0:
                continue
            e = torch.logsumexp(s, 1, keepdim=True)
            p = torch.where(torch.isinf(e), torch.zeros_like(s), torch.exp(s - e))
            o[at:at + t, h], mean[at:at + t, h] = p @ v[h // group], p @ v[h // group].abs()
            lse[at:at + t, h] = e[:, 0]
        at += t
    if b.gate is not None:
        gate = torch.sigmoid(b.gate.cpu().double())
        o, mean = o * gate, mean * gate
    return o, (BF16_HALF + 2.0 ** -15) * mean + BF16_HALF * (1 + 2.0 ** -7) * o.abs(), lse


class DeltaBatch:
    """Inputs of gdn_verify_tree.  `extra` tokens behind the last sequence."""

    def __init__(self, t, hk, hv, dtype, seed=0, extra=0, decay=1.0, state=True, kinds=None, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.t, self.hk, self.hv = list(t), hk, hv
        tokens, n = sum(t) + extra, len(t)
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32

        def normal(*shape):
            return torch.randn(*shape, generator=g)

        self.q, self.k = ((lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dt).to(device))(normal(tokens, hk, 128))
                          for _ in range(2))
        self.v = normal(tokens, hv, 128).to(dt).to(device)
        self.g = (-decay * torch.log1p(torch.exp(normal(tokens, hv)))).to(device)
        self.beta = torch.sigmoid(normal(tokens, hv)).to(device)
        self.state = (0.1 * normal(n, hv, 128, 128)).to(device) if state else None
        self.parents = trees(t, seed) if kinds is None else trees(t, seed, kinds)
        self.up = packed(self.parents + [[0] * extra], device)
        self.cu = torch.tensor([0] + list(np.cumsum(t)), dtype=torch.int32).to(device)

    def args(self):
        return self.q, self.k, self.v, self.g, self.beta, self.state, self.cu, self.up


def delta_rule(b):
    """(o, delta, each node's state) token by token in 64 bits, every node from its parent's state."""
    rep = b.hv // b.hk
    q, k, v, g, beta = (x.cpu().double() for x in (b.q, b.k, b.v, b.g, b.beta))
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    o, delta, states, at = torch.zeros_like(v), torch.zeros_like(v), [], 0
    for n, (t, up) in enumerate(zip(b.t, b.parents)):
        own = []
        root = torch.zeros(b.hv, 128, 128, dtype=torch.float64) if b.state is None else b.state[n].cpu().double()
        for i, p in enumerate(up):
            x = at + i
            s = (own[p] if 0 <= p < i else root) * torch.exp(g[x])[:, None, None]
            delta[x] = (v[x] - torch.einsum("hi,hij->hj", k[x], s)) * beta[x][:, None]
            s = s + k[x][:, :, None] * delta[x][:, None, :]
            o[x] = torch.einsum("hi,hij->hj", q[x], s)
            own.append(s)
        states.append(own)
        at += t
    return o, delta, states
