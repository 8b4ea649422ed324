"""The attention layer's operators: inputs, plain forms and calls, for measuring.

The hybrid decoders this library serves alternate gated delta-rule layers with gated softmax
attention layers.  Four operators make up the attention layer beside the matrix products:

  append   per-head RMS norm of q and k, rotary positions (one or several axes), and the
           scatter of k and v into a paged cache
  attend   attention over the paged cache: one token per sequence, drafts, or prompts
  prefix   the same for a batch whose sequences share one long prefix
  norm     residual addition + RMS norm, output in the input's type or in e4m3 with scales

``own`` False computes the plain forms below from elementary torch operations in 32 bits
(positions times frequencies in 64); True calls the library.
"""
import math
import random

import numpy as np
import torch

own = False

PAGES = (16, 32, 64, 128)


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step of a batch of 32: 256-wide heads, a quarter of each rotated, q/k norms
        dict(name="append_step", op="append", n=32, t_lo=1, t_hi=1, past_lo=100, past_hi=900,
             hq=16, hkv=4, d=256, page=64, rot=64, axes=1, norm=True, fused=True),
        # packed image-and-text prompts: three position axes, rows of a fused projection
        dict(name="append_prompts", op="append", n=8, t_lo=256, t_hi=8192, past_lo=0, past_hi=0,
             hq=32, hkv=8, d=128, page=32, rot=128, axes=3, norm=False, fused=True),
        # a few chats, one token each: latency
        dict(name="attend_step_few", op="attend", n=3, t_lo=1, t_hi=1, past_lo=300, past_hi=1500,
             hq=16, hkv=4, d=128, page=16, gate=False, step=True),
        # a serving batch, one token each, ragged contexts
        dict(name="attend_step_batch", op="attend", n=64, t_lo=1, t_hi=1, past_lo=255, past_hi=8191,
             hq=32, hkv=8, d=128, page=64, gate=False, step=True),
        # two very long documents, one token each: the split over the cache, 256-wide gated heads
        dict(name="attend_step_long", op="attend", n=2, t_lo=1, t_hi=1, past_lo=90000,
             past_hi=131070, hq=16, hkv=2, d=256, page=64, gate=True, step=True),
        # a prompt-lookup check: 16 draft tokens for each of 128 sequences
        dict(name="attend_drafts", op="attend", n=128, t_lo=16, t_hi=16, past_lo=200, past_hi=4000,
             hq=32, hkv=4, d=128, page=64, gate=False, step=False),
        # one prompt of 4096 tokens, 16 gated heads of 256
        dict(name="attend_prompt", op="attend", n=1, t_lo=4096, t_hi=4096, past_lo=0, past_hi=0,
             hq=16, hkv=4, d=256, page=64, gate=True, step=False),
        # eight packed prompts of 256 to 8192 tokens, 32 heads of 128
        dict(name="attend_prompts", op="attend", n=8, t_lo=256, t_hi=8192, past_lo=0, past_hi=0,
             hq=32, hkv=8, d=128, page=128, gate=False, step=False),
        # a few requests behind one short system prompt
        dict(name="prefix_few", op="prefix", n=5, prefix=777, own_lo=1, own_hi=90,
             hq=16, hkv=4, d=128, page=16, gate=False),
        # 128 requests behind one long document
        dict(name="prefix_batch", op="prefix", n=128, prefix=16389, own_lo=1, own_hi=1000,
             hq=32, hkv=8, d=128, page=64, gate=False),
        # the norm before a decode step's projections
        dict(name="norm_step", op="norm", rows=32, cols=4096, dtype="bf16", out="e4m3", group=0),
        # the norm before a prompt's projections, 128-wide scale groups, odd number of rows
        dict(name="norm_prompt", op="norm", rows=16383, cols=4096, dtype="bf16", out="e4m3",
             group=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["append", "attend", "attend", "attend", "prefix", "norm"])
    if op == "norm":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        cols = 128 * _log_int(rng, 8, 64)
        rows = _log_int(rng, 1, 8000)
        out = rng.choice(["same", "e4m3", "e4m3"])
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, out=out,
                    group=rng.choice([0, 128]) if out == "e4m3" else 0)
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8, 16])
    while hkv * group > 32:
        group = rng.choice([1, 2, 3, 4, 5, 8, 16])
    d = rng.choice([128, 256])
    c = dict(op=op, hq=hkv * group, hkv=hkv, d=d, page=rng.choice(PAGES))
    if op == "append":
        step = rng.random() < 0.5
        n = _log_int(rng, 1, 200) if step else rng.randint(1, 6)
        t_hi = 1 if step else _log_int(rng, 16, 3500)
        past = _log_int(rng, 1, 500) if rng.random() < 0.5 else 0
        c.update(n=n, t_lo=1 if step else max(1, t_hi // 3), t_hi=t_hi, past_lo=past // 2,
                 past_hi=past, rot=rng.choice([d // 4, d // 2, d]), axes=rng.choice([1, 3]),
                 norm=rng.random() < 0.5, fused=rng.random() < 0.5)
        return c
    c["gate"] = rng.random() < 0.5
    width = c["hkv"] * d
    if op == "prefix":
        n = _log_int(rng, 2, 128)
        hi = _log_int(rng, 2, 800)
        c.update(n=n, prefix=_log_int(rng, 200, 16000), own_lo=max(1, hi // 8), own_hi=hi)
        return c
    kind = rng.choice(["step", "drafts", "prompts"])
    if kind == "step":
        n = _log_int(rng, 1, 128)
        most = max(64, min(131000, (1 << 28) // (n * width)))  # keys that the batch's cache holds
        hi = _log_int(rng, 32, most)
        c.update(n=n, t_lo=1, t_hi=1, past_lo=hi // 4, past_hi=hi, step=True)
    elif kind == "drafts":
        n = _log_int(rng, 1, 128)
        most = max(64, min(16000, (1 << 27) // (n * width)))
        hi = _log_int(rng, 32, most)
        t = rng.randint(2, 24)
        c.update(n=n, t_lo=max(1, t // 2), t_hi=t, past_lo=hi // 4, past_hi=hi, step=False)
    else:
        n = rng.randint(1, 3)
        t = _log_int(rng, 64, 2500)
        past = _log_int(rng, 1, 3000) if rng.random() < 0.5 else 0
        c.update(n=n, t_lo=max(1, t // 3), t_hi=t, past_lo=past // 2, past_hi=past, step=False)
    return c


# ------------------------------------------------------------------ lengths, tables, inputs

def _lengths(case):
    """Query lengths and context lengths: the case's own, whatever the inputs' seed, so that its
    work does not change with them."""
    key = sorted((k, str(v)) for k, v in case.items() if k != "name")
    rng = random.Random(repr(key))
    n = case["n"]
    if case["op"] == "prefix":
        t = [1] * n
        own_len = [rng.randint(case["own_lo"], case["own_hi"]) for _ in range(n)]
        return t, own_len
    t = [rng.randint(case["t_lo"], case["t_hi"]) for _ in range(n)]
    past = [rng.randint(case["past_lo"], case["past_hi"]) for _ in range(n)]
    return t, [a + b for a, b in zip(t, past)]


def _pages_of(lens, page):
    return [(x + page - 1) // page for x in lens]


def _table(lens, page, g, first, total):
    """Page table [n, most] over a random order of the pages `first`..total - 1."""
    need = _pages_of(lens, page)
    order = torch.randperm(total - first, generator=g) + first
    tab = torch.zeros(len(lens), max(1, max(need)), dtype=torch.int32)
    at = 0
    for i, m in enumerate(need):
        tab[i, :m] = order[at:at + m].to(torch.int32)
        at += m
    return tab.cuda()


def _int32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _cu(t):
    return _int32([0] + list(np.cumsum(t)))


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed * 7919 + 17)
    gg = torch.Generator(device="cuda").manual_seed(seed * 7919 + 18)

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return (torch.randn(*shape, generator=gg, device="cuda") * std).to(dtype)

    s = {"case": dict(case)}
    if case["op"] == "norm":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        rows, cols = case["rows"], case["cols"]
        # a residual stream: unequal channels, a few far larger than the rest
        gain = torch.exp(normal(cols, dtype=torch.float32, std=0.5))
        gain[torch.randperm(cols, generator=g)[:4].cuda()] *= 30
        s["x"] = normal(rows, cols, dtype=torch.float32, std=0.3).to(dt)
        s["residual"] = (normal(rows, cols, dtype=torch.float32) * gain).to(dt)
        s["weight"] = 1 + 0.1 * normal(cols, dtype=torch.float32)
        return s
    hq, hkv, d, page, n = case["hq"], case["hkv"], case["d"], case["page"], case["n"]
    t, lens = _lengths(case)
    tokens = sum(t)
    shared = case.get("prefix", 0)
    first = (shared + page - 1) // page
    total = first + sum(_pages_of(lens, page)) + 3  # a few pages belong to nobody
    s["lens"], s["t"] = lens, t
    s["kv_lens"] = _int32(lens)
    s["cu_seqlens"] = _cu(t)
    s["k_cache"] = normal(total, hkv, page, d)
    s["v_cache"] = normal(total, hkv, page, d)
    s["page_table"] = _table(lens, page, g, first, total)
    if case["op"] == "append":
        if case["fused"]:  # rows of one fused projection
            row = normal(tokens, (hq + 2 * hkv) * d)
            s["q"] = row[:, :hq * d].view(tokens, hq, d)
            s["k"] = row[:, hq * d:(hq + hkv) * d].view(tokens, hkv, d)
            s["v"] = row[:, (hq + hkv) * d:].view(tokens, hkv, d)
        else:
            s["q"], s["k"], s["v"] = (normal(tokens, h, d) for h in (hq, hkv, hkv))
        rot = case["rot"]
        s["inv_freq"] = torch.tensor([1e7 ** (-2.0 * i / rot) for i in range(rot // 2)],
                                     dtype=torch.float64).cuda()
        s["rope_axis"], s["positions"] = None, None
        if case["axes"] > 1:  # sections of time, height and width; later tokens far along
            m = rot // 2
            s["rope_axis"] = _int32([0 if i < m // 4 else 1 if i < m // 4 + 3 * m // 8 else 2
                                     for i in range(m)])
            s["positions"] = torch.randint(0, 250000, (case["axes"], tokens), generator=g,
                                           dtype=torch.int32).cuda()
        s["q_norm"] = s["k_norm"] = None
        if case["norm"]:
            s["q_norm"] = 1 + 0.1 * normal(d, dtype=torch.float32)
            s["k_norm"] = 1 + 0.1 * normal(d, dtype=torch.float32)
        return s
    s["q"] = normal(tokens, hq, d, std=1.5)  # scores of a standard deviation of 1.5
    s["gate"] = normal(tokens, hq, d) if case["gate"] else None
    if shared:
        s["prefix_table"] = torch.randperm(first, generator=g).to(torch.int32).cuda()
    return s


# ------------------------------------------------------------------ plain forms

EPS = 1e-6


def _head_norm(x, w):
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _rotate(x, angle):
    """x [tokens, heads, d] in 32 bits; angle [tokens, rot / 2] in 64."""
    m = angle.shape[1]
    c, sn = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    a, b, rest = x[..., :m], x[..., m:2 * m], x[..., 2 * m:]
    return torch.cat([a * c - b * sn, b * c + a * sn, rest], -1)


def _token_places(s):
    """Sequence of each token and its place in that sequence's cache."""
    cu, lens = s["cu_seqlens"].long(), s["kv_lens"].long()
    tok = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(cu[1:], tok, right=True)
    return seq, lens[seq] - (cu[seq + 1] - tok)


def _plain_append(s):
    page = s["case"]["page"]
    seq, place = _token_places(s)
    if s["positions"] is None:
        angle = place.double()[:, None] * s["inv_freq"]
    else:
        angle = s["positions"].double()[s["rope_axis"].long()].T * s["inv_freq"]
    q = _rotate(_head_norm(s["q"].float(), s["q_norm"]), angle).to(s["q"].dtype)
    k = _rotate(_head_norm(s["k"].float(), s["k_norm"]), angle).to(s["k"].dtype)
    where = s["page_table"][seq, place // page].long()
    s["k_cache"][where, :, place % page] = k
    s["v_cache"][where, :, place % page] = s["v"]
    return q, s["k_cache"], s["v_cache"]


def _gather(cache, pages, keys):
    """Keys of one page list [..., pages] as [..., hkv, keys, d] in 32 bits."""
    x = cache[pages.long()].float()  # [..., pages, hkv, page, d]
    x = x.movedim(-3, -4)
    return x.reshape(*x.shape[:-3], -1, x.shape[-1])[..., :keys, :]


def _gated(o, gate, dtype):
    if gate is not None:
        o = o * torch.sigmoid(gate.float())
    return o.to(dtype)


def _plain_step(s):
    """One token per sequence, all sequences padded to the longest; a shared prefix, if there
    is one, takes part through one product for the whole batch."""
    c, q = s["case"], s["q"]
    n, hq, d = q.shape
    hkv = c["hkv"]
    most = max(s["lens"])
    x = q.float().view(n, hkv, hq // hkv, d) / math.sqrt(d)
    k, v = (_gather(s[name], s["page_table"], most) for name in ("k_cache", "v_cache"))
    sc = x @ k.transpose(-1, -2)
    valid = torch.arange(most, device="cuda") < s["kv_lens"][:, None]
    sc = sc.masked_fill(~valid[:, None, None], -math.inf)
    shared = c.get("prefix", 0)
    if shared:
        pk, pv = (_gather(s[name], s["prefix_table"], shared) for name in ("k_cache", "v_cache"))
        rows = x.transpose(0, 1).reshape(hkv, -1, d)
        ps = (rows @ pk.transpose(-1, -2)).view(hkv, n, hq // hkv, shared).transpose(0, 1)
        sc = torch.cat([ps, sc], -1)
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = p[..., shared:] @ v
    if shared:
        rows = p[..., :shared].transpose(0, 1).reshape(hkv, -1, shared)
        o = o + (rows @ pv).view(hkv, n, hq // hkv, d).transpose(0, 1)
    return _gated(o.reshape(n, hq, d), s["gate"], q.dtype)


def _plain_equal(s, a, b, most):
    """Sequences a to b - 1, padded to the longest query and context among them."""
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    cu, lens = s["cu_seqlens"].long(), s["kv_lens"].long()
    t = max(s["t"][a:b])
    at = torch.arange(t, device="cuda")
    row = cu[a:b, None] + at  # [m, t], past the end of the shorter ones
    live = row < cu[a + 1:b + 1, None]
    x = s["q"][row.clamp(max=s["q"].shape[0] - 1)].float() / math.sqrt(d)
    x = x.view(b - a, t, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b - a, hkv, -1, d)
    k, v = (_gather(s[name], s["page_table"][a:b, :-(-most // c["page"])], most)
            for name in ("k_cache", "v_cache"))
    sc = (x @ k.transpose(-1, -2)).view(b - a, hkv, hq // hkv, t, most)
    last = lens[a:b, None] - (cu[a + 1:b + 1, None] - row)  # the key a query sees last
    seen = torch.arange(most, device="cuda") <= last[..., None]
    sc = sc.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).view(b - a, hkv, -1, most)
    o = (p @ v).view(b - a, hkv, hq // hkv, t, d).permute(0, 3, 1, 2, 4).reshape(b - a, t, hq, d)
    return o[live]


def _plain_attend(s):
    """Batches of sequences whose scores fit about 8 GB: drafts in a few of them, prompts one
    by one."""
    c, lens, t = s["case"], s["lens"], s["t"]
    outs, a = [], 0
    while a < len(t):
        b = a + 1
        while b < len(t) and ((b + 1 - a) * max(t[a:b + 1]) * max(lens[a:b + 1])) * c["hq"] < 2 << 30:
            b += 1
        outs.append(_plain_equal(s, a, b, max(lens[a:b])))
        a = b
    return _gated(torch.cat(outs), s["gate"], s["q"].dtype)


def _plain_norm(s):
    c = s["case"]
    h = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    f = h.float()
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * s["weight"]
    if c["out"] == "same":
        return y.to(h.dtype), h
    grouped = y.view(c["rows"], -1, c["group"] or c["cols"])
    scale = grouped.abs().amax(-1, keepdim=True).clamp(min=1e-12) / 448
    y8 = (grouped / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(c["rows"], c["cols"])
    return y8, scale[..., 0], h


# ------------------------------------------------------------------ the calls

def _workspace(s, gdn):
    """What a program keeps from step to step: the attention calls' scratch."""
    if "workspace" not in s:
        c = s["case"]
        s["workspace"] = gdn.gdn_attn_workspace(c["n"], s["q"].shape[0], c["hq"], c["hkv"], c["d"],
                                                prefix_len=c.get("prefix", 0))
    return s["workspace"]


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op == "append":
            return _plain_append(s)
        if op == "norm":
            return _plain_norm(s)
        return _plain_step(s) if op == "prefix" or c["step"] else _plain_attend(s)
    import gated_deltanet_linear_05_gb300 as gdn
    if op == "append":
        q = gdn.gdn_kv_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"],
                              s["kv_lens"], s["inv_freq"],
                              cu_seqlens=None if c["t_hi"] == 1 else s["cu_seqlens"],
                              positions=s["positions"], rope_axis=s["rope_axis"],
                              q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
        return q, s["k_cache"], s["v_cache"]
    if op == "norm":
        return gdn.gdn_add_rmsnorm(s["x"], s["residual"], s["weight"], EPS, out=c["out"],
                                   group=c["group"])
    ws = _workspace(s, gdn)
    if op == "prefix":
        return gdn.gdn_shared_prefix_attention(s["q"], s["k_cache"], s["v_cache"],
                                               s["prefix_table"], c["prefix"], s["page_table"],
                                               s["kv_lens"], gate=s["gate"], workspace=ws)
    return gdn.gdn_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_lens"],
                                   cu_seqlens=None if c["step"] else s["cu_seqlens"],
                                   gate=s["gate"], workspace=ws)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["cols"]
        el = 2 if case["dtype"] == "bf16" else 4
        out = n if case["out"] == "e4m3" else n * el
        scales = 4 * case["rows"] * (case["cols"] // case["group"] if case["group"] else 1)
        return {"bytes": 3 * n * el + out + (scales if case["out"] == "e4m3" else 0)
                + 4 * case["cols"], "flops": 8 * n}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    t, lens = _lengths(case)
    tokens = sum(t)
    if case["op"] == "append":
        row = (hq + 2 * hkv) * d * 2
        return {"bytes": tokens * (2 * row + 4 * case["axes"]) + 8 * len(t),
                "flops": tokens * (hq + hkv) * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    shared = case.get("prefix", 0)
    q_bytes = tokens * hq * d * 2 * (3 if case["gate"] else 2)
    kv_bytes = (sum(lens) + shared) * hkv * d * 4
    pairs = tokens * shared + sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(t, lens))
    return {"bytes": q_bytes + kv_bytes, "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "norm":
            return _exact_norm(case, s)
        if case["op"] == "append":
            return _exact_append(case, s)
        return _exact_attention(case, s)


def _exact_norm(case, s):
    h = (s["x"].double() + s["residual"].double())
    stored = h.to(s["x"].dtype)
    f = stored.double()
    rms = torch.sqrt(f.pow(2).sum(1, keepdim=True) / case["cols"] + EPS)
    y = f / rms * s["weight"].double()
    if case["out"] == "same":
        return y, h
    width = case["group"] or case["cols"]
    scale = y.abs().unflatten(1, (-1, width)).amax(2).clamp(min=1e-12) / 448
    return y / scale.repeat_interleave(width, 1), scale, h


def _exact_append(case, s):
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    page, m = case["page"], case["rot"] // 2
    cu, lens = np.cumsum([0] + s["t"]), s["lens"]
    table = s["page_table"].cpu().numpy()
    place = np.concatenate([np.arange(l - t, l) for t, l in zip(s["t"], lens)])
    seq = np.repeat(np.arange(len(lens)), s["t"])
    assert cu[-1] == len(place)
    freq = s["inv_freq"].cpu().numpy()
    if s["positions"] is None:
        ang = place[:, None].astype(np.float64) * freq[None]
    else:
        pos, axis = s["positions"].cpu().numpy(), s["rope_axis"].cpu().numpy()
        ang = np.stack([pos[axis[i]] * freq[i] for i in range(m)], 1)
    turn = torch.polar(torch.ones(ang.shape, dtype=torch.float64), torch.from_numpy(ang)).cuda()[:, None]

    def head(x, w):
        x = x.double().clone()
        if w is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / case["d"] + EPS) * w.double()
        z = torch.complex(x[..., :m].contiguous(), x[..., m:2 * m].contiguous()) * turn
        x[..., :m], x[..., m:2 * m] = z.real, z.imag
        return x

    q, k = head(s["q"], s["q_norm"]), head(s["k"], s["k_norm"])
    at = torch.from_numpy(table[seq, place // page].astype(np.int64)).cuda()
    off = torch.from_numpy(place % page).cuda()
    k_cache[at, :, off] = k
    v_cache[at, :, off] = s["v"].double()
    return q, k_cache, v_cache


def _exact_attention(case, s):
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    group = hq // hkv
    shared = case.get("prefix", 0)
    out = torch.empty(sum(s["t"]), hq, d, dtype=torch.float64, device="cuda")
    if 4.0 * d * hq * sum(t * (l + shared) for t, l in zip(s["t"], s["lens"])) > 5e12:
        return None  # over about 20 seconds in 64 bits
    at = 0
    for i, (t, l) in enumerate(zip(s["t"], s["lens"])):
        places = [s["page_table"][i, j // page].item() * page + j % page for j in range(0, l, page)]
        pages = [p // page for p in places]
        k = s["k_cache"][pages].transpose(0, 1).reshape(hkv, -1, d)[:, :l]
        v = s["v_cache"][pages].transpose(0, 1).reshape(hkv, -1, d)[:, :l]
        if shared:
            head = s["prefix_table"].long()
            k = torch.cat([s["k_cache"][head].transpose(0, 1).reshape(hkv, -1, d)[:, :shared], k], 1)
            v = torch.cat([s["v_cache"][head].transpose(0, 1).reshape(hkv, -1, d)[:, :shared], v], 1)
        keys = k.shape[1]
        limit = torch.arange(keys - t, keys, device="cuda")[:, None]
        hide = torch.arange(keys, device="cuda")[None] > limit
        for h in range(hkv):
            kk, vv = k[h].double(), v[h].double()
            qq = s["q"][at:at + t, h * group:(h + 1) * group].double()
            sc = torch.einsum("tgd,kd->gtk", qq, kk) * d ** -0.5
            sc.masked_fill_(hide, -math.inf)
            out[at:at + t, h * group:(h + 1) * group] = torch.einsum(
                "gtk,kd->tgd", torch.softmax(sc, -1), vv)
        at += t
    if s["gate"] is not None:
        out = out / (1 + torch.exp(-s["gate"].double()))
    return out
