"""Operators for several continuations of one context: inputs, plain forms and calls, for measuring.

A hybrid decoder (gated delta-rule layers and softmax attention layers) goes on from a context in more
than one way at a time when a tree of drafted tokens is checked in one pass, and when it keeps several
beams.  Four operators do that beside the matrix products:

  attend   attention of a tree's nodes over a paged cache: each node sees the context, its
           ancestors and itself
  verify   the gated delta rule over such a tree from an untouched state: each node's state comes
           from its parent's; the outputs and each node's delta
  select   the best continuations of a group's beams over beams and vocabulary (also how a tree of
           drafts is grown, a level at a time)
  reorder  the rows of a state, of a convolution's last inputs or of a page table follow the beams
           that were selected, in place

``own`` False computes the plain forms below from elementary torch operations in 32 bits (the
scores of beams in 64: they are compared with each other); True calls the library.
"""
import math
import random

import torch

own = False

PAGES = (16, 32, 64, 128)


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # two chats, small trees: latency
        dict(name="tree_attend_few", op="attend", n=2, t_lo=5, t_hi=13, past_lo=300, past_hi=1500,
             hq=16, hkv=4, d=128, page=16, gate=False, prefix=0),
        # a serving batch, a tree each, ragged contexts
        dict(name="tree_attend_batch", op="attend", n=64, t_lo=11, t_hi=40, past_lo=255, past_hi=8191,
             hq=32, hkv=8, d=128, page=64, gate=False, prefix=0),
        # two very long documents with the widest trees, 256-wide gated heads
        dict(name="tree_attend_long", op="attend", n=2, t_lo=49, t_hi=64, past_lo=90000,
             past_hi=131000, hq=16, hkv=2, d=256, page=64, gate=True, prefix=0),
        # requests behind one system prompt
        dict(name="tree_attend_prefix", op="attend", n=24, t_lo=7, t_hi=32, past_lo=0, past_hi=700,
             hq=16, hkv=4, d=128, page=32, gate=True, prefix=4099),
        # two chats' delta-rule layers, small trees: latency
        dict(name="tree_verify_few", op="verify", n=2, t_lo=5, t_hi=13, chunk=16, hk=16, hv=16,
             dtype="bf16"),
        # the serving batch, two value heads to a key head
        dict(name="tree_verify_batch", op="verify", n=64, t_lo=11, t_hi=32, chunk=32, hk=16, hv=32,
             dtype="bf16"),
        # wide trees, everything in 32 bits
        dict(name="tree_verify_f32", op="verify", n=24, t_lo=40, t_hi=64, chunk=64, hk=16, hv=32,
             dtype="f32"),
        # one level of two requests' trees of drafts
        dict(name="select_step", op="select", groups=2, beams=4, top=4, vocab=32000, dtype="bf16",
             done=False, masked=False),
        # beam search in a serving batch: an odd vocabulary, some beams finished, some tokens forbidden
        dict(name="select_batch", op="select", groups=64, beams=8, top=8, vocab=150001, dtype="f32",
             done=True, masked=True),
        # many beams for few requests
        dict(name="select_wide", op="select", groups=4, beams=48, top=48, vocab=99999, dtype="bf16",
             done=False, masked=False),
        # the last inputs of one layer's convolution
        dict(name="reorder_fifo", op="reorder", layers=1, groups=4, beams=4, kind="fifo", heads=64),
        # the states of three layers
        dict(name="reorder_states", op="reorder", layers=3, groups=16, beams=8, kind="state",
             heads=32),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["attend", "attend", "verify", "verify", "select", "select", "reorder"])
    if op == "attend":
        hkv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 5, 8, 16])
        while hkv * group > 32:
            group = rng.choice([1, 2, 3, 4, 5, 8, 16])
        d = rng.choice([128, 256])
        n = _log_int(rng, 1, 100)
        most = max(64, min(131000, (1 << 27) // (n * hkv * d)))  # keys that the batch's cache holds
        hi = _log_int(rng, 32, most)
        t = _log_int(rng, 1, 64)
        prefix = _log_int(rng, 100, 8000) if rng.random() < 0.25 else 0
        return dict(op=op, n=n, t_lo=max(1, t // 3), t_hi=t, past_lo=hi // 4, past_hi=hi,
                    hq=hkv * group, hkv=hkv, d=d, page=rng.choice(PAGES), gate=rng.random() < 0.5,
                    prefix=prefix)
    if op == "verify":
        hk = rng.choice([1, 2, 4, 8, 16])
        hv = hk * rng.choice([1, 2, 4])
        chunk = rng.choice([16, 32, 64])
        t = rng.randint(1, chunk)
        return dict(op=op, n=_log_int(rng, 1, max(2, 2000 // hv)), t_lo=max(1, t // 3), t_hi=t,
                    chunk=chunk, hk=hk, hv=hv, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "select":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 16, 32, 64])
        vocab = _log_int(rng, 500, 262144)
        groups = _log_int(rng, 1, max(1, min(256, (1 << 26) // (beams * vocab))))
        return dict(op=op, groups=groups, beams=beams, top=rng.choice([1, 2, 4, 7, 8, 16, 33, 64]),
                    vocab=vocab, dtype=rng.choice(["bf16", "f32"]), done=rng.random() < 0.5,
                    masked=rng.random() < 0.5)
    beams = rng.choice([2, 3, 4, 5, 8, 16, 32, 64])
    kind = rng.choice(["fifo", "state"])
    heads = rng.choice([2, 4, 8, 16, 32])
    layers = rng.randint(1, 6)
    row = _row_bytes(dict(kind=kind, heads=heads))
    groups = _log_int(rng, 1, max(1, min(64, (700 << 20) // (layers * beams * row))))
    return dict(op=op, layers=layers, groups=groups, beams=beams, kind=kind, heads=heads)


# ------------------------------------------------------------------ lengths, trees, inputs

def _rng(case, what):
    """The case's own, whatever the inputs' seed, so that its work does not change with them."""
    return random.Random(what + repr(sorted((k, str(v)) for k, v in case.items() if k != "name")))


def _lengths(case):
    """Nodes of each tree, and keys before it (the shared prefix apart)."""
    rng = _rng(case, "lengths")
    t = [rng.randint(case["t_lo"], case["t_hi"]) for _ in range(case["n"])]
    past = [rng.randint(case.get("past_lo", 0), case.get("past_hi", 0)) for _ in range(case["n"])]
    return t, past


def _tree(case):
    """Parents of all nodes, by their index in the own tree; -1 hangs on the context.  As a search
    grows them: a node continues one of the last few."""
    rng = _rng(case, "tree")
    out = []
    for t in _lengths(case)[0]:
        wide = rng.choice([1, 3, 8, 20])  # 1: a chain, as prompt lookup drafts it
        out += [max(-1, i - 1 - int(rng.random() ** 2 * wide)) if i else -1 for i in range(t)]
    return out


def _beam_parents(case):
    """Where the beams continue from: the better beams, which stand first, more often."""
    rng = _rng(case, "parents")
    w = case["beams"]
    return [sorted(int(w * rng.random() ** 1.5) for _ in range(w)) for _ in range(case["groups"])]


def _row_bytes(case):
    return case["heads"] * 128 * 128 * 4 if case["kind"] == "state" else 3 * case["heads"] * 128 * 2


def _int32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _pages_of(x, page):
    return (x + page - 1) // page


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed * 7919 + 23)
    gg = torch.Generator(device="cuda").manual_seed(seed * 7919 + 24)

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        x = torch.randn(*shape, generator=gg, device="cuda")
        return (x.mul_(std) if std != 1.0 else x).to(dtype)

    s = {"case": dict(case)}
    if case["op"] == "reorder":
        rows = case["groups"] * case["beams"]
        if case["kind"] == "state":
            s["rows"] = normal(case["layers"], rows, case["heads"], 128, 128, dtype=torch.float32, std=0.1)
        else:
            s["rows"] = normal(case["layers"], rows, 3, case["heads"] * 128)
        s["parents"] = _int32(_beam_parents(case))
        return s
    if case["op"] == "select":
        groups, beams, vocab = case["groups"], case["beams"], case["vocab"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # a few likely tokens before a long tail
        x = normal(groups * beams, vocab, dtype=torch.float32, std=2.5)
        likely = torch.randint(0, vocab, (groups * beams, 20), generator=gg, device="cuda")
        x.scatter_add_(1, likely, 6 * torch.rand(likely.shape, generator=gg, device="cuda"))
        if case["masked"]:  # a grammar forbids part of the vocabulary
            x[:, torch.rand(vocab, generator=gg, device="cuda") < 0.4] = -math.inf
        s["logits"] = x.to(dt).view(groups, beams, vocab)
        s["scores"] = -10 * torch.rand(groups, beams, generator=gg, device="cuda")
        s["finished"] = None
        if case["done"]:
            s["finished"] = torch.rand(groups, beams, generator=gg, device="cuda") < 0.2
        s["pad"] = int(torch.randint(0, vocab, (1,), generator=g))
        return s
    t, past = _lengths(case)
    tokens = sum(t)
    s["t"], s["past"] = t, past
    s["cu_seqlens"] = _int32([sum(t[:i]) for i in range(len(t) + 1)])
    s["parents"] = _int32(_tree(case))
    if case["op"] == "verify":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        hk, hv, n = case["hk"], case["hv"], case["n"]
        for name in ("q", "k"):
            x = normal(tokens, hk, 128, dtype=torch.float32)
            s[name] = (x / torch.sqrt((x * x).sum(-1, keepdim=True))).to(dt)
        s["v"] = normal(tokens, hv, 128, dtype=dt)
        s["g"] = -torch.log1p(torch.exp(normal(tokens, hv, dtype=torch.float32)))
        s["beta"] = torch.sigmoid(normal(tokens, hv, dtype=torch.float32))
        s["state"] = normal(n, hv, 128, 128, dtype=torch.float32, std=0.1)
        return s
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    shared = case["prefix"]
    lens = [a + b for a, b in zip(t, past)]
    need = [_pages_of(x, page) for x in lens]
    first = _pages_of(shared, page)
    total = first + sum(need) + 3  # a few pages belong to nobody
    s["lens"] = lens
    s["kv_lens"] = _int32(lens)
    s["k_cache"] = normal(total, hkv, page, d)
    s["v_cache"] = normal(total, hkv, page, d)
    order = (torch.randperm(total - first, generator=g) + first).to(torch.int32)
    table = torch.zeros(len(lens), max(need), dtype=torch.int32)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    s["page_table"] = table.cuda()
    s["prefix_table"] = torch.randperm(first, generator=g).to(torch.int32).cuda() if shared else None
    s["q"] = normal(tokens, hq, d, std=1.5)  # scores of a standard deviation of 1.5
    s["gate"] = normal(tokens, hq, d) if case["gate"] else None
    return s


# ------------------------------------------------------------------ plain forms

def _padded(s):
    """Rows of each sequence's nodes [n, t] (past the last: some other node), and which are real."""
    cu = s["cu_seqlens"].long()
    row = cu[:-1, None] + torch.arange(max(s["t"]), device="cuda")
    live = row < cu[1:, None]
    return row.clamp(max=int(s["parents"].shape[0]) - 1), live


def _ancestors(s, row, live):
    """[n, t, t]: node i (rows) has node j above it, or is it."""
    n, t = row.shape
    parents = torch.where(live, s["parents"][row], -1).long()
    up = torch.zeros(n, t, t, dtype=torch.bool, device="cuda")
    which = torch.arange(n, device="cuda")
    for i in range(t):
        p = parents[:, i]
        up[:, i] = up[which, p.clamp(min=0)] & (p >= 0)[:, None]
        up[:, i, i] = True
    return up


def _gather(cache, pages, keys):
    """Keys of page lists [..., pages] as [..., hkv, keys, d] in 32 bits."""
    x = cache[pages.long()].float().movedim(-3, -4)
    return x.reshape(*x.shape[:-3], -1, x.shape[-1])[..., :keys, :]


def _plain_attend_some(s, a, b, row, live, up):
    """Sequences a to b - 1, padded to the longest of them."""
    c = s["case"]
    hq, hkv, d, shared = c["hq"], c["hkv"], c["d"], c["prefix"]
    m, most, t = b - a, max(s["lens"][a:b]), max(s["t"][a:b])
    row, live, up = row[a:b, :t], live[a:b, :t], up[a:b, :t, :t]
    x = s["q"][row].float() / math.sqrt(d)
    x = x.view(m, t, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(m, hkv, -1, d)
    k, v = (_gather(s[name], s["page_table"][a:b, :_pages_of(most, c["page"])], most)
            for name in ("k_cache", "v_cache"))
    node = torch.arange(most, device="cuda") - (s["kv_lens"][a:b] - s["cu_seqlens"].diff()[a:b])[:, None]
    seen = torch.gather(up, 2, node.clamp(0, t - 1).long()[:, None].expand(m, t, most))
    seen = (node < 0)[:, None] | (seen & (node < t)[:, None])
    sc = (x @ k.transpose(-1, -2)).view(m, hkv, hq // hkv, t, most)
    sc = sc.masked_fill(~seen[:, None, None], -math.inf).view(m, hkv, -1, most)
    if shared:
        pk, pv = (_gather(s[name], s["prefix_table"], shared) for name in ("k_cache", "v_cache"))
        sc = torch.cat([x @ pk.transpose(-1, -2), sc], -1)
        v = torch.cat([pv.expand(m, -1, -1, -1), v], -2)
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = (p @ v).view(m, hkv, hq // hkv, t, d).permute(0, 3, 1, 2, 4).reshape(m, t, hq, d)
    return o[live]


def _plain_attend(s):
    """In batches of sequences whose scores fit about 8 GB."""
    c, t = s["case"], s["t"]
    row, live = _padded(s)
    up = _ancestors(s, row, live)
    lens = [x + c["prefix"] for x in s["lens"]]
    outs, a = [], 0
    while a < len(t):
        b = a + 1
        while b < len(t) and (b + 1 - a) * max(lens[a:b + 1]) * \
                max(max(t[a:b + 1]) * c["hq"], 4 * c["hkv"] * c["d"]) < 2 << 30:
            b += 1
        outs.append(_plain_attend_some(s, a, b, row, live, up))
        a = b
    o = torch.cat(outs)
    if s["gate"] is not None:
        o = o * torch.sigmoid(s["gate"].float())
    return o.to(s["q"].dtype)


def _plain_verify(s):
    """The chunkwise form with ancestors in place of earlier tokens: with G the sum of g over a
    node's path, D_i = beta_i (v_i - e^G_i S^T k_i - sum_{j above i} e^(G_i - G_j) (k_i.k_j) D_j)
    node by node, then O = e^G Q S + (decays . Q K^T) D."""
    c = s["case"]
    rep = c["hv"] // c["hk"]
    row, live = _padded(s)
    up = _ancestors(s, row, live)[:, None]  # [n, 1, t, t]
    t = row.shape[1]
    heads = lambda x: x[row].float().transpose(1, 2)  # [n, heads, t, ...]
    q, k = (heads(s[name]).repeat_interleave(rep, 1) for name in ("q", "k"))
    v, g, beta = heads(s["v"]), heads(s["g"]), heads(s["beta"])
    path = torch.where(up, g[:, :, None], 0.0).sum(-1)
    decay = torch.exp(torch.where(up, path[..., None] - path[:, :, None], -math.inf))
    from_state = torch.exp(path)[..., None]
    kk = decay * (k @ k.transpose(-1, -2))
    kk.diagonal(dim1=-2, dim2=-1).zero_()
    right = v - from_state * (k @ s["state"])
    d = torch.zeros_like(right)
    for i in range(t):
        below = (kk[:, :, i, :i, None] * d[:, :, :i]).sum(2)
        d[:, :, i] = beta[:, :, i, None] * (right[:, :, i] - below)
    o = from_state * (q @ s["state"]) + (decay * (q @ k.transpose(-1, -2))) @ d
    return o.transpose(1, 2)[live].to(s["v"].dtype), d.transpose(1, 2)[live].contiguous()


def _plain_select(s):
    c = s["case"]
    groups, beams, vocab, top = c["groups"], c["beams"], c["vocab"], c["top"]
    scores, tokens, parents = [], [], []
    for a in range(0, groups, max(1, (1 << 25) // (beams * vocab))):  # (the sort's memory)
        b = min(groups, a + max(1, (1 << 25) // (beams * vocab)))
        x = s["logits"][a:b].double()
        e = x - x.amax(-1, keepdim=True)
        x = s["scores"][a:b, :, None].double() + (e - torch.log(torch.exp(e).sum(-1, keepdim=True)))
        if s["finished"] is not None:  # a finished beam goes on as it is, with the padding token
            stays = torch.full((vocab,), -math.inf, dtype=torch.float64, device="cuda")
            stays[s["pad"]] = 0.0
            x = torch.where(s["finished"][a:b, :, None], s["scores"][a:b, :, None].double() + stays, x)
        x = torch.where(torch.isnan(x), -math.inf, x).view(b - a, -1)
        best, at = torch.sort(x, dim=-1, descending=True, stable=True)
        scores.append(best[:, :top].float())
        parents.append((at[:, :top] // vocab).to(torch.int32))
        tokens.append((at[:, :top] % vocab).to(torch.int32))
    return torch.cat(scores), torch.cat(parents), torch.cat(tokens)


def _plain_reorder(s):
    c, x = s["case"], s["rows"]
    first = torch.arange(c["groups"], device="cuda")[:, None] * c["beams"]
    x.copy_(x[:, (first + s["parents"]).flatten().long()])
    return x


# ------------------------------------------------------------------ the calls

def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"attend": _plain_attend, "verify": _plain_verify, "select": _plain_select,
                "reorder": _plain_reorder}[op](s)
    import gated_deltanet_linear_05_gb300 as gdn
    if op == "reorder":
        return gdn.gdn_beam_reorder(s["rows"], s["parents"])
    if op == "select":
        if "workspace" not in s:  # what a program keeps from step to step
            s["workspace"] = gdn.gdn_beam_workspace(c["groups"], c["beams"], c["vocab"], c["top"])
        return gdn.gdn_beam_select(s["logits"], s["scores"], c["top"], finished=s["finished"],
                                   pad_token=s["pad"], workspace=s["workspace"])
    if op == "verify":
        return gdn.gdn_verify_tree(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"],
                                   s["cu_seqlens"], s["parents"], chunk=c["chunk"])
    if "workspace" not in s:
        s["workspace"] = gdn.gdn_attn_workspace(c["n"], s["q"].shape[0], c["hq"], c["hkv"], c["d"],
                                                prefix_len=c["prefix"])
    return gdn.gdn_tree_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_lens"],
                                  s["cu_seqlens"], s["parents"], gate=s["gate"],
                                  prefix_table=s["prefix_table"], prefix_len=c["prefix"],
                                  workspace=s["workspace"])


# ------------------------------------------------------------------ what a pass cannot do without

def _depths(case):
    """Ancestors of each node, itself included."""
    out, parents = [], _tree(case)
    at = 0
    for t in _lengths(case)[0]:
        for i in range(t):
            p = parents[at + i]
            out.append(1 + (out[at + p] if p >= 0 else 0))
        at += t
    return out


def work(case):
    if case["op"] == "reorder":
        # rows that change are written; those they come from are read
        moved = [[(i, p) for i, p in enumerate(row) if i != p] for row in _beam_parents(case)]
        rows = sum(len(m) + len({p for _, p in m}) for m in moved)
        return {"bytes": rows * case["layers"] * _row_bytes(case) + 4 * case["groups"] * case["beams"],
                "flops": 0}
    if case["op"] == "select":
        n = case["groups"] * case["beams"]
        el = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * (case["vocab"] * el + 5) + 12 * case["groups"] * case["top"],
                "flops": 3 * n * case["vocab"]}
    t, past = _lengths(case)
    tokens, pairs = sum(t), sum(_depths(case))
    if case["op"] == "verify":
        el = 2 if case["dtype"] == "bf16" else 4
        hk, hv = case["hk"], case["hv"]
        return {"bytes": case["n"] * hv * 65536 + tokens * (2 * hk * 128 * el + hv * (2 * 128 * el + 512 + 8))
                + 4 * tokens,
                "flops": tokens * hv * 4 * 128 * 128 + pairs * (hk * 4 * 128 + hv * 4 * 128)}
    hq, hkv, d, shared = case["hq"], case["hkv"], case["d"], case["prefix"]
    q_bytes = tokens * hq * d * 2 * (3 if case["gate"] else 2)
    kv_bytes = (tokens + sum(past) + shared) * hkv * d * 4
    seen = tokens * shared + sum(a * b for a, b in zip(t, past)) + pairs
    return {"bytes": q_bytes + kv_bytes + 4 * tokens, "flops": 4 * seen * hq * d}


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"attend": _exact_attend, "verify": _exact_verify, "select": _exact_select,
                "reorder": _exact_reorder}[case["op"]](case, s)


def _paths(case):
    """For each sequence, for each node: its ancestors from the context down, itself last."""
    parents, at, out = _tree(case), 0, []
    for t in _lengths(case)[0]:
        paths = []
        for i in range(t):
            p = parents[at + i]
            paths.append((paths[p] if p >= 0 else []) + [i])
        out.append(paths)
        at += t
    return out


def _exact_attend(case, s):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    group, shared = hq // hkv, case["prefix"]
    if 4.0 * d * hq * sum(t * (l + shared) for t, l in zip(s["t"], s["lens"])) > 5e12:
        return None  # over about 20 seconds in 64 bits
    out = torch.empty(sum(s["t"]), hq, d, dtype=torch.float64, device="cuda")
    at = 0
    for i, (t, l, paths) in enumerate(zip(s["t"], s["lens"], _paths(case))):
        pages = s["page_table"][i, :_pages_of(l, case["page"])].long()
        k, v = (s[name][pages].transpose(0, 1).reshape(hkv, -1, d)[:, :l] for name in ("k_cache", "v_cache"))
        if shared:
            head = s["prefix_table"].long()
            k, v = (torch.cat([s[name][head].transpose(0, 1).reshape(hkv, -1, d)[:, :shared], x], 1)
                    for name, x in (("k_cache", k), ("v_cache", v)))
        before = shared + l - t
        hide = torch.ones(t, before + t, dtype=torch.bool)
        hide[:, :before] = False
        for j, path in enumerate(paths):
            hide[j, [before + x for x in path]] = False
        hide = hide.cuda()
        for h in range(hkv):
            qq = s["q"][at:at + t, h * group:(h + 1) * group].double()
            sc = torch.einsum("tgd,kd->gtk", qq, k[h].double()) * d ** -0.5
            sc.masked_fill_(hide, -math.inf)
            out[at:at + t, h * group:(h + 1) * group] = torch.einsum(
                "gtk,kd->tgd", torch.softmax(sc, -1), v[h].double())
        at += t
    if s["gate"] is not None:
        out = out / (1 + torch.exp(-s["gate"].double()))
    return out


def _exact_verify(case, s):
    """Node by node: the parent's state, decayed, corrected and read."""
    rep = case["hv"] // case["hk"]
    o = torch.empty(s["v"].shape, dtype=torch.float64, device="cuda")
    delta = torch.empty_like(o)
    parents, at = _tree(case), 0
    for n, t in enumerate(s["t"]):
        states = []
        for i in range(t):
            x, p = at + i, parents[at + i]
            k, q = (s[name][x].double().repeat_interleave(rep, 0) for name in ("k", "q"))
            S = (states[p] if p >= 0 else s["state"][n].double()) * torch.exp(s["g"][x].double())[:, None, None]
            kv = torch.einsum("hi,hij->hj", k, S)
            delta[x] = (s["v"][x].double() - kv) * s["beta"][x].double()[:, None]
            S = S + k[:, :, None] * delta[x][:, None, :]
            o[x] = torch.einsum("hi,hij->hj", q, S)
            states.append(S)
        at += t
    return o, delta


def _exact_select(case, s):
    groups, beams, vocab, top = (case[name] for name in ("groups", "beams", "vocab", "top"))
    score = torch.empty(groups, top, dtype=torch.float64, device="cuda")
    parent = torch.empty(groups, top, dtype=torch.int32, device="cuda")
    token = torch.empty_like(parent)
    index = torch.arange(beams * vocab, device="cuda")
    for i in range(groups):
        x = torch.log_softmax(s["logits"][i].double(), -1) + s["scores"][i].double()[:, None]
        if s["finished"] is not None:
            for w in torch.nonzero(s["finished"][i]).flatten().tolist():
                x[w] = -math.inf
                x[w, s["pad"]] = s["scores"][i, w].double()
        x = x.flatten()
        # everything as good as the last of the best, then those in order of score and index
        least = torch.topk(x, top).values[-1]
        some = index[x >= least]
        some = some[torch.sort(x[some], descending=True, stable=True).indices][:top]
        score[i], parent[i], token[i] = x[some], some // vocab, some % vocab
    return score, parent, token


def _exact_reorder(case, s):
    x = s["rows"].double()
    out = torch.empty_like(x)
    for g, row in enumerate(_beam_parents(case)):
        for i, p in enumerate(row):
            out[:, g * case["beams"] + i] = x[:, g * case["beams"] + p]
    return out
