"""Several continuations at a time in the hybrid decoder of hybrid_decoder.py: trees of drafts, grown level
by level and checked in one pass, and beam search.  Random weights, random "tokens".

    python examples/branching_decoder.py

Drafts: a small head guesses on from each request's last hidden state; the best continuations over beams and
vocabulary make the next level of its tree.  One pass checks all nodes: each sees its own path alone, in
the delta-rule layers through its parent's state, in the attention layers through its ancestors' keys.  A
path is accepted, the states and the cache follow it, and the requests go on from there.

Beams: every beam is a row of the batch; after each step the rows' states, convolution inputs and keys follow
the beams that were selected.

Both are compared with the same tokens read in order.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from hybrid_decoder import BF16, Batch, Model, gdn  # noqa: E402


def _ints(values, device):
    return torch.tensor(values, dtype=torch.int32).to(device)


class Tree:
    """Trees of one check: token ids and parents of every request's nodes, packed."""

    def __init__(self, ids, parents, device):
        self.counts = [len(p) for p in parents]
        first = [sum(self.counts[:i]) for i in range(len(parents))]
        self.ids = torch.cat(ids)
        self.parents = _ints([p for up in parents for p in up], device)
        self.cu = _ints(first + [len(self.parents)], device)
        self.path = []  # of each node: its ancestors' rows from the context down, its own last
        for at, up in zip(first, parents):
            for i, p in enumerate(up):
                self.path.append((self.path[at + p] if p >= 0 else []) + [at + i])
        self.depth = _ints([len(p) - 1 for p in self.path], device)
        self.sequence = torch.repeat_interleave(torch.arange(len(parents)), torch.tensor(self.counts)).to(device)
        # rows of the last three inputs before each node: those of ancestors, else -1, -2, -3 places before the tree
        self.before = torch.tensor([[p[len(p) - 1 - back] if len(p) > back else len(p) - 1 - back
                                     for back in (3, 2, 1)] for p in self.path]).to(device)


class Branching(Model):
    def __init__(self, vocab=1000, **kw):
        super().__init__(**kw)
        g = torch.Generator().manual_seed(99)
        self.embed = torch.randn(vocab, self.hidden, generator=g).to(BF16).to(self.device)
        self.draft = (torch.randn(self.hidden, self.hidden, generator=g) / self.hidden ** 0.5).to(BF16).to(self.device)

    def logits(self, hidden):
        return hidden @ self.embed.T / self.hidden ** 0.5

    # ---------------------------------------------------------------- trees of drafts

    def grow(self, hidden, levels, width):
        """A tree for each row of hidden: `levels` levels of `width` nodes, by the draft head."""
        n, dev = hidden.shape[0], self.device
        state = hidden[:, None]
        scores = torch.zeros(n, 1, device=dev)
        ids, up = [], []
        for level in range(levels):
            logits = self.logits(state.reshape(-1, self.hidden)).view(n, -1, self.embed.shape[0])
            scores, beam, token = gdn.gdn_beam_select(logits.contiguous(), scores, width)
            state = torch.gather(state, 1, beam.long()[..., None].expand(-1, -1, self.hidden))
            state = torch.tanh(state @ self.draft + self.embed[token.long()])
            ids.append(token.long())
            up.append(beam + (level - 1) * width if level else torch.full_like(beam, -1))
        return Tree(list(torch.cat(ids, 1)), torch.cat(up, 1).tolist(), dev)

    def check(self, tree, batch):
        """Hidden states of the tree's nodes after the batch's tokens, and what `accept` needs.  The batch stays
        as it is but for the cache's rows behind its keys."""
        lens = batch.lens + _ints(tree.counts, self.device)
        places = batch.shared + batch.lens[tree.sequence] + tree.depth
        x, residual, kept = self.embed[tree.ids], None, []
        for i, l in enumerate(self.layers):
            if l.kind == "delta":
                y, residual = gdn.gdn_add_rmsnorm(x, residual, l.norm)
                x, keep = self._check_delta(i, l, y, tree, batch)
            else:
                y8, scale, residual = gdn.gdn_add_rmsnorm(x, residual, l.norm, out="e4m3")
                x, keep = self._check_attention(i, l, y8, scale, tree, batch, lens, places)
            kept.append(keep)
        return gdn.gdn_add_rmsnorm(x, residual, self.final)[0], kept

    def _check_delta(self, i, l, x, tree, batch):
        raw, z = (x @ l.w_in.T).split([l.width, l.hv * 128], 1)
        raw = raw.contiguous()
        a, b = (t.float().contiguous() for t in (x @ l.w_gates.T).split(l.hv, 1))
        # each node as a sequence of one token, behind the three inputs on its own path
        fifo = batch.conv[i][tree.sequence[:, None], (3 + tree.before).clamp(0, 2)]
        window = torch.where((tree.before >= 0)[..., None], raw[tree.before.clamp(min=0)], fifo).contiguous()
        split = [t.contiguous().view(x.shape[0], -1, 128) for t in raw.split([l.hk * 128, l.hk * 128, l.hv * 128], 1)]
        q, k, v, g, beta = gdn.gdn_input_prologue(*split, a, b, l.conv, l.A_log, l.dt_bias, window, None)
        o = torch.empty(v.shape, dtype=torch.float32, device=v.device)
        _, delta = gdn.gdn_verify_tree(q, k, v, g, beta, batch.state[i], tree.cu, tree.parents, o=o)
        y = gdn.gdn_gated_rmsnorm(o, z.contiguous().view(v.shape), l.out_norm)
        return y.flatten(1) @ l.w_out.T, (split, k, g, delta)

    def _check_attention(self, i, l, codes, scale, tree, batch, lens, places):
        row = ((codes.to(BF16) @ l.w_in.T).float() * scale).to(BF16)
        q, gate, k, v = (t.unflatten(1, (-1, l.d)) for t in
                         row.split([l.hq * l.d, l.hq * l.d, l.hkv * l.d, l.hkv * l.d], 1))
        c, ws = self.caches[i], self.workspace("attention", batch, row.shape[0], l)
        r = gdn.gdn_kv_append(q, k, v, c.k, c.v, batch.tables, lens, l.inv_freq, cu_seqlens=tree.cu, positions=places,
                              q_norm=l.q_norm, k_norm=l.k_norm)
        prefix = {} if batch.prefix is None else dict(prefix_table=batch.prefix.tables[0], prefix_len=batch.shared)
        o = gdn.gdn_tree_attention(r, c.k, c.v, batch.tables, lens, tree.cu, tree.parents, gate=gate, workspace=ws, **prefix)
        return o.flatten(1) @ l.w_out.T, (q, k, v)

    def accept(self, tree, batch, leaves, kept):
        """The batch's states and cache follow the path to node leaves[n] of each tree (-1: none of it)."""
        first = [0] + torch.tensor(tree.counts).cumsum(0).tolist()
        taken = [tree.path[first[n] + leaf] if leaf >= 0 else [] for n, leaf in enumerate(leaves)]
        rows = torch.tensor([r for path in taken for r in path], dtype=torch.long, device=self.device)
        lens = _ints([len(path) for path in taken], self.device)
        cu = torch.cat([lens.new_zeros(1), lens.cumsum(0).to(torch.int32)])
        batch.lens += lens
        for i, l in enumerate(self.layers):
            if l.kind == "delta":
                split, k, g, delta = kept[i]
                gdn.gdn_state_rollback(k[rows], g[rows], delta[rows], batch.state[i], lens, batch.state[i], cu)
                gdn.gdn_conv_state_rollback(*(t[rows] for t in split), batch.conv[i], lens, batch.conv[i], cu)
            else:  # the path's keys move together, at the places that they have been rotated to
                q, k, v = (t[rows] for t in kept[i])
                gdn.gdn_kv_append(q, k, v, self.caches[i].k, self.caches[i].v, batch.tables, batch.lens, l.inv_freq,
                                  cu_seqlens=cu, q_norm=l.q_norm, k_norm=l.k_norm, prefix_len=batch.shared)

    # ---------------------------------------------------------------- beams

    def beam_search(self, batch, hidden, beams, steps):
        """From `batch`, whose rows are the requests' beams, all alike, and their last hidden states
        [requests * beams, hidden].  Returns (scores, token ids [requests, beams, steps], the hidden states
        after them)."""
        n, dev = hidden.shape[0] // beams, self.device
        scores = torch.full((n, beams), -float("inf"), device=dev)
        scores[:, 0] = 0  # the beams are still one
        ids = torch.zeros(1, n * beams, 0, dtype=torch.int32, device=dev)
        ws = gdn.gdn_beam_workspace(n, beams, self.embed.shape[0], beams)
        for _ in range(steps):
            logits = self.logits(hidden).view(n, beams, -1)
            scores, parents, tokens = gdn.gdn_beam_select(logits, scores, beams, workspace=ws)
            for i, l in enumerate(self.layers):
                if l.kind == "delta":
                    gdn.gdn_beam_reorder(batch.state[i][None], parents)
                    gdn.gdn_beam_reorder(batch.conv[i][None], parents)
                else:  # each row writes to its own pages, so their contents follow
                    rows = (torch.arange(n, device=dev)[:, None] * beams + parents).flatten()
                    for cache in (self.caches[i].k, self.caches[i].v):
                        cache[batch.tables.long()] = cache[batch.tables[rows].long()]
            if ids.shape[2]:
                gdn.gdn_beam_reorder(ids, parents)
            ids = torch.cat([ids, tokens.view(1, -1, 1)], 2)
            hidden = self.forward(self.embed[tokens.flatten().long()], batch)
        return scores, ids.view(n, beams, steps), hidden.view(n, beams, -1)


def _difference(a, b):
    return ((a.float() - b.float()).norm() / b.float().norm()).item()


def drafts(model, requests=3, system=60, prompts=(9, 40, 1), levels=4, width=5, seed=1):
    """Largest relative difference of the nodes' hidden states, and of those after a path was accepted, from the
    same tokens read in order."""
    g = torch.Generator().manual_seed(seed)
    vocab = model.embed.shape[0]
    head, own = torch.randint(vocab, (system,), generator=g).cuda(), [torch.randint(vocab, (n,), generator=g).cuda() for n in prompts]
    most = max(prompts) + levels * width + 4
    prefix = Batch(model, 1, system)
    model.forward(model.embed[head], prefix, [system])
    prefix.length = system
    served = Batch(model, requests, most, prefix)
    hidden = model.forward(model.embed[torch.cat(own)], served, list(prompts))
    last = hidden[torch.tensor(prompts).cumsum(0) - 1]
    tree = model.grow(last, levels, width)
    nodes, kept = model.check(tree, served)
    rng = torch.Generator().manual_seed(seed)
    leaves = [int(torch.randint(-1, c, (1,), generator=rng)) for c in tree.counts]
    model.accept(tree, served, leaves, kept)
    more = torch.randint(vocab, (requests, 2), generator=g).cuda()
    after = torch.cat([model.forward(model.embed[more[:, i]], served) for i in range(2)])
    # a few whole paths, and the accepted ones with what came after them
    worst = 0.0
    for n in range(requests):
        at = sum(tree.counts[:n])
        for leaf in (tree.counts[n] - 1, tree.counts[n] // 2, leaves[n]):
            path = tree.path[at + leaf] if leaf >= 0 else []
            tail = more[n] if leaf == leaves[n] else more[n, :0]
            x = model.embed[torch.cat([head, own[n], tree.ids[path], tail])]
            whole = Batch(model, 1, len(x))
            want = model.forward(x, whole, [len(x)])[system + prompts[n]:]
            got = nodes[path]
            if leaf == leaves[n]:
                got = torch.cat([got, after[n::requests]])
            if len(got):
                worst = max(worst, _difference(got, want))
            model.free = torch.cat([whole.tables.flatten(), model.free])
    return worst


def beams(model, requests=2, prompts=(12, 33), width=4, steps=5, seed=2):
    """Largest relative difference of the beams' last hidden states, and largest difference of their scores, from
    those of the same tokens read in order."""
    g = torch.Generator().manual_seed(seed)
    vocab = model.embed.shape[0]
    own = [torch.randint(vocab, (n,), generator=g).cuda() for n in prompts]
    batch = Batch(model, requests * width, max(prompts) + steps)
    rows = [x for x in own for _ in range(width)]
    hidden = model.forward(model.embed[torch.cat(rows)], batch, [len(x) for x in rows])
    hidden = hidden[torch.tensor([len(x) for x in rows]).cumsum(0) - 1]
    scores, ids, last = model.beam_search(batch, hidden, width, steps)
    worst, off = 0.0, 0.0
    for n in range(requests):
        assert len({tuple(r) for r in ids[n].tolist()}) == width  # all different
        for w in range(width):
            x = torch.cat([own[n], ids[n, w].long()])
            whole = Batch(model, 1, len(x))
            h = model.forward(model.embed[x], whole, [len(x)])
            worst = max(worst, _difference(last[n, w], h[-1]))
            logs = torch.log_softmax(model.logits(h[len(own[n]) - 1:-1]).double(), -1)
            off = max(off, abs(scores[n, w].item() - logs.gather(1, ids[n, w].long()[:, None]).sum().item()))
            model.free = torch.cat([whole.tables.flatten(), model.free])
    return worst, off


if __name__ == "__main__":
    model = Branching()
    print("nodes of drafted trees and tokens after an accepted path, against the same read in order: relative "
          "difference %.2e" % drafts(model))
    print("beams against the same tokens read in order: relative difference of hidden states %.2e, difference of scores "
          "%.2e" % beams(model))
    torch.cuda.synchronize()
