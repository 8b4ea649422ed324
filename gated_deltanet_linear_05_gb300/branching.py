"""Binding of the operators for several continuations of a context: the delta rule over trees of
drafts, the selection of the best continuations over beams and vocabulary, and the reordering of the
rows that follow the beams.

Argument marshalling only, as in the package itself; include/gdn.h has the contract of each call.  A
call that is given a stream runs with that stream current, so that what it allocates belongs to it.
A call whose combination of sizes, strides and types has been seen goes through _marshal
(csrc/marshal.c), as the attention layer's do.
"""
from __future__ import annotations

import ctypes

import torch

from . import (GDN_BF16, GDN_ERR_INVALID_ARG, GDN_F32, GDN_OK, GdnError, _check_tensors, lib,
               make_shape)
from . import attention as _attention
from .attention import _current_device, _raw_stream, _remember

_CODES = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}
_I32, _F32 = torch.int32, torch.float32
_made = {}  # by sizes, strides and types: what follows from them


def _quick():
    return _attention._quick or _attention._fast()


def _kind(t):
    return (None, None) if t is None else (t.shape, t.dtype)


def _verify_plan(q, k, v, g, beta, state_in, cu_seqlens, parents, o, delta, chunk):
    """The C struct after checking the tensors' shapes and types against each other."""
    if q.dim() != 3 or v.dim() != 3 or cu_seqlens.dim() != 1:
        raise ValueError("q, k and v must be [tokens, heads, head_dim] and cu_seqlens [num_seqs + 1]")
    tokens, hk, dk = q.shape
    hv, dv = v.shape[1:]
    n = cu_seqlens.shape[0] - 1
    for what, t, dtype, size in (("k", k, q.dtype, q.shape), ("v", v, q.dtype, (tokens, hv, dv)),
                                 ("g", g, _F32, (tokens, hv)), ("beta", beta, _F32, (tokens, hv)),
                                 ("state_in", state_in, _F32, (n, hv, dk, dv)),
                                 ("cu_seqlens", cu_seqlens, _I32, (n + 1,)),
                                 ("parents", parents, _I32, (tokens,)),
                                 ("o", o, None if o is None else o.dtype, v.shape),
                                 ("delta", delta, _F32, v.shape)):
        if t is not None and (t.dtype != dtype or t.shape != size):
            raise ValueError("%s must be %s of shape %s" % (what, dtype, tuple(size)))
    if q.dtype not in _CODES or (o is not None and o.dtype not in (q.dtype, _F32)):
        raise TypeError("q, k and v must be bfloat16 or float32, and o of their type or float32")
    s = make_shape(n, tokens, hk, hv, dk, dv, chunk, _CODES[q.dtype], int(o is not None and o.dtype != q.dtype))
    return s, ctypes.byref(s), ctypes.addressof(s)


def gdn_verify_tree(q, k, v, g, beta, state_in, cu_seqlens, parents, o=None, delta=None,
                    chunk: int = 64, stream=None):
    """Draft-verify block whose drafts form a tree: parents [T] int32, each node's parent as an
    index into its own sequence's nodes (it stands before its child; -1: the node hangs on the
    snapshot).  q, k [T, Hk, 128], v [T, Hv, 128] bf16 or fp32; g, beta [T, Hv] fp32; state_in
    [N, Hv, 128, 128] fp32 (or None) is left unchanged and no state is written; o in q's type (or
    fp32, if given), delta [T, Hv, 128] fp32.  chunk (16, 32, 64): the most nodes of a tree.  The
    state after an accepted path: gdn_state_rollback on the path's rows of k, g and delta.
    Returns (o, delta)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gdn_verify_tree(q, k, v, g, beta, state_in, cu_seqlens, parents, o, delta, chunk)
    r = _quick().verify(_made, q, k, v, g, beta, state_in, cu_seqlens, parents, o, delta, chunk)
    if type(r) is int:
        raise GdnError(r, "gdn_verify_tree")
    if r is not None:
        return r
    _check_tensors(q, k, v, g, beta, state_in, cu_seqlens, parents, o, delta)
    key = ("verify", *_kind(q), *_kind(k), *_kind(v), *_kind(g), *_kind(beta), *_kind(state_in),
           *_kind(cu_seqlens), *_kind(parents), *_kind(o), *_kind(delta), chunk)
    pointer = (_made.get(key) or _remember(key, _verify_plan(
        q, k, v, g, beta, state_in, cu_seqlens, parents, o, delta, chunk), _made))[1]
    o = torch.empty_like(v) if o is None else o
    delta = torch.empty_like(v, dtype=_F32) if delta is None else delta
    st = lib().gdn_verify_tree(pointer, *[None if t is None else t.data_ptr() for t in (
        q, k, v, g, beta, state_in, cu_seqlens, parents, o, delta)], _raw_stream(q.get_device()))
    if st != GDN_OK:
        raise GdnError(st, "gdn_verify_tree")
    return o, delta


class GdnBeamShape(ctypes.Structure):
    """gdn_beam_shape (include/gdn.h)."""
    _fields_ = [("num_groups", ctypes.c_int32), ("beams", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("top", ctypes.c_int32), ("dtype", ctypes.c_int32), ("pad_token", ctypes.c_int32),
                ("row_stride", ctypes.c_int64)]


def make_beam_shape(num_groups: int, beams: int, vocab: int, top: int, dtype: int = GDN_BF16,
                    pad_token: int = 0, row_stride: int = 0) -> GdnBeamShape:
    """row_stride 0: contiguous logits."""
    return GdnBeamShape(num_groups, beams, vocab, top, dtype, pad_token, row_stride or vocab)


def gdn_beam_workspace_size(shape: GdnBeamShape) -> int:
    n = lib().gdn_beam_workspace_size(ctypes.byref(shape))
    if n == ctypes.c_size_t(-1).value:
        raise GdnError(GDN_ERR_INVALID_ARG, "gdn_beam_workspace_size")
    return n


def gdn_beam_workspace(num_groups: int, beams: int, vocab: int, top: int, device="cuda"):
    """A workspace for gdn_beam_select up to these sizes, for logits of either type, to be kept and
    given to every call (one per stream)."""
    size = max(gdn_beam_workspace_size(make_beam_shape(num_groups, beams, vocab, top, dtype))
               for dtype in (GDN_BF16, GDN_F32))
    return torch.empty(max(size, 1), dtype=torch.uint8, device=device)


def _on_current(what, t, dtype, shape):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() < 0 \
            or t.get_device() != _current_device():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on the current CUDA device"
                         % (what, dtype, tuple(shape)))
    return t.data_ptr()


def _select_plan(logits, scores, top, finished, pad_token):
    if logits.dim() != 3 or logits.dtype not in _CODES:
        raise ValueError("logits must be [groups, beams, vocab] in bfloat16 or float32")
    groups, beams, vocab = logits.shape
    st = logits.stride()
    row = st[1] if beams > 1 else st[0] if groups > 1 else vocab
    if (vocab > 1 and st[2] != 1) or (groups > 1 and st[0] != beams * row):
        raise ValueError("the rows of logits must be contiguous, and at equal distances")
    if row < vocab:  # (several rows: expanded logits, or views that overlap)
        raise ValueError("the rows of logits must not lie over each other (expanded logits: give a copy)")
    for what, t, dtype in (("scores", scores, _F32), ("finished", finished, torch.bool)):
        if t is not None and (t.dtype is not dtype or t.shape != (groups, beams)):
            raise ValueError("%s must be %s of shape %s" % (what, dtype, (groups, beams)))
    s = make_beam_shape(groups, beams, vocab, top, _CODES[logits.dtype], pad_token, row)
    return s, ctypes.byref(s), ctypes.addressof(s), (groups, top)


def gdn_beam_select(logits, scores, top: int, finished=None, pad_token: int = 0, scores_out=None,
                    parents=None, tokens=None, workspace=None, stream=None):
    """The `top` best continuations of each group's beams by scores + log_softmax(logits): logits
    [G, W, V] bf16 or fp32 (rows at equal distances of at least V, so no expanded ones), scores
    [G, W] fp32, finished [G, W] bool or None (a finished beam goes on with pad_token and keeps its
    score).  Returns (scores [G, top] fp32, parents [G, top] int32, tokens [G, top] int32), best
    first, equal ones in order of beam and token.  workspace: from gdn_beam_workspace (None: a
    fresh one)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gdn_beam_select(logits, scores, top, finished, pad_token, scores_out, parents, tokens,
                                   workspace)
    if scores_out is None and parents is None and tokens is None:
        r = _quick().select(_made, logits, scores, top, finished, pad_token, workspace)
        if type(r) is int:
            raise GdnError(r, "gdn_beam_select")
        if r is not None:
            return r
    key = ("select", logits.shape, logits.stride(), logits.dtype, *_kind(scores), *_kind(finished), top, pad_token)
    shape, pointer, _, out = _made.get(key) or _remember(
        key, _select_plan(logits, scores, top, finished, pad_token), _made)
    device = logits.get_device()
    if device < 0 or device != _current_device():
        raise ValueError("logits must be on the current CUDA device")
    rows = logits.shape[:2]
    given = _on_current("scores", scores, _F32, rows)
    done = None if finished is None else _on_current("finished", finished, torch.bool, rows)
    where = logits.device
    if scores_out is None:
        scores_out = torch.empty(out, dtype=_F32, device=where)
    if parents is None:
        parents = torch.empty(out, dtype=_I32, device=where)
    if tokens is None:
        tokens = torch.empty(out, dtype=_I32, device=where)
    if workspace is None:
        workspace = torch.empty(gdn_beam_workspace_size(shape), dtype=torch.uint8, device=where)
    elif workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the logits' device")
    st = lib().gdn_beam_select(pointer, logits.data_ptr(), given, done,
                               _on_current("scores_out", scores_out, _F32, out),
                               _on_current("parents", parents, _I32, out),
                               _on_current("tokens", tokens, _I32, out), workspace.data_ptr(),
                               workspace.nbytes, _raw_stream(device))
    if st != GDN_OK:
        raise GdnError(st, "gdn_beam_select")
    return scores_out, parents, tokens


def _reorder_plan(rows, parents):
    """(layers, groups, beams, bytes of a row)."""
    if parents.dim() != 2 or parents.dtype is not _I32:
        raise ValueError("parents must be int32 [groups, beams]")
    groups, beams = parents.shape
    if rows.dim() < 2 or rows.shape[1] != groups * beams:
        raise ValueError("rows must be [layers, groups * beams, ...]")
    return rows.shape[0], groups, beams, rows.nbytes // max(rows.shape[0] * rows.shape[1], 1)


def gdn_beam_reorder(rows, parents, stream=None):
    """In place: row (l, g, w) of rows becomes the row (l, g, parents[g, w]) from before.  rows: a
    contiguous CUDA tensor [layers, G * W, ...] of any type whose rows are multiples of 4 bytes;
    parents [G, W] int32.  Returns rows."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gdn_beam_reorder(rows, parents)
    r = _quick().reorder(_made, rows, parents)
    if type(r) is int:
        raise GdnError(r, "gdn_beam_reorder")
    if r is not None:
        return r
    _check_tensors(rows, parents)
    key = ("reorder", *_kind(rows), *_kind(parents))
    plan = _made.get(key) or _remember(key, _reorder_plan(rows, parents), _made)
    st = lib().gdn_beam_reorder(*plan, parents.data_ptr(), rows.data_ptr(), _raw_stream(rows.get_device()))
    if st != GDN_OK:
        raise GdnError(st, "gdn_beam_reorder")
    return rows
