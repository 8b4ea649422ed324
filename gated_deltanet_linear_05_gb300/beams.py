"""Binding of the beams' operators: the selection of the best continuations over beams and
vocabulary, and the reordering of the rows that follow the beams.

Argument marshalling only, as in the package itself; include/gdn.h has the contract of each call.  A
call that is given a stream runs with that stream current, so that what it allocates belongs to it.
"""
from __future__ import annotations

import ctypes

import torch

from . import GDN_BF16, GDN_ERR_INVALID_ARG, GDN_F32, GDN_OK, GdnError, lib
from .attention import _current_device, _raw_stream, _remember


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
    """A workspace for gdn_beam_select at these sizes, for logits of either type, to be kept and
    given to every call (one per stream)."""
    size = max(gdn_beam_workspace_size(make_beam_shape(num_groups, beams, vocab, top, dtype))
               for dtype in (GDN_BF16, GDN_F32))
    return torch.empty(max(size, 1), dtype=torch.uint8, device=device)


_made = {}  # by sizes and strides: the shape and a pointer to it
_CODES = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}
_I32, _F32 = torch.int32, torch.float32


def _on_current(what, t, dtype, shape):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() < 0 \
            or t.get_device() != _current_device():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on the current CUDA device"
                         % (what, dtype, tuple(shape)))
    return t.data_ptr()


def _plan(logits, top, pad_token):
    if logits.dim() != 3 or logits.dtype not in _CODES:
        raise ValueError("logits must be [groups, beams, vocab] in bfloat16 or float32")
    groups, beams, vocab = logits.shape
    st = logits.stride()
    row = st[1] if beams > 1 else st[0] if groups > 1 else vocab
    if (vocab > 1 and st[2] != 1) or (groups > 1 and st[0] != beams * row):
        raise ValueError("the rows of logits must be contiguous, and at equal distances")
    s = make_beam_shape(groups, beams, vocab, top, _CODES[logits.dtype], pad_token, row)
    return s, ctypes.byref(s), (groups, beams), (groups, top)


def gdn_beam_select(logits, scores, top: int, finished=None, pad_token: int = 0, scores_out=None,
                    parents=None, tokens=None, workspace=None, stream=None):
    """The `top` best continuations of each group's beams by scores + log_softmax(logits): logits
    [G, W, V] bf16 or fp32 (rows at equal distances), scores [G, W] fp32, finished [G, W] bool or
    None (a finished beam goes on with pad_token and keeps its score).  Returns (scores [G, top]
    fp32, parents [G, top] int32, tokens [G, top] int32), best first, equal ones in order of beam
    and token.  workspace: from gdn_beam_workspace (None: a fresh one)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gdn_beam_select(logits, scores, top, finished, pad_token, scores_out, parents, tokens,
                                   workspace)
    key = (logits.shape, logits.stride(), logits.dtype, top, pad_token)
    shape, pointer, rows, out = _made.get(key) or _remember(key, _plan(logits, top, pad_token), _made)
    device = logits.get_device()
    if device < 0 or device != _current_device():
        raise ValueError("logits must be on the current CUDA device")
    given = _on_current("scores", scores, _F32, rows)
    done = None
    if finished is not None:
        done = _on_current("finished", finished, torch.bool, rows)
    where = logits.device
    if scores_out is None:
        scores_out = torch.empty(out, dtype=_F32, device=where)
    if parents is None:
        parents = torch.empty(out, dtype=_I32, device=where)
    if tokens is None:
        tokens = torch.empty(out, dtype=_I32, device=where)
    if workspace is None:
        workspace = torch.empty(gdn_beam_workspace_size(shape) + 256, dtype=torch.uint8, device=where)
    elif workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the logits' device")
    base = workspace.data_ptr()
    at = (base + 255) & ~255
    st = lib().gdn_beam_select(pointer, logits.data_ptr(), given, done,
                               _on_current("scores_out", scores_out, _F32, out),
                               _on_current("parents", parents, _I32, out),
                               _on_current("tokens", tokens, _I32, out), at,
                               max(workspace.nbytes - (at - base), 0), _raw_stream(device))
    if st != GDN_OK:
        raise GdnError(st, "gdn_beam_select")
    return scores_out, parents, tokens


def gdn_beam_reorder(rows, parents, stream=None):
    """In place: row (l, g, w) of rows becomes the row (l, g, parents[g, w]) from before.  rows: a
    contiguous CUDA tensor [layers, G * W, ...] of any type whose rows are multiples of 4 bytes;
    parents [G, W] int32.  Returns rows."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gdn_beam_reorder(rows, parents)
    groups, beams = parents.shape
    p = _on_current("parents", parents, _I32, parents.shape)
    if rows.dim() < 2 or rows.shape[1] != groups * beams or not rows.is_contiguous() \
            or rows.get_device() != parents.get_device():
        raise ValueError("rows must be a contiguous [layers, groups * beams, ...] tensor on parents' device")
    layers, count = rows.shape[:2]
    st = lib().gdn_beam_reorder(layers, groups, beams, rows.nbytes // max(layers * count, 1), p,
                                rows.data_ptr(), _raw_stream(rows.get_device()))
    if st != GDN_OK:
        raise GdnError(st, "gdn_beam_reorder")
    return rows
