"""Binding of the attention-layer operators: residual + RMS norm, rotary positions and the
append to the paged cache, attention over the cache, and the same behind a shared prefix.

Argument marshalling only, as in the package itself; include/gdn.h has the contract of each
call.  A call that is given a stream runs with that stream current, so that what it allocates
belongs to it: outputs come as if made under torch.cuda.stream(stream).

The shape structs are kept by sizes and strides, so that a decode loop builds them once; a call
whose combination has been seen goes through _marshal (csrc/marshal.c), which does the same
checks in C and hands anything unusual back to the functions here.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from . import GDN_BF16, GDN_ERR_INVALID_ARG, GDN_F32, GDN_OK, GdnError, lib

I64x2 = ctypes.c_int64 * 2
_COUNTER_BYTES = 2048  # GDN_ATTN_COUNTER_BYTES (include/gdn.h)


class GdnAttnShape(ctypes.Structure):
    """gdn_attn_shape (include/gdn.h)."""
    _fields_ = [("num_seqs", ctypes.c_int32), ("total_tokens", ctypes.c_int32),
                ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("prefix_len", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("num_axes", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("scale", ctypes.c_float),
                ("q_stride", I64x2), ("k_stride", I64x2), ("v_stride", I64x2),
                ("gate_stride", I64x2), ("page_stride", ctypes.c_int64)]


def make_attn_shape(num_seqs: int, total_tokens: int, num_q_heads: int, num_kv_heads: int,
                    head_dim: int = 128, page_size: int = 64, num_pages: int = 0,
                    max_pages: int = 0, prefix_len: int = 0, rotary_dim: int = 0,
                    num_axes: int = 1, scale: Optional[float] = None,
                    dtype: int = GDN_BF16) -> GdnAttnShape:
    """A shape with contiguous tensors; the stride fields may be changed afterwards."""
    s = GdnAttnShape(num_seqs, total_tokens, num_q_heads, num_kv_heads, head_dim, page_size,
                     num_pages, max_pages, prefix_len, rotary_dim, num_axes, dtype,
                     1.0 / math.sqrt(max(head_dim, 1)) if scale is None else scale)
    s.q_stride[:] = s.gate_stride[:] = (num_q_heads * head_dim, head_dim)
    s.k_stride[:] = s.v_stride[:] = (num_kv_heads * head_dim, head_dim)
    s.page_stride = num_kv_heads * page_size * head_dim
    return s


def _shape(n, tokens, hq, hkv, d, page_size, num_pages, max_pages, prefix_len, rotary_dim, axes,
           scale, page_stride, q_stride, k_stride=None, v_stride=None, gate_stride=None):
    """The C struct for these sizes and strides (never changed once made)."""
    s = make_attn_shape(n, tokens, hq, hkv, d, page_size, num_pages, max_pages, prefix_len,
                        rotary_dim, axes, scale)
    s.page_stride = page_stride
    for field, st in (("q_stride", q_stride), ("k_stride", k_stride), ("v_stride", v_stride),
                      ("gate_stride", gate_stride)):
        if st is not None:
            getattr(s, field)[:] = st
    return s, ctypes.byref(s), ctypes.addressof(s)


def gdn_attn_workspace_size(shape: GdnAttnShape) -> int:
    n = lib().gdn_attn_workspace_size(ctypes.byref(shape))
    if n == ctypes.c_size_t(-1).value:
        raise GdnError(GDN_ERR_INVALID_ARG, "gdn_attn_workspace_size")
    return n


def gdn_attn_workspace(num_seqs: int, total_tokens: int, num_q_heads: int, num_kv_heads: int,
                       head_dim: int, prefix_len: int = 0, device="cuda"):
    """A workspace for the attention calls up to these sizes, ready for the first, to be kept and
    given to every call (one per stream)."""
    shape = make_attn_shape(num_seqs, total_tokens, num_q_heads, num_kv_heads, head_dim,
                            prefix_len=prefix_len)
    return _new_workspace(shape, device)


def _new_workspace(shape, device):
    """Its counters zeroed; the rest may hold anything.  (The caching allocator's blocks start on
    512-byte boundaries.)"""
    ws = torch.empty(max(gdn_attn_workspace_size(shape), 1), dtype=torch.uint8, device=device)
    ws[:_COUNTER_BYTES].zero_()
    return ws


def _strides3(t, what):
    """(token, head) strides of a [T, H, D] bf16 tensor whose rows are contiguous."""
    st = t.stride()
    if len(st) != 3 or st[2] != 1:
        raise ValueError("%s must be a [tokens, heads, head_dim] CUDA tensor with contiguous rows"
                         % what)
    if t.shape[0] <= 1 or t.shape[1] <= 1:  # torch leaves the stride of a size of 1 open
        d = t.shape[2]
        head = st[1] if t.shape[1] > 1 else d
        return (st[0] if t.shape[0] > 1 else max(t.shape[1] * head, d), head)
    return st[:2]


def _cache(k_cache, v_cache):
    """(num_pages, hkv, page_size, d, page_stride) of a pair of caches."""
    shape, st = k_cache.shape, k_cache.stride()
    if len(shape) != 4 or v_cache.shape != shape or v_cache.stride() != st:
        raise ValueError("the caches must be two alike [pages, kv_heads, page_size, head_dim] "
                         "bfloat16 CUDA tensors")
    pages, hkv, size, d = shape
    if st[3] != 1 or (size > 1 and st[2] != d) or (hkv > 1 and st[1] != size * d):
        raise ValueError("a page's heads must be contiguous in the caches")
    return pages, hkv, size, d, (st[0] if pages > 1 else hkv * size * d)


_BF16, _I32, _F32 = torch.bfloat16, torch.int32, torch.float32
_DENSE = torch.contiguous_format


def _check(device, bf16, index):
    """Types and places of a call's tensors.  (Written out in one expression where it passes: a call
    for each tensor costs as much as the launch.)"""
    for t in bf16:
        if t.dtype is not _BF16 or t.get_device() != device:
            break
    else:
        for t in index:
            if t is not None and (t.dtype is not _I32 or t.get_device() != device
                                  or not t.is_contiguous()):
                break
        else:
            if device >= 0 and device == _current_device():
                return
    for t in bf16:
        if t.dtype is not _BF16:
            raise TypeError("q, k, v, gate and the caches must be bfloat16, got %s" % t.dtype)
    if device >= 0:
        _check_device(device)
    raise ValueError("the tensors must be CUDA tensors of one device, and those of indices contiguous "
                     "int32")


def _check_device(device):
    """The library launches on the current device."""
    if device != _current_device():
        raise ValueError("the tensors must be of the current device (cuda:%d), got cuda:%d"
                         % (_current_device(), device))


def _float(device, t, shape, what):
    if t.dtype is not _F32 or t.get_device() != device or not t.is_contiguous() or t.shape != shape:
        raise ValueError("%s must be a contiguous float32 CUDA tensor of shape %s"
                         % (what, tuple(shape)))
    return t.data_ptr()


def _output(device, t, like, what):
    if t.shape != like.shape or t.dtype is not _BF16 or t.get_device() != device \
            or not t.is_contiguous():
        raise ValueError("%s must be a contiguous bfloat16 CUDA tensor of q's shape" % what)
    return t


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
# The device's current stream as a raw handle: making a Stream object costs as much as the rest of
# the marshalling.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)


def _sequences(page_table, kv_lens, cu_seqlens):
    """(num_seqs, max_pages) after checking the index tensors' shapes against each other."""
    n = kv_lens.shape[0]
    if page_table.dim() != 2 or page_table.shape[0] != n or kv_lens.dim() != 1:
        raise ValueError("page_table must be [num_seqs, max_pages] and kv_lens [num_seqs]")
    if cu_seqlens is not None and tuple(cu_seqlens.shape) != (n + 1,):
        raise ValueError("cu_seqlens must be [num_seqs + 1]")
    return n, page_table.shape[1]


# What follows from the tensors' sizes and strides alone is checked and built once for each
# combination of them: (shape struct, pointer to it).
_made = {}


def _remember(key, value):
    if len(_made) >= 4096:
        _made.clear()
    _made[key] = value
    return value


_quick = None


class _Unbuilt:
    """In _marshal's place: every call is left to the functions here."""
    @staticmethod
    def attend(*args):
        return None

    append = norm = attend


def _fast():
    """The marshalling module, bound to torch and to the library's entry points; where it has not
    been built, a stand-in that has seen no call."""
    global _quick
    if _quick is None:
        L = lib()
        try:
            from . import _marshal
        except ImportError:
            _quick = _Unbuilt
            return _quick
        _marshal.bind(_BF16, _F32, torch.float64, _I32, torch.empty, torch.empty_like, _raw_stream,
                      _DENSE, _current_device, *(ctypes.cast(getattr(L, f), ctypes.c_void_p).value for f in
                                ("gdn_paged_attention", "gdn_shared_prefix_attention", "gdn_kv_append",
                                 "gdn_add_rmsnorm")))
        _quick = _marshal
    return _quick


def _append_shape(q, k, v, k_cache, v_cache, page_table, kv_lens, inv_freq, cu_seqlens, positions,
                  rope_axis, prefix_len):
    pages, hkv, size, d, page_stride = _cache(k_cache, v_cache)
    n, max_pages = _sequences(page_table, kv_lens, cu_seqlens)
    qs = _strides3(q, "q"), _strides3(k, "k"), _strides3(v, "v")
    tokens, hq = q.shape[0], q.shape[1]
    if q.shape[2] != d or k.shape != (tokens, hkv, d) or v.shape != (tokens, hkv, d):
        raise ValueError("q, k, v and the caches must agree in tokens, kv heads and head_dim")
    axes = 1
    if positions is not None:
        axes = 1 if positions.dim() == 1 else positions.shape[0]
        if positions.shape[-1] != tokens or positions.dim() > 2:
            raise ValueError("positions must be [tokens] or [axes, tokens]")
    rot = 0
    if inv_freq is not None:
        rot = 2 * inv_freq.shape[0]
        if rope_axis is not None and rope_axis.shape != inv_freq.shape:
            raise ValueError("rope_axis must have one entry per frequency")
    return _shape(n, tokens, hq, hkv, d, size, pages, max_pages, prefix_len, rot, axes, None,
                  page_stride, *qs)


def gdn_kv_append(q, k, v, k_cache, v_cache, page_table, kv_lens, inv_freq=None, cu_seqlens=None,
                  positions=None, rope_axis=None, q_norm=None, k_norm=None, eps: float = 1e-6,
                  q_out=None, prefix_len: int = 0, stream=None):
    """Per-head RMS norm of q and k (with q_norm / k_norm [D] fp32), rotation of their first
    2 * len(inv_freq) elements, q to q_out, k and v to their place in the paged cache.
    q [T, Hq, D], k, v [T, Hkv, D] bf16, any token and head strides; caches
    [pages, Hkv, page_size, D]; page_table [N, max_pages], kv_lens [N] (the call's tokens
    included), cu_seqlens [N+1] int32 or None (one token per sequence); inv_freq [R/2] fp64
    or None (no rotation); positions [T] or [axes, T] int32 (None: prefix_len + place) with
    rope_axis [R/2] int32.  q_out None: a new tensor.  Returns q_out."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gdn_kv_append(q, k, v, k_cache, v_cache, page_table, kv_lens, inv_freq, cu_seqlens,
                                 positions, rope_axis, q_norm, k_norm, eps, q_out, prefix_len)
    r = (_quick or _fast()).append(_made, q, k, v, k_cache, v_cache, page_table, kv_lens, inv_freq,
                                   cu_seqlens, positions, rope_axis, q_norm, k_norm, eps, q_out,
                                   prefix_len)
    if type(r) is int:
        raise GdnError(r, "gdn_kv_append")
    if r is not None:
        return r
    device = q.get_device()
    _check(device, (q, k, v, k_cache, v_cache),
           (page_table, kv_lens, cu_seqlens, positions, rope_axis))
    if inv_freq is not None and (inv_freq.dtype is not torch.float64 or inv_freq.get_device() != device
                                 or not inv_freq.is_contiguous()):
        raise ValueError("inv_freq must be a contiguous float64 CUDA tensor")
    key = (q.shape, q.stride(), k.shape, k.stride(), v.shape, v.stride(), k_cache.shape,
           k_cache.stride(), v_cache.shape, v_cache.stride(), page_table.shape, kv_lens.shape,
           None if inv_freq is None else inv_freq.shape,
           None if cu_seqlens is None else cu_seqlens.shape,
           None if positions is None else positions.shape,
           None if rope_axis is None else rope_axis.shape, prefix_len)
    made = _made.get(key) or _remember(key, _append_shape(
        q, k, v, k_cache, v_cache, page_table, kv_lens, inv_freq, cu_seqlens, positions, rope_axis,
        prefix_len))
    d = k_cache.shape[3:]
    q_out = torch.empty_like(q, memory_format=_DENSE) if q_out is None \
        else _output(device, q_out, q, "q_out")
    st = lib().gdn_kv_append(
        made[1], q.data_ptr(), k.data_ptr(), v.data_ptr(),
        None if q_norm is None else _float(device, q_norm, d, "q_norm"),
        None if k_norm is None else _float(device, k_norm, d, "k_norm"), eps,
        None if inv_freq is None else inv_freq.data_ptr(),
        None if rope_axis is None else rope_axis.data_ptr(),
        None if positions is None else positions.data_ptr(),
        page_table.data_ptr(), kv_lens.data_ptr(),
        None if cu_seqlens is None else cu_seqlens.data_ptr(),
        q_out.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _raw_stream(device))
    if st != GDN_OK:
        raise GdnError(st, "gdn_kv_append")
    return q_out


def _attend_shape(q, k_cache, v_cache, prefix_table, prefix_len, page_table, kv_lens, cu_seqlens,
                  gate, scale):
    pages, hkv, size, d, page_stride = _cache(k_cache, v_cache)
    n, max_pages = _sequences(page_table, kv_lens, cu_seqlens)
    q_stride = _strides3(q, "q")
    if q.shape[2] != d:
        raise ValueError("q and the caches must agree in head_dim")
    if gate is not None and gate.shape != q.shape:
        raise ValueError("gate must have q's shape")
    if prefix_table is not None and prefix_table.numel() * size < prefix_len:
        raise ValueError("prefix_table must cover prefix_len keys")
    return _shape(n, q.shape[0], q.shape[1], hkv, d, size, pages, max_pages, prefix_len, 0, 1,
                  scale, page_stride, q_stride, None, None,
                  None if gate is None else _strides3(gate, "gate"))


def _attend(name, q, k_cache, v_cache, prefix_table, prefix_len, page_table, kv_lens, cu_seqlens,
            gate, scale, o, lse, workspace, stream):
    if stream is not None:
        with torch.cuda.stream(stream):
            return _attend(name, q, k_cache, v_cache, prefix_table, prefix_len, page_table, kv_lens,
                           cu_seqlens, gate, scale, o, lse, workspace, None)
    if lse is None:
        r = (_quick or _fast()).attend(_made, q, k_cache, v_cache, prefix_table, prefix_len, page_table,
                                       kv_lens, cu_seqlens, gate, scale, o, workspace)
        if type(r) is int:
            raise GdnError(r, name)
        if r is not None:
            return r
    device = q.get_device()
    _check(device, (q, k_cache, v_cache) if gate is None else (q, k_cache, v_cache, gate),
           (page_table, kv_lens, cu_seqlens, prefix_table))
    key = (q.shape, q.stride(), k_cache.shape, k_cache.stride(), v_cache.shape, v_cache.stride(),
           page_table.shape, kv_lens.shape, None if cu_seqlens is None else cu_seqlens.shape,
           None if gate is None else (gate.shape, gate.stride()), scale,
           None if prefix_table is None else prefix_table.shape, prefix_len)
    made = _made.get(key) or _remember(key, _attend_shape(
        q, k_cache, v_cache, prefix_table, prefix_len, page_table, kv_lens, cu_seqlens, gate, scale))
    o = torch.empty_like(q, memory_format=_DENSE) if o is None \
        else _output(device, o, q, "o")
    if workspace is None:
        workspace = _new_workspace(made[0], q.device)
    elif workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the queries' device")
    args = [made[1], q.data_ptr(), None if gate is None else gate.data_ptr(), k_cache.data_ptr(),
            v_cache.data_ptr(), page_table.data_ptr(), kv_lens.data_ptr(),
            None if cu_seqlens is None else cu_seqlens.data_ptr(), o.data_ptr(),
            None if lse is None else _float(device, lse, q.shape[:2], "lse"), workspace.data_ptr(),
            workspace.nbytes, _raw_stream(device)]
    if prefix_table is None:
        st = lib().gdn_paged_attention(*args)
    else:
        args.insert(5, prefix_table.data_ptr())
        st = lib().gdn_shared_prefix_attention(*args)
    if st != GDN_OK:
        raise GdnError(st, name)
    return o


def gdn_paged_attention(q, k_cache, v_cache, page_table, kv_lens, cu_seqlens=None, gate=None,
                        scale: Optional[float] = None, o=None, lse=None, workspace=None,
                        stream=None):
    """Causal attention of q [T, Hq, D] over each sequence's keys in the paged cache, times
    sigmoid(gate) with a gate.  cu_seqlens None: one token per sequence.  scale None:
    1 / sqrt(D).  lse (fp32 [T, Hq], optional) receives ln of each row's sum of exp(scores).
    workspace: from gdn_attn_workspace, kept by the caller (None: a fresh one per call).  Returns o."""
    return _attend("gdn_paged_attention", q, k_cache, v_cache, None, 0, page_table, kv_lens,
                   cu_seqlens, gate, scale, o, lse, workspace, stream)


def gdn_shared_prefix_attention(q, k_cache, v_cache, prefix_table, prefix_len: int, page_table,
                                kv_lens, cu_seqlens=None, gate=None,
                                scale: Optional[float] = None, o=None, lse=None, workspace=None,
                                stream=None):
    """gdn_paged_attention with prefix_len keys in front that every sequence shares: the pages
    in prefix_table [ceil(prefix_len / page_size)] int32.  kv_lens counts the sequences' own
    keys alone.  Returns o."""
    return _attend("gdn_shared_prefix_attention", q, k_cache, v_cache, prefix_table, prefix_len,
                   page_table, kv_lens, cu_seqlens, gate, scale, o, lse, workspace, stream)


def _norm_plan(x, out, group):
    """(rows, columns, dtype code, output type, shape of the scales)."""
    cols = x.shape[-1]
    code = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}.get(x.dtype)
    if code is None:
        raise TypeError("x must be bfloat16 or float32, got %s" % x.dtype)
    if out not in ("same", "e4m3"):
        raise ValueError("out must be 'same' or 'e4m3'")
    if out == "same" and group:
        raise ValueError("groups go with out='e4m3'")
    if group and (group != 128 or cols % 128):
        raise ValueError("group must be 0, or 128 and divide the columns")
    scales = None if out == "same" else x.shape[:-1] + ((cols // group if group else 1),)
    return (x.numel() // max(cols, 1), cols, code, x.dtype if out == "same" else torch.float8_e4m3fn,
            scales)


def _alike(device, x, t):
    if t.dtype is not x.dtype or t.shape != x.shape or t.get_device() != device \
            or not t.is_contiguous():
        raise ValueError("x, residual and residual_out must be alike, contiguous CUDA tensors")
    return t.data_ptr()


def gdn_add_rmsnorm(x, residual, weight, eps: float = 1e-6, residual_out=None, y=None, scale=None,
                    out: str = "same", group: int = 0, stream=None):
    """h = x + residual (rounded to x's type; x itself with residual None) and its RMS norm
    y = h / sqrt(mean(h^2) + eps) * weight over the last dimension.  out "same": y in x's
    type, returns (y, h); out "e4m3": y in float8_e4m3fn with fp32 scales per row (group 0) or
    per 128 columns (group 128), returns (y, scale, h).  x, residual bf16 or fp32; weight
    fp32.  residual_out may be residual or x."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gdn_add_rmsnorm(x, residual, weight, eps, residual_out, y, scale, out, group)
    if residual_out is None and y is None and scale is None:
        r = (_quick or _fast()).norm(_made, x, residual, weight, eps, out, group)
        if type(r) is int:
            raise GdnError(r, "gdn_add_rmsnorm")
        if r is not None:
            return r
    device = x.get_device()
    key = ("norm", x.shape, x.dtype, out, group)
    rows, cols, code, kind, scales = _made.get(key) or _remember(key, _norm_plan(x, out, group))
    if device < 0:
        raise ValueError("x must be a CUDA tensor")
    _check_device(device)
    xp = _alike(device, x, x)
    rp = None if residual is None else _alike(device, x, residual)
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(x)
        hp = residual_out.data_ptr()
    else:
        hp = None if residual_out is None else _alike(device, x, residual_out)
    if y is None:
        y = torch.empty_like(x, dtype=kind)
    elif y.dtype is not kind or y.shape != x.shape or y.get_device() != device \
            or not y.is_contiguous():
        raise ValueError("y must be a contiguous %s CUDA tensor of x's shape" % kind)
    sp = None
    if scales is not None:
        if scale is None:
            scale = torch.empty(scales, dtype=_F32, device=x.device)
            sp = scale.data_ptr()
        else:
            sp = _float(device, scale, scales, "scale")
    st = lib().gdn_add_rmsnorm(rows, cols, code, xp, rp, _float(device, weight, x.shape[-1:], "weight"),
                               eps, hp, y.data_ptr(), sp, group, _raw_stream(device))
    if st != GDN_OK:
        raise GdnError(st, "gdn_add_rmsnorm")
    h = x if residual_out is None else residual_out
    return (y, h) if out == "same" else (y, scale, h)
