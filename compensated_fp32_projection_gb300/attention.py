"""Attention and its paged cache, bound to torch tensors.

As in the projections' binding, these functions only marshal arguments into
``libcompfp32.so``; every step runs in its CUDA kernels, on the current stream
unless one is given, and nothing waits for the host.  Outputs that are not
given are allocated with ``torch.empty``.

Caches are pairs of float16 tensors ``k_pages``, ``v_pages``
[pages, kv_heads, page_size, head_dim]; a page table is an int32 tensor
[rows, width] whose unused entries are -1.
"""
from __future__ import annotations

import ctypes

import torch

from . import _native

__all__ = [
    "comp_attn_f32",
    "comp_attn_f32x16",
    "comp_attn_decode_f32x16",
    "comp_kv_append_f32",
    "comp_kv_reserve",
    "comp_kv_fork",
    "comp_kv_free",
    "comp_kv_compact",
    "comp_kv_copy_pages",
]


_F32, _F16, _I32, _U8 = torch.float32, torch.float16, torch.int32, torch.uint8
_empty, _raw_stream = torch.empty, torch._C._cuda_getCurrentRawStream


def _stream(device, stream):
    if stream is None:
        return _raw_stream(device.index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _refuse(t, dtype, name, device, shape, dense):
    """Say what is wrong with an argument (the checks themselves are in _check and _heads)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on another device")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must be [tokens, heads, head_dim], contiguous in its last dimension")


def _check(t, dtype, name, device, shape):
    """A dense tensor of this type and shape; its address."""
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.is_cuda and t.device == device
            and t.shape == shape and t.is_contiguous()):
        _refuse(t, dtype, name, device, shape, True)
    return t.data_ptr()


def _heads(t, dtype, name, device=None):
    """A [tokens, heads, head_dim] tensor with any token and head strides; its shape and strides."""
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.is_cuda
            and (device is None or t.device == device) and t.dim() == 3):
        _refuse(t, dtype, name, device, None, False)
    shape, strides = t.shape, t.stride()
    if strides[2] != 1 and shape[2] > 1 and t.numel() > 0:
        _refuse(t, dtype, name, device, None, False)
    return shape, strides


def _workspace(given, nbytes, device):
    """(the tensor that holds it, its address, its bytes)"""
    if given is None:
        if nbytes <= 0:
            return None, None, 0
        given = _empty(nbytes, dtype=_U8, device=device)
        return given, given.data_ptr(), nbytes
    if given.device != device or not given.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return given, given.data_ptr(), given.nbytes


def _attn(name, kv_dtype, q, k, v, cu_q, cu_k, scale, causal, out, lse, workspace, stream):
    q_shape, q_stride = _heads(q, _F32, "q")
    device = q.device
    k_shape, k_stride = _heads(k, kv_dtype, "k", device)
    v_shape, v_stride = _heads(v, kv_dtype, "v", device)
    tokens, heads, dim = q_shape
    keys, kv_heads, k_dim = k_shape
    if k_shape != v_shape or k_dim != dim:
        raise ValueError("k and v must be [keys, kv_heads, head_dim] with q's head_dim")
    if kv_heads == 0 or heads == 0 or heads % kv_heads:
        raise ValueError("q's heads must be a multiple of the key/value heads")
    n_seq, at_q, at_k = 1, None, None
    if cu_q is not None or cu_k is not None:
        if cu_q is None or cu_k is None:
            raise ValueError("cu_q and cu_k go together")
        if not isinstance(cu_q, torch.Tensor) or cu_q.dim() != 1 or cu_q.shape[0] < 1:
            raise ValueError("cu_q and cu_k must be [sequences + 1]")
        shape = cu_q.shape
        n_seq = shape[0] - 1
        at_q = _check(cu_q, _I32, "cu_q", device, shape)
        at_k = at_q if cu_k is cu_q else _check(cu_k, _I32, "cu_k", device, shape)
    if out is None:
        out = _empty(q_shape, dtype=_F32, device=device)
        out_stride = (heads * dim, dim)
    else:
        out_shape, out_stride = _heads(out, _F32, "out", device)
        if out_shape != q_shape:
            raise ValueError("out must have the shape of q")
    at_lse = None if lse is None else _check(lse, _F32, "lse", device, (tokens, heads))
    lib = _native.load()
    a = ctypes.byref(_native.Attn(n_seq, tokens, keys, heads, kv_heads, dim, 1 if causal else 0,
                                  dim ** -0.5 if scale is None else scale, q_stride[0], q_stride[1], k_stride[0],
                                  k_stride[1], v_stride[0], v_stride[1], out_stride[0], out_stride[1]))
    k_at, v_at = k.data_ptr(), v.data_ptr()
    need = lib.comp_attn_workspace_bytes(a, 4 if kv_dtype is _F32 else 2, k_at, v_at)
    held, ws, ws_bytes = _workspace(workspace, need, device)
    status = getattr(lib, name)(a, q.data_ptr(), k_at, v_at, at_q, at_k, out.data_ptr(), at_lse, ws, ws_bytes,
                                _stream(device, stream))
    if status:
        raise _native.CompError(status, name)
    return out


def comp_attn_f32(q, k, v, cu_q=None, cu_k=None, *, scale=None, causal=True, out=None, lse=None, workspace=None,
                  stream=None):
    """Attention of packed prompts: softmax(scale q k^T) v, all in float32.

    q [tokens, heads, head_dim]; k, v [keys, kv_heads, head_dim]; any token and
    head strides.  Sequence i has the queries cu_q[i]:cu_q[i+1] and the keys
    cu_k[i]:cu_k[i+1] (int32; without them there is one sequence).  causal: the
    last query sees every key of its sequence, each earlier one a key less.
    scale defaults to head_dim ** -0.5.  lse, if given ([tokens, heads]),
    receives the log-sum-exp of each row.  A row that sees no key gives zeros
    and -inf."""
    return _attn("comp_attn_f32", _F32, q, k, v, cu_q, cu_k, scale, causal, out, lse, workspace, stream)


def comp_attn_f32x16(q, k, v, cu_q=None, cu_k=None, *, scale=None, causal=True, out=None, lse=None, workspace=None,
                     stream=None):
    """comp_attn_f32 with float16 keys and values, which enter the products exactly."""
    return _attn("comp_attn_f32x16", _F16, q, k, v, cu_q, cu_k, scale, causal, out, lse, workspace, stream)


def _cache(k_pages, v_pages):
    """(the descriptor, its shape, the device)"""
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise ValueError("k_pages must be [pages, kv_heads, page_size, head_dim]")
    device, shape = k_pages.device, k_pages.shape
    at_k = _check(k_pages, _F16, "k_pages", device, shape)
    at_v = _check(v_pages, _F16, "v_pages", device, shape)
    return _native.KvCache(at_k, at_v, shape[0], shape[2], shape[1], shape[3]), shape, device


def _table(table, device):
    """(rows, width, address)"""
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be [rows, width]")
    rows, width = table.shape
    return rows, width, _check(table, _I32, "table", device, (rows, width))


def _list(t, name, device):
    """An int32 list: its length and address."""
    if not isinstance(t, torch.Tensor) or t.dim() != 1:
        raise ValueError(f"{name} must be a one-dimensional tensor")
    n = t.shape[0]
    return n, _check(t, _I32, name, device, (n,))


def _new(given, name, device, shape):
    """An int32 output, new unless given: itself and its address."""
    if given is None:
        given = _empty(shape, dtype=_I32, device=device)
        return given, given.data_ptr()
    return given, _check(given, _I32, name, device, shape)


def _call(name, *args):
    status = getattr(_native.load(), name)(*args)
    if status:
        raise _native.CompError(status, name)


def comp_kv_append_f32(k, v, k_pages, v_pages, table, start, cu=None, stream=None):
    """Write new tokens' float32 k, v [tokens, kv_heads, head_dim] into the cache
    (rounded to float16).  Row r's tokens cu[r]:cu[r+1] (without cu: one for each
    row) go to positions start[r], start[r] + 1, ... of its pages."""
    c, shape, device = _cache(k_pages, v_pages)
    rows, width, at_table = _table(table, device)
    k_shape, k_stride = _heads(k, _F32, "k", device)
    v_shape, v_stride = _heads(v, _F32, "v", device)
    tokens = k_shape[0]
    if k_shape != v_shape or k_shape[1] != shape[1] or k_shape[2] != shape[3]:
        raise ValueError("k and v must be [tokens, kv_heads, head_dim] as the cache has them")
    at_start = _check(start, _I32, "start", device, (rows,))
    at_cu = None
    if cu is not None:
        at_cu = _check(cu, _I32, "cu", device, (rows + 1,))
    elif tokens != rows:
        raise ValueError("without cu there must be one token for each row of table")
    _call("comp_kv_append_f32", ctypes.byref(c), k.data_ptr(), v.data_ptr(), k_stride[0], k_stride[1], v_stride[0],
          v_stride[1], tokens, at_table, rows, width, at_cu, at_start, _stream(device, stream))


def comp_attn_decode_f32x16(q, k_pages, v_pages, table, lengths, *, shared=0, scale=None, out=None, lse=None,
                            workspace=None, stream=None):
    """Attention of one token for each sequence over the paged cache.

    q [batch, heads, head_dim] float32 (any token and head strides); sequence b
    sees the tokens 0 .. lengths[b] - 1 on the pages that row b of table lists.
    The first `shared` entries are the same in all rows: those pages are read
    once for the whole batch.  lse [batch, heads] as in comp_attn_f32."""
    c, shape, device = _cache(k_pages, v_pages)
    batch, width, at_table = _table(table, device)
    q_shape, q_stride = _heads(q, _F32, "q", device)
    tokens, heads, dim = q_shape
    if tokens != batch or dim != shape[3] or shape[1] == 0 or heads == 0 or heads % shape[1]:
        raise ValueError("q must be [rows of table, a multiple of kv_heads, head_dim]")
    at_lengths = _check(lengths, _I32, "lengths", device, (batch,))
    if out is None:
        out = _empty(q_shape, dtype=_F32, device=device)
        at_out = out.data_ptr()
    else:
        at_out = _check(out, _F32, "out", device, q_shape)
    at_lse = None if lse is None else _check(lse, _F32, "lse", device, (batch, heads))
    lib, ref, shared = _native.load(), ctypes.byref(c), int(shared)
    need = lib.comp_attn_decode_workspace_bytes(ref, batch, heads, width, shared)
    held, ws, ws_bytes = _workspace(workspace, need, device)
    status = lib.comp_attn_decode_f32x16(ref, q.data_ptr(), q_stride[0], q_stride[1], heads,
                                         dim ** -0.5 if scale is None else scale, at_table, batch, width, at_lengths,
                                         shared, at_out, at_lse, ws, ws_bytes, _stream(device, stream))
    if status:
        raise _native.CompError(status, "comp_attn_decode_f32x16")
    return out


def comp_kv_reserve(table, want, refs, page_size, table_out=None, refs_out=None, left=None, stream=None):
    """Give row r of table the pages that want[r] tokens need, lowest free page
    first.  Returns (table, refs, left), new tensors unless given (the inputs
    themselves may be given: updated in place).  left[0] is the number of free
    pages that remain; where it is negative that many are missing and nothing
    was changed."""
    device = table.device
    rows, width, at_table = _table(table, device)
    at_want = _check(want, _I32, "want", device, (rows,))
    pages, at_refs = _list(refs, "refs", device)
    table_out, to_table = _new(table_out, "table_out", device, (rows, width))
    refs_out, to_refs = _new(refs_out, "refs_out", device, (pages,))
    left, to_left = _new(left, "left", device, (1,))
    _call("comp_kv_reserve", pages, int(page_size), at_table, at_refs, rows, width, at_want, to_table, to_refs, to_left,
          _stream(device, stream))
    return table_out, refs_out, left


def comp_kv_fork(k_pages, v_pages, table, lengths, refs, parents, children, table_out=None, lengths_out=None,
                 refs_out=None, left=None, stream=None):
    """Make the empty rows children[i] copies of rows parents[i]: full pages are
    shared, a partly filled last page is copied to a free one.  Returns (table,
    lengths, refs, left), new tensors unless given (see comp_kv_reserve); the
    caches are written in place."""
    c, shape, device = _cache(k_pages, v_pages)
    rows, width, at_table = _table(table, device)
    pages = shape[0]
    at_lengths = _check(lengths, _I32, "lengths", device, (rows,))
    at_refs = _check(refs, _I32, "refs", device, (pages,))
    n, at_parents = _list(parents, "parents", device)
    at_children = _check(children, _I32, "children", device, (n,))
    table_out, to_table = _new(table_out, "table_out", device, (rows, width))
    lengths_out, to_lengths = _new(lengths_out, "lengths_out", device, (rows,))
    refs_out, to_refs = _new(refs_out, "refs_out", device, (pages,))
    left, to_left = _new(left, "left", device, (1,))
    _call("comp_kv_fork", ctypes.byref(c), at_table, at_lengths, at_refs, rows, width, at_parents, at_children, n,
          to_table, to_lengths, to_refs, to_left, _stream(device, stream))
    return table_out, lengths_out, refs_out, left


def comp_kv_free(table, lengths, refs, seqs, table_out=None, lengths_out=None, refs_out=None, stream=None):
    """Give back the pages of the rows seqs and empty them.  Returns (table,
    lengths, refs), new tensors unless given (see comp_kv_reserve)."""
    device = table.device
    rows, width, at_table = _table(table, device)
    at_lengths = _check(lengths, _I32, "lengths", device, (rows,))
    pages, at_refs = _list(refs, "refs", device)
    n, at_seqs = _list(seqs, "seqs", device)
    table_out, to_table = _new(table_out, "table_out", device, (rows, width))
    lengths_out, to_lengths = _new(lengths_out, "lengths_out", device, (rows,))
    refs_out, to_refs = _new(refs_out, "refs_out", device, (pages,))
    _call("comp_kv_free", pages, at_table, at_lengths, at_refs, rows, width, at_seqs, n, to_table, to_lengths, to_refs,
          _stream(device, stream))
    return table_out, lengths_out, refs_out


def comp_kv_compact(k_pages, v_pages, table, refs, table_out=None, refs_out=None, remap=None, live=None, stream=None):
    """Move the pages in use to the front of the cache and renumber table and
    refs.  Returns (table, refs, remap, live), new tensors unless given (see
    comp_kv_reserve): remap[p] is page p's new number (-1: free), live[0] the
    number of pages in use."""
    c, shape, device = _cache(k_pages, v_pages)
    rows, width, at_table = _table(table, device)
    pages = shape[0]
    at_refs = _check(refs, _I32, "refs", device, (pages,))
    table_out, to_table = _new(table_out, "table_out", device, (rows, width))
    refs_out, to_refs = _new(refs_out, "refs_out", device, (pages,))
    remap, to_remap = _new(remap, "remap", device, (pages,))
    live, to_live = _new(live, "live", device, (1,))
    _call("comp_kv_compact", ctypes.byref(c), at_table, at_refs, rows, width, to_table, to_refs, to_remap, to_live,
          _stream(device, stream))
    return table_out, refs_out, remap, live


def comp_kv_copy_pages(k_pages, v_pages, src, dst, stream=None):
    """Copy page src[i] of the cache to page dst[i]; the dst are distinct and no src."""
    c, _, device = _cache(k_pages, v_pages)
    n, at_src = _list(src, "src", device)
    at_dst = _check(dst, _I32, "dst", device, (n,))
    _call("comp_kv_copy_pages", ctypes.byref(c), at_src, at_dst, n, _stream(device, stream))
