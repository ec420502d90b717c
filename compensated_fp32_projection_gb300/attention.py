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


def _stream(t, stream):
    if stream is not None:
        return int(stream) if isinstance(stream, int) else stream.cuda_stream
    return torch.cuda.current_stream(t.device).cuda_stream


def _check(t, dtype, name, like=None, shape=None, dense=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if like is not None and t.device != like.device:
        raise ValueError(f"{name} is on another device")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _heads(t, dtype, name, like=None):
    """A [tokens, heads, head_dim] tensor with any token and head strides."""
    _check(t, dtype, name, like, dense=False)
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    if t.shape[2] > 1 and t.stride(2) != 1 and t.numel() > 0:
        raise ValueError(f"{name} must be contiguous in its last dimension")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _workspace(given, nbytes, like):
    if given is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device) if nbytes > 0 else None
    if given.device != like.device or not given.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return given


def _attn(name, kv_dtype, q, k, v, cu_q, cu_k, scale, causal, out, lse, workspace, stream):
    _heads(q, torch.float32, "q")
    _heads(k, kv_dtype, "k", q)
    _heads(v, kv_dtype, "v", q)
    tokens, heads, dim = q.shape
    if k.shape != v.shape or k.shape[2] != dim:
        raise ValueError("k and v must be [keys, kv_heads, head_dim] with q's head_dim")
    if k.shape[1] == 0 or heads == 0 or heads % k.shape[1]:
        raise ValueError("q's heads must be a multiple of the key/value heads")
    if (cu_q is None) != (cu_k is None):
        raise ValueError("cu_q and cu_k go together")
    n_seq = 1
    if cu_q is not None:
        _check(cu_q, torch.int32, "cu_q", q)
        _check(cu_k, torch.int32, "cu_k", q, cu_q.shape)
        if cu_q.dim() != 1 or cu_q.shape[0] < 1:
            raise ValueError("cu_q and cu_k must be [sequences + 1]")
        n_seq = cu_q.shape[0] - 1
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=torch.float32, device=q.device)
    _heads(out, torch.float32, "out", q)
    if out.shape != q.shape:
        raise ValueError("out must have the shape of q")
    if lse is not None:
        _check(lse, torch.float32, "lse", q, (tokens, heads))
    a = _native.Attn(n_seq, tokens, k.shape[0], heads, k.shape[1], dim, int(bool(causal)),
                     dim ** -0.5 if scale is None else scale, q.stride(0), q.stride(1), k.stride(0), k.stride(1),
                     v.stride(0), v.stride(1), out.stride(0), out.stride(1))
    need = int(_native.load().comp_attn_workspace_bytes(ctypes.byref(a), k.element_size(), k.data_ptr(),
                                                        v.data_ptr()))
    workspace = _workspace(workspace, need, q)
    _native.call(name, ctypes.byref(a), q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(cu_q), _ptr(cu_k),
                 out.data_ptr(), _ptr(lse), _ptr(workspace), 0 if workspace is None else workspace.nbytes,
                 _stream(q, stream))
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
    return _attn("comp_attn_f32", torch.float32, q, k, v, cu_q, cu_k, scale, causal, out, lse, workspace, stream)


def comp_attn_f32x16(q, k, v, cu_q=None, cu_k=None, *, scale=None, causal=True, out=None, lse=None, workspace=None,
                     stream=None):
    """comp_attn_f32 with float16 keys and values, which enter the products exactly."""
    return _attn("comp_attn_f32x16", torch.float16, q, k, v, cu_q, cu_k, scale, causal, out, lse, workspace, stream)


def _cache(k_pages, v_pages):
    _check(k_pages, torch.float16, "k_pages")
    _check(v_pages, torch.float16, "v_pages", k_pages, k_pages.shape)
    if k_pages.dim() != 4:
        raise ValueError("k_pages must be [pages, kv_heads, page_size, head_dim]")
    pages, heads, size, dim = k_pages.shape
    return _native.KvCache(k_pages.data_ptr(), v_pages.data_ptr(), pages, size, heads, dim)


def _table(table, like):
    _check(table, torch.int32, "table", like)
    if table.dim() != 2:
        raise ValueError("table must be [rows, width]")
    return table.shape


def _new(given, like, name):
    if given is None:
        return torch.empty_like(like)
    _check(given, like.dtype, name, like, like.shape)
    return given


def _one(given, like, name):
    if given is None:
        return torch.empty(1, dtype=torch.int32, device=like.device)
    _check(given, torch.int32, name, like, (1,))
    return given


def comp_kv_append_f32(k, v, k_pages, v_pages, table, start, cu=None, stream=None):
    """Write new tokens' float32 k, v [tokens, kv_heads, head_dim] into the cache
    (rounded to float16).  Row r's tokens cu[r]:cu[r+1] (without cu: one for each
    row) go to positions start[r], start[r] + 1, ... of its pages."""
    c = _cache(k_pages, v_pages)
    rows, width = _table(table, k_pages)
    _heads(k, torch.float32, "k", k_pages)
    _heads(v, torch.float32, "v", k_pages)
    if k.shape != v.shape or tuple(k.shape[1:]) != (c.kv_heads, c.head_dim):
        raise ValueError("k and v must be [tokens, kv_heads, head_dim] as the cache has them")
    _check(start, torch.int32, "start", k_pages, (rows,))
    if cu is not None:
        _check(cu, torch.int32, "cu", k_pages, (rows + 1,))
    elif k.shape[0] != rows:
        raise ValueError("without cu there must be one token for each row of table")
    _native.call("comp_kv_append_f32", ctypes.byref(c), k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1),
                 v.stride(0), v.stride(1), k.shape[0], table.data_ptr(), rows, width, _ptr(cu), start.data_ptr(),
                 _stream(k_pages, stream))


def comp_attn_decode_f32x16(q, k_pages, v_pages, table, lengths, *, shared=0, scale=None, out=None, lse=None,
                            workspace=None, stream=None):
    """Attention of one token for each sequence over the paged cache.

    q [batch, heads, head_dim] float32 (any token and head strides); sequence b
    sees the tokens 0 .. lengths[b] - 1 on the pages that row b of table lists.
    The first `shared` entries are the same in all rows: those pages are read
    once for the whole batch.  lse [batch, heads] as in comp_attn_f32."""
    c = _cache(k_pages, v_pages)
    batch, width = _table(table, k_pages)
    _heads(q, torch.float32, "q", k_pages)
    heads, dim = q.shape[1:]
    if q.shape[0] != batch or dim != c.head_dim or c.kv_heads == 0 or heads == 0 or heads % c.kv_heads:
        raise ValueError("q must be [rows of table, a multiple of kv_heads, head_dim]")
    _check(lengths, torch.int32, "lengths", k_pages, (batch,))
    out = torch.empty((batch, heads, dim), dtype=torch.float32, device=q.device) if out is None else out
    _check(out, torch.float32, "out", q, (batch, heads, dim))
    if lse is not None:
        _check(lse, torch.float32, "lse", q, (batch, heads))
    need = int(_native.load().comp_attn_decode_workspace_bytes(ctypes.byref(c), batch, heads, width, int(shared)))
    workspace = _workspace(workspace, need, q)
    _native.call("comp_attn_decode_f32x16", ctypes.byref(c), q.data_ptr(), q.stride(0), q.stride(1), heads,
                 dim ** -0.5 if scale is None else scale, table.data_ptr(), batch, width, lengths.data_ptr(),
                 int(shared), out.data_ptr(), _ptr(lse), _ptr(workspace),
                 0 if workspace is None else workspace.nbytes, _stream(q, stream))
    return out


def comp_kv_reserve(table, want, refs, page_size, table_out=None, refs_out=None, left=None, stream=None):
    """Give row r of table the pages that want[r] tokens need, lowest free page
    first.  Returns (table, refs, left), new tensors unless given (the inputs
    themselves may be given: updated in place).  left[0] is the number of free
    pages that remain; where it is negative that many are missing and nothing
    was changed."""
    rows, width = _table(table, table)
    _check(want, torch.int32, "want", table, (rows,))
    _check(refs, torch.int32, "refs", table, (refs.numel(),))
    table_out, refs_out = _new(table_out, table, "table_out"), _new(refs_out, refs, "refs_out")
    left = _one(left, table, "left")
    _native.call("comp_kv_reserve", refs.numel(), int(page_size), table.data_ptr(), refs.data_ptr(), rows, width,
                 want.data_ptr(), table_out.data_ptr(), refs_out.data_ptr(), left.data_ptr(), _stream(table, stream))
    return table_out, refs_out, left


def comp_kv_fork(k_pages, v_pages, table, lengths, refs, parents, children, table_out=None, lengths_out=None,
                 refs_out=None, left=None, stream=None):
    """Make the empty rows children[i] copies of rows parents[i]: full pages are
    shared, a partly filled last page is copied to a free one.  Returns (table,
    lengths, refs, left), new tensors unless given (see comp_kv_reserve); the
    caches are written in place."""
    c = _cache(k_pages, v_pages)
    rows, width = _table(table, k_pages)
    _check(lengths, torch.int32, "lengths", k_pages, (rows,))
    _check(refs, torch.int32, "refs", k_pages, (c.pages,))
    _check(parents, torch.int32, "parents", k_pages, (parents.numel(),))
    _check(children, torch.int32, "children", k_pages, parents.shape)
    table_out, lengths_out = _new(table_out, table, "table_out"), _new(lengths_out, lengths, "lengths_out")
    refs_out, left = _new(refs_out, refs, "refs_out"), _one(left, table, "left")
    _native.call("comp_kv_fork", ctypes.byref(c), table.data_ptr(), lengths.data_ptr(), refs.data_ptr(), rows, width,
                 parents.data_ptr(), children.data_ptr(), parents.numel(), table_out.data_ptr(),
                 lengths_out.data_ptr(), refs_out.data_ptr(), left.data_ptr(), _stream(k_pages, stream))
    return table_out, lengths_out, refs_out, left


def comp_kv_free(table, lengths, refs, seqs, table_out=None, lengths_out=None, refs_out=None, stream=None):
    """Give back the pages of the rows seqs and empty them.  Returns (table,
    lengths, refs), new tensors unless given (see comp_kv_reserve)."""
    rows, width = _table(table, table)
    _check(lengths, torch.int32, "lengths", table, (rows,))
    _check(refs, torch.int32, "refs", table, (refs.numel(),))
    _check(seqs, torch.int32, "seqs", table, (seqs.numel(),))
    table_out, lengths_out = _new(table_out, table, "table_out"), _new(lengths_out, lengths, "lengths_out")
    refs_out = _new(refs_out, refs, "refs_out")
    _native.call("comp_kv_free", refs.numel(), table.data_ptr(), lengths.data_ptr(), refs.data_ptr(), rows, width,
                 seqs.data_ptr(), seqs.numel(), table_out.data_ptr(), lengths_out.data_ptr(), refs_out.data_ptr(),
                 _stream(table, stream))
    return table_out, lengths_out, refs_out


def comp_kv_compact(k_pages, v_pages, table, refs, table_out=None, refs_out=None, remap=None, live=None, stream=None):
    """Move the pages in use to the front of the cache and renumber table and
    refs.  Returns (table, refs, remap, live), new tensors unless given (see
    comp_kv_reserve): remap[p] is page p's new number (-1: free), live[0] the
    number of pages in use."""
    c = _cache(k_pages, v_pages)
    rows, width = _table(table, k_pages)
    _check(refs, torch.int32, "refs", k_pages, (c.pages,))
    table_out, refs_out = _new(table_out, table, "table_out"), _new(refs_out, refs, "refs_out")
    remap, live = _new(remap, refs, "remap"), _one(live, table, "live")
    _native.call("comp_kv_compact", ctypes.byref(c), table.data_ptr(), refs.data_ptr(), rows, width,
                 table_out.data_ptr(), refs_out.data_ptr(), remap.data_ptr(), live.data_ptr(),
                 _stream(k_pages, stream))
    return table_out, refs_out, remap, live


def comp_kv_copy_pages(k_pages, v_pages, src, dst, stream=None):
    """Copy page src[i] of the cache to page dst[i]; the dst are distinct and no src."""
    c = _cache(k_pages, v_pages)
    _check(src, torch.int32, "src", k_pages, (src.numel(),))
    _check(dst, torch.int32, "dst", k_pages, src.shape)
    _native.call("comp_kv_copy_pages", ctypes.byref(c), src.data_ptr(), dst.data_ptr(), src.numel(),
                 _stream(k_pages, stream))
