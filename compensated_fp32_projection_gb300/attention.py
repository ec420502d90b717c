"""Attention and its paged cache, bound to torch tensors.

As in the projections' binding, these functions only marshal arguments into
``libcompfp32.so`` (here by a small C++ module, ``_attn_binding``, because the
smallest calls take less time on the device than checks in Python): every step
runs in the library's CUDA kernels, on the current stream unless one is given,
and nothing waits for the host.  Outputs that are not given are allocated.

Caches are pairs of float16 tensors ``k_pages``, ``v_pages``
[pages, kv_heads, page_size, head_dim]; a page table is an int32 tensor
[rows, width] whose unused entries are -1.
"""
from __future__ import annotations

import os

import torch  # noqa: F401  (the binding's libraries)

from . import _native

_native.load()
if not os.path.exists(_native.BINDING_PATH):
    raise RuntimeError(f"{_native.BINDING_PATH} is missing: build the CUDA library first "
                       "(python -c 'import __graft_entry__ as g; g.build()'); there is no fallback")
from . import _attn_binding as _b  # noqa: E402

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


def comp_attn_f32(q, k, v, cu_q=None, cu_k=None, *, scale=None, causal=True, out=None, lse=None, workspace=None,
                  stream=None):
    """Attention of packed prompts: softmax(scale q k^T) v, all in float32.

    q [tokens, heads, head_dim]; k, v [keys, kv_heads, head_dim]; any token and
    head strides.  Sequence i has the queries cu_q[i]:cu_q[i+1] and the keys
    cu_k[i]:cu_k[i+1] (int32; without them there is one sequence).  causal: the
    last query sees every key of its sequence, each earlier one a key less.
    Magnitudes stay below 65520; float32 values below 1e-4 enter with an absolute
    error of 2^-35 (float16 keys and values are exact).
    scale defaults to head_dim ** -0.5.  lse, if given ([tokens, heads]),
    receives the log-sum-exp of each row.  A row that sees no key gives zeros
    and -inf, as do the tokens beyond the last sequence."""
    return _b.attn(True, q, k, v, cu_q, cu_k, scale, causal, out, lse, workspace, stream)


def comp_attn_f32x16(q, k, v, cu_q=None, cu_k=None, *, scale=None, causal=True, out=None, lse=None, workspace=None,
                     stream=None):
    """comp_attn_f32 with float16 keys and values, which enter the products exactly."""
    return _b.attn(False, q, k, v, cu_q, cu_k, scale, causal, out, lse, workspace, stream)


def comp_kv_append_f32(k, v, k_pages, v_pages, table, start, cu=None, stream=None):
    """Write new tokens' float32 k, v [tokens, kv_heads, head_dim] into the cache
    (rounded to float16, beyond its range to infinities).  Row r's tokens cu[r]:cu[r+1] (without cu: one for each
    row) go to positions start[r], start[r] + 1, ... of its pages."""
    _b.append(k, v, k_pages, v_pages, table, start, cu, stream)


def comp_attn_decode_f32x16(q, k_pages, v_pages, table, lengths, *, shared=0, scale=None, out=None, lse=None,
                            workspace=None, stream=None):
    """Attention of one token for each sequence over the paged cache.

    q [batch, heads, head_dim] float32 (any token and head strides); sequence b
    sees the tokens 0 .. lengths[b] - 1 on the pages that row b of table lists.
    The first `shared` entries are the same in all rows: those pages are read
    once for the whole batch.  lse [batch, heads] as in comp_attn_f32."""
    return _b.decode(q, k_pages, v_pages, table, lengths, shared, scale, out, lse, workspace, stream)


def comp_kv_reserve(table, want, refs, page_size, table_out=None, refs_out=None, left=None, stream=None):
    """Give row r of table the pages that want[r] tokens need (at most as many as
    the table is wide), lowest free page first.  Returns (table, refs, left), new tensors unless given (the inputs
    themselves may be given: updated in place).  left[0] is the number of free
    pages that remain; where it is negative that many are missing and nothing
    was changed."""
    return _b.reserve(table, want, refs, page_size, table_out, refs_out, left, stream)


def comp_kv_fork(k_pages, v_pages, table, lengths, refs, parents, children, table_out=None, lengths_out=None,
                 refs_out=None, left=None, stream=None):
    """Make the empty rows children[i] copies of rows parents[i]: full pages are
    shared, a partly filled last page is copied to a free one.  Returns (table,
    lengths, refs, left), new tensors unless given (see comp_kv_reserve); the
    caches are written in place."""
    return _b.fork(k_pages, v_pages, table, lengths, refs, parents, children, table_out, lengths_out, refs_out, left,
                   stream)


def comp_kv_free(table, lengths, refs, seqs, table_out=None, lengths_out=None, refs_out=None, stream=None):
    """Give back the pages of the rows seqs and empty them.  Returns (table,
    lengths, refs), new tensors unless given (see comp_kv_reserve)."""
    return _b.free(table, lengths, refs, seqs, table_out, lengths_out, refs_out, stream)


def comp_kv_compact(k_pages, v_pages, table, refs, table_out=None, refs_out=None, remap=None, live=None, stream=None):
    """Move the pages in use to the front of the cache and renumber table and
    refs.  Returns (table, refs, remap, live), new tensors unless given (see
    comp_kv_reserve): remap[p] is page p's new number (-1: free), live[0] the
    number of pages in use."""
    return _b.compact(k_pages, v_pages, table, refs, table_out, refs_out, remap, live, stream)


def comp_kv_copy_pages(k_pages, v_pages, src, dst, stream=None):
    """Copy page src[i] of the cache to page dst[i]; the dst are distinct and no src."""
    _b.copy_pages(k_pages, v_pages, src, dst, stream)
