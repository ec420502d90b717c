"""Plain loops for rotary positions and the 8-bit cache, in the calls' own 32-bit operations (CPU tensors).

Every operation of the rotation and of the quantisation is a binary32 one that is
rounded to nearest even, and torch's elementwise operations on the CPU are those,
one at a time: results are compared bit for bit.
"""
from __future__ import annotations

import math

import torch

from attn_check import compare, exact_rows, gather_pages

BLOCK = 16


def table(positions, rot, base=10000.0, factor=1.0, context=0.0, low=1.0, high=32.0, magnitude=1.0, first=0):
    """(table in 64 bits, the angles) from the formulas."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = base ** (-2 * i / rot)
    g = torch.zeros_like(f)
    if context > 0:
        g = ((context * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
    a = f * (g + (1 - g) / factor)
    angle = (first + torch.arange(positions, dtype=torch.float64))[:, None] * a
    return magnitude * torch.stack([angle.cos(), angle.sin()], -1), angle


def rotate(x, angles, positions, interleaved, inverse=False):
    """x [tokens, heads, dim] float32, angles [n, rot / 2, 2]; a position that is not there: NaN."""
    rot = 2 * angles.shape[1]
    out = x.clone()
    there = (positions >= 0) & (positions < angles.shape[0])
    cs = angles[positions.clamp(0, max(angles.shape[0] - 1, 0))] if angles.shape[0] else torch.zeros(
        len(positions), rot // 2, 2)
    cs = torch.where(there[:, None, None], cs, torch.full_like(cs, math.nan))[:, None]
    c, s = cs[..., 0], -cs[..., 1] if inverse else cs[..., 1]
    i = torch.arange(rot // 2)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    a, b = x[..., one], x[..., two]
    out[..., one] = a * c - b * s
    out[..., two] = b * c + a * s
    return out


class Cache:
    """An 8-bit cache's keys or values."""

    def __init__(self, codes, scales):
        self.codes, self.scales = codes.cpu().clone(), scales.cpu().clone()

    def write(self, x, row, start):
        """x [n, heads, dim] to positions start ... of the sequence on these pages."""
        pages, heads, size, _ = self.codes.shape
        for block in range(start // BLOCK, -(-(start + len(x)) // BLOCK) if len(x) else start // BLOCK):
            at = block * BLOCK
            if at < 0 or at // size >= len(row) or not 0 <= row[at // size] < pages:
                continue
            page, slot = row[at // size], at % size
            first, last = max(start, at), min(start + len(x), at + BLOCK)
            for h in range(heads):
                self.join(x[first - start:last - start, h], page, h, slot, first - at)

    def join(self, x, page, h, slot, lead):
        block = slot // BLOCK
        old = self.scales[page, h, block] if lead else torch.tensor(0.0)
        finite = x.isfinite()
        top = torch.where(finite, x.abs(), torch.zeros_like(x)).max()
        scale = top * torch.tensor(1 / 127, dtype=torch.float32)
        if float(scale) < 2.0 ** -126:
            scale = torch.tensor(0.0)
        scale = torch.maximum(scale, old.abs())
        before = self.codes[page, h, slot:slot + lead]
        if float(scale) > 0:
            grown = (before.float() * (old.abs() / scale)).round().to(torch.int8)
            new = (x * (torch.ones(()) / scale)).nan_to_num(0.0).round().clamp(-127, 127)
        else:
            grown, new = torch.zeros_like(before), torch.zeros_like(x)
        self.codes[page, h, slot:slot + lead] = torch.where(before == -128, before, grown)
        new = torch.where(finite, new, torch.full_like(new, -128.0)).to(torch.int8)
        self.codes[page, h, slot + lead:slot + lead + len(x)] = new
        odd = bool((~finite).any()) or math.copysign(1.0, float(old)) < 0
        self.scales[page, h, block] = -scale if odd else scale

    def values(self, dtype=torch.float32):
        """What the codes stand for, [pages, heads, size, dim]."""
        x = self.codes.to(dtype) * self.scales.abs().to(dtype).repeat_interleave(BLOCK, 2)[..., None]
        return torch.where(self.codes == -128, torch.full_like(x, math.nan), x)


def append(k_cache, v_cache, k, v, table, start, cu=None, angles=None, interleaved=False):
    k, v = k.cpu(), v.cpu()
    cu = list(range(len(table) + 1)) if cu is None else cu
    for row, s, a, b in zip(table, start, cu, cu[1:]):
        x = k[a:b]
        if angles is not None:
            x = rotate(x, angles, s + torch.arange(b - a), interleaved)
        k_cache.write(x, row, s)
        v_cache.write(v[a:b], row, s)


def read(values, table, start, cu, total):
    """Packed tokens of values [pages, heads, size, dim]; zeros where there is no page."""
    pages, heads, size, dim = values.shape
    out = torch.zeros(total, heads, dim, dtype=values.dtype)
    for row, s, a, b in zip(table, start, cu, cu[1:]):
        for t in range(a, b):
            at = s + t - a
            if at >= 0 and at // size < len(row) and 0 <= row[at // size] < pages:
                out[t] = values[row[at // size], :, at % size]
    return out


def check_rows(out, lse, q, k, v, scale):
    """One row (each [1, dim] and [1]) against 64-bit sums over k, v [n, dim].

    To the tolerance of attn_check, which is relative to sum_j p_j |v_j|, comes what
    the weights lose at their lower end: 2^14 p enters as two binary16 values of
    which the second ends at 2^-24, so p is off by up to 2^-39 however small it is.
    A code of 0 under the one key that has the weight leaves only such weights in a
    component: 2^-39 sum_j |v_j|."""
    x_out, x_lse, tol, ltol = exact_rows(q, k, v, torch.ones(1, len(k), dtype=torch.bool), scale)
    compare(out, lse, x_out, x_lse, tol + 2.0 ** -39 * v.double().abs().sum(0), ltol)


def check_decode(out, lse, q, k_pages, v_pages, table, lengths, scale):
    """Every row of a decode call against 64-bit sums over the pages' values."""
    out, lse, q = (x.detach().cpu() for x in (out, lse, q))
    group = q.shape[1] // k_pages.shape[1]
    width, size = table.shape[1], k_pages.shape[2]
    for b, (row, n) in enumerate(zip(table.tolist(), lengths.tolist())):
        n = max(0, min(n, width * size))
        k, v = gather_pages(k_pages, row, n), gather_pages(v_pages, row, n)
        for h in range(q.shape[1]):
            check_rows(out[b, h][None], lse[b, h][None], q[b, h][None], k[h // group], v[h // group], scale)
