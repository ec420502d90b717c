"""Plain 64-bit attention and cache bookkeeping, and the tolerance of the attention tests.

Tolerance.  The projections hold 4e-6 * sum |x||w| per output (22 bits of the
split operand, FP32 accumulation in chains of 128).  A score is such a product
times the scale, so its error is at most E = 4e-6 * scale * max_j sum_d |q||k|.
That changes each exp(s_j - m) by a factor within exp(+-E), and the numerator
sum_j p_j v_j and the denominator with it; the product with v adds another
4e-6 of sum_j p_j |v_j|, and exp2, the maximum's rounding and the sum stay
below that again.  Hence, with p the exact weights,
    |out - exact| <= (2 (e^E - 1) + 8e-6) * sum_j p_j |v_j| + 1e-30
    |lse - exact| <= E + 4e-6 (1 + |exact|).
Both hold for FP16 and for FP32 keys and values (whose split has 22 bits too).
"""
from __future__ import annotations

import math

import torch

GATE = 4e-6


def exact_rows(q, k, v, visible, scale):
    """(out, lse, out's and lse's tolerance) of one head, in 64 bits on the CPU.

    q [n, d], k and v [m, d], visible [n, m].  Keys that a row does not see are
    left out of its sums, whatever they hold."""
    n, d = q.shape
    out, tol = torch.zeros(n, d, dtype=torch.float64), torch.zeros(n, d, dtype=torch.float64)
    lse, ltol = torch.full((n,), -math.inf, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
    for i in range(n):
        at = visible[i].nonzero()[:, 0]
        if at.numel() == 0:
            continue
        qi, ki, vi = q[i].double(), k[at].double(), v[at].double()
        s = (ki @ qi) * scale
        e = GATE * scale * float((ki.abs() @ qi.abs()).max())
        lse[i] = torch.logsumexp(s, 0)
        p = torch.exp(s - lse[i])
        out[i] = p @ vi
        tol[i] = (2 * math.expm1(min(e, 50.0)) + 2 * GATE) * (p @ vi.abs()) + 1e-30
        ltol[i] = e + GATE * (1 + abs(float(lse[i])))
    return out, lse, tol, ltol


def check_attn(out, lse, q, k, v, cu_q, cu_k, causal, scale):
    """Compare packed attention (any device) with exact_rows, sequence by sequence."""
    out, lse, q, k, v = (x.detach().cpu() for x in (out, lse, q, k, v))
    group = q.shape[1] // k.shape[1]
    for a, b, c, e in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        n, m = b - a, e - c
        seen = torch.ones(n, m, dtype=torch.bool)
        if causal:
            seen = torch.arange(m)[None] <= torch.arange(n)[:, None] + (m - n)
        for h in range(q.shape[1]):
            compare(out[a:b, h], lse[a:b, h], *exact_rows(q[a:b, h], k[c:e, h // group], v[c:e, h // group], seen,
                                                          scale))


def compare(out, lse, x_out, x_lse, tol, ltol):
    assert torch.equal(torch.isneginf(lse), torch.isneginf(x_lse))
    there = ~torch.isneginf(x_lse)
    assert torch.equal(out[~there], torch.zeros_like(out[~there]))
    over = ((out[there].double() - x_out[there]).abs() / tol[there]).nan_to_num(math.inf)
    assert over.numel() == 0 or float(over.max()) <= 1, f"out at {float(over.max()):.3g} of its tolerance"
    over = ((lse[there].double() - x_lse[there]).abs() / ltol[there]).nan_to_num(math.inf)
    assert over.numel() == 0 or float(over.max()) <= 1, f"lse at {float(over.max()):.3g} of its tolerance"


def gather_pages(pages, row, n):
    """The first n tokens of a sequence, [kv_heads, n, dim] (zeros for pages that are not there)."""
    size = pages.shape[2]
    got = [pages[p] if 0 <= p < pages.shape[0] else torch.zeros_like(pages[0]) for p in row[:-(-n // size)]]
    return torch.cat(got, 1)[:, :n] if got else pages[0][:, :0]


def check_decode(out, lse, q, k_pages, v_pages, table, lengths, scale):
    out, lse, q, k_pages, v_pages = (x.detach().cpu() for x in (out, lse, q, k_pages, v_pages))
    group = q.shape[1] // k_pages.shape[1]
    width, size = table.shape[1], k_pages.shape[2]
    for b, (row, n) in enumerate(zip(table.tolist(), lengths.tolist())):
        n = max(0, min(n, width * size))
        k, v = gather_pages(k_pages, row, n), gather_pages(v_pages, row, n)
        for h in range(q.shape[1]):
            compare(out[b, h][None], lse[b, h][None],
                    *exact_rows(q[b, h][None], k[h // group], v[h // group], torch.ones(1, n, dtype=torch.bool),
                                scale))
