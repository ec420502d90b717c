"""Rotary positions and the 8-bit cache as measured work: inputs, plain forms, exact forms.

Three operators that stand next to attention and its paged cache:

* ``rope``    rotary positions of queries and keys, in halves or interleaved
              pairs, of the whole head or its first part (comp_rope_f32, from a
              table as comp_rope_table makes it);
* ``append``, ``read``  a paged cache of keys and values in 8 bits, with a scale
              for each 16 tokens of a head: new tokens rotated and quantised as
              they are written, and tokens read back (comp_kv8_append_f32,
              comp_kv8_read_f32, comp_kv8_read_f16);
* ``decode``  one token for each sequence, rotated, attending to its sequence in
              that cache (comp_attn_decode_f32x8).

``own`` selects the side: False computes the plain form from elementary torch
operations in 32 bits, True calls the framework.
"""
from __future__ import annotations

import math
import random

import torch

own = False

BLOCK = 16                       # tokens of a head that share a scale
LEAST_SCALE = 2.0 ** -126        # a smaller scale is 0
RECIPROCAL = 1.0 / 127.0         # rounded to 32 bits where it is used


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one user's next token: queries and keys of one projection's output, only latency counts
        _rope("rope one token", 1, 40, 128, 128, False, 5000),
        # prompts of a batch packed together, part of the head, positions in pairs
        _rope("rope packed prompts", 4999, 20, 96, 64, True, 4096),
        # one long document, far positions
        _rope("rope long prompt", 16384, 40, 128, 128, False, 120000),
        # a batch's next tokens: each joins a block that is partly filled
        _append("append next tokens", 64, 1, 1, 2000, 16, 8, 128, 128, False),
        # follow-up turns of very different lengths, beginning anywhere
        _append("append ragged turns", 24, 23, 2011, 777, 32, 8, 128, 64, True),
        # a long document's keys and values at once, no positions in the keys
        _append("append long prompt", 1, 32768, 32768, 0, 64, 8, 128, 0, False),
        # a conversation's past in front of its next turn's packed attention
        _read("read one past", 1, 1333, 1333, 16, 8, 128, "f32"),
        # the pasts of a batch, as 16-bit keys and values
        _read("read ragged pasts", 24, 129, 9001, 32, 16, 64, "f16"),
        # a single user's next token
        _decode("decode one sequence", 1, 777, 777, 16, 32, 8, 128, 128, False),
        # ordinary serving: lengths far apart
        _decode("decode ragged batch", 48, 129, 6001, 16, 32, 8, 128, 128, False),
        # a head for each query head, small heads, part of them rotated
        _decode("decode small heads", 96, 33, 2500, 64, 16, 16, 64, 32, True),
        # long contexts, many query heads on few key heads
        _decode("decode long contexts", 16, 20001, 65536, 128, 64, 4, 128, 0, False),
    ]


def _rope(name, tokens, heads, dim, rot, interleaved, farthest):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "dim": dim, "rot": rot,
            "interleaved": interleaved, "farthest": farthest}


def _append(name, seqs, shortest, longest, past, page, kv_heads, dim, rot, interleaved):
    return {"name": name, "op": "append", "seqs": seqs, "shortest": shortest, "longest": longest, "past": past,
            "page": page, "kv_heads": kv_heads, "dim": dim, "rot": rot, "interleaved": interleaved}


def _read(name, seqs, shortest, longest, page, kv_heads, dim, to):
    return {"name": name, "op": "read", "seqs": seqs, "shortest": shortest, "longest": longest, "page": page,
            "kv_heads": kv_heads, "dim": dim, "to": to}


def _decode(name, seqs, shortest, longest, page, heads, kv_heads, dim, rot, interleaved):
    return {"name": name, "op": "decode", "seqs": seqs, "shortest": shortest, "longest": longest, "page": page,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot, "interleaved": interleaved}


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "read", "decode", "decode", "decode"])
    heads, kv_heads, dim = rng.choice([(16, 16, 64), (32, 8, 128), (32, 32, 128), (8, 1, 64), (12, 4, 128), (16, 2, 96),
                                       (28, 4, 128), (10, 5, 80), (64, 4, 128), (40, 1, 112)])
    rot, interleaved = rng.choice([dim, dim, dim // 2, dim // 4 // 2 * 2]), rng.random() < 0.4
    seqs = _log_int(rng, 1, 100)
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        c = _rope("", _log_int(rng, 1, 80_000_000 // ((heads + kv_heads) * dim)), heads + kv_heads, dim, rot,
                  interleaved, _log_int(rng, 10, 200000))
    elif op == "append":
        longest = _log_int(rng, 1, max(2, 30_000_000 // (seqs * kv_heads * dim)))
        c = _append("", seqs, max(1, longest // rng.choice([1, 2, 5, 30])), longest, rng.choice([0, 1, 9, 300, 1500]),
                    page, kv_heads, dim, rng.choice([0, rot, rot]), interleaved)
    elif op == "read":
        longest = _log_int(rng, 5, 60_000_000 // (seqs * kv_heads * dim))
        c = _read("", seqs, max(1, longest // rng.choice([1, 2, 5, 30])), longest, page, kv_heads, dim,
                  rng.choice(["f32", "f16"]))
    else:
        longest = _log_int(rng, 3, min(70000, 250_000_000 // (seqs * kv_heads * dim)))
        c = _decode("", seqs, max(1, longest // rng.choice([1, 2, 5, 30])), longest, page, heads, kv_heads, dim,
                    rng.choice([0, rot, rot]), interleaved)
    c.pop("name", None)
    return c


def _lengths(case):
    """The lengths of a case's sequences: spread over their logarithm, the longest among them."""
    n = case["seqs"]
    rng = random.Random("%d %d %d" % (n, case["shortest"], case["longest"]))
    return [case["longest"]] + [_log_int(rng, case["shortest"], case["longest"]) for _ in range(n - 1)]


def _pasts(case):
    rng = random.Random("%d past %d" % (case["seqs"], case["past"]))
    return [rng.randint(0, case["past"]) for _ in range(case["seqs"])]


def work(case):
    """Each input read once, each output written once; two products of 2 D operations for each visible pair."""
    d = case["dim"]
    if case["op"] == "rope":
        n = case["tokens"]
        rows = min(n, case["farthest"] + 1)
        return {"bytes": n * (8 * case["heads"] * d + 4) + 4 * rows * case["rot"],
                "flops": 3.0 * n * case["heads"] * case["rot"]}
    hk, lens = case["kv_heads"], _lengths(case)
    slot, scales = 2 * hk * d, 2 * 4 * hk  # a token's codes, a block's scales
    if case["op"] == "append":
        new, back = sum(lens), sum(n + p % BLOCK for n, p in zip(lens, _pasts(case)))
        blocks = sum(-(-(n + p % BLOCK) // BLOCK) for n, p in zip(lens, _pasts(case)))
        return {"bytes": new * (4 * slot + 4 * case["rot"]) + back * (slot + 4 * slot) + 2 * blocks * scales,
                "flops": 6.0 * new * slot}
    if case["op"] == "read":
        size = 4 if case["to"] == "f32" else 2
        return {"bytes": sum(lens) * (1 + size) * slot + sum(-(-n // BLOCK) for n in lens) * scales,
                "flops": 1.0 * sum(lens) * slot}
    h = case["heads"]
    return {"bytes": sum(lens) * slot + sum(-(-n // BLOCK) for n in lens) * scales + len(lens) * (8 * h * d + 4 * h),
            "flops": 4.0 * d * h * sum(lens)}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _angles(positions, rot):
    """The rotary table as a program keeps it: cosine and sine of p / 10000^(2 i / rot)."""
    freq = torch.pow(10000.0, -torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.stack([a.cos(), a.sin()], -1).float()


def _pool8(pages, case, g):
    """A cache that holds keys or values whose channels differ in size, and its scales."""
    hk, page, d = case["kv_heads"], case["page"], case["dim"]
    x = torch.randn(pages, hk, page // BLOCK, BLOCK, d, generator=g, device="cuda")
    x.mul_(torch.randn(hk, 1, 1, d, generator=g, device="cuda").mul_(0.5).exp_())
    scales = x.abs().amax((3, 4)) * RECIPROCAL
    codes = x.mul_(scales.reciprocal()[..., None, None]).round_().to(torch.int8)
    return codes.view(pages, hk, page, d), scales


def prepare(case, seed):
    import compensated_fp32_projection_gb300 as pkg

    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    s = {"pkg": pkg, "case": case, "rope": None}

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda") * scale

    d = case["dim"]
    if case["op"] == "rope":
        n, h = case["tokens"], case["heads"]
        s["rope"] = _angles(case["farthest"] + 1, case["rot"])
        # queries and keys side by side in one projection's output, values behind them
        s["x"] = normal(n, (h + max(1, h // 5)) * d)[:, :h * d].view(n, h, d)
        at, positions = 0, []
        while at < n:  # prompts one after the other, the last token at the farthest position
            m = min(n - at, case["farthest"] + 1)
            first = case["farthest"] + 1 - m if at + m == n else 0
            positions += range(first, first + m)
            at += m
        s["positions"] = _ints(positions)
        return s
    lens, p, hk = _lengths(case), case["page"], case["kv_heads"]
    pasts = _pasts(case) if case["op"] == "append" else [0] * len(lens)
    count = [-(-(a + n) // p) for a, n in zip(pasts, lens)]
    pages = sum(count) + 5
    s["k_pages"], s["k_scales"] = _pool8(pages, case, g)
    s["v_pages"], s["v_scales"] = _pool8(pages, case, g)
    order = rng.sample(range(pages), sum(count))
    table, at = [], 0
    for n in count:
        table.append(order[at:at + n] + [-1] * (max(count) - n))
        at += n
    s["table"] = _ints(table)
    if case["op"] == "decode":
        s["lengths"] = _ints(lens)
        s["q"] = normal(len(lens), case["heads"], d, scale=1.5)
        if case["rot"]:
            s["rope"] = _angles(max(lens), case["rot"])
        return s

    def packed(lens):
        return _ints([0] + [sum(lens[:i + 1]) for i in range(len(lens))])

    s["total"], s["cu"], s["start"] = sum(lens), packed(lens), _ints(pasts)
    if case["op"] == "append":
        if case["rot"]:
            s["rope"] = _angles(max(a + n for a, n in zip(pasts, lens)), case["rot"])
        # keys and values as parts of one projection's output
        kv = normal(s["total"], 2 * hk * d).mul_(normal(2 * hk * d).mul_(0.5).exp_())
        s["k"], s["v"] = kv[:, :hk * d].view(-1, hk, d), kv[:, hk * d:].view(-1, hk, d)
        # what is read back: the new tokens, from the beginning of the blocks that they begin in
        back = [n + a % BLOCK for a, n in zip(pasts, lens)]
        s["back"], s["back_cu"], s["back_start"] = sum(back), packed(back), _ints([a - a % BLOCK for a in pasts])
    return s


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "read": _plain_read, "decode": _plain_decode}[op](s)
    pkg = s["pkg"]
    if op == "rope":
        return pkg.comp_rope_f32(s["x"], s["rope"], s["positions"], interleaved=case["interleaved"])
    cache = (s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
    if op == "append":
        pkg.comp_kv8_append_f32(s["k"], s["v"], *cache, s["table"], s["start"], s["cu"], rope=s["rope"],
                                interleaved=case["interleaved"])
        k, v = pkg.comp_kv8_read_f32(*cache, s["table"], s["back_start"], s["back_cu"], s["back"])
        return {"k": k, "v": v, "k_scales": s["k_scales"], "v_scales": s["v_scales"]}
    if op == "read":
        call = pkg.comp_kv8_read_f32 if case["to"] == "f32" else pkg.comp_kv8_read_f16
        k, v = call(*cache, s["table"], s["start"], s["cu"], s["total"])
        return {"k": k, "v": v}
    lse = torch.empty(s["q"].shape[:2], device="cuda")
    out = pkg.comp_attn_decode_f32x8(s["q"], *cache, s["table"], s["lengths"], rope=s["rope"],
                                     interleaved=case["interleaved"], lse=lse)
    return {"out": out, "lse": lse}


def _rotated(x, angles, interleaved):
    """x [tokens, heads, dim] with its first dimensions rotated by angles [tokens, rot / 2, 2]."""
    rot = 2 * angles.shape[1]
    c, z = angles[:, None, :, 0], angles[:, None, :, 1]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    turned = [a * c - b * z, b * c + a * z]
    turned = torch.stack(turned, -1).flatten(-2) if interleaved else torch.cat(turned, -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rope(s):
    return _rotated(s["x"], s["rope"][s["positions"].long()], s["case"]["interleaved"])


def _tokens(s, cu, start, total):
    """Row, position, page and slot of packed tokens."""
    at = torch.arange(total, device="cuda")
    row = torch.searchsorted(cu, at, right=True) - 1
    position = at - cu[row] + start[row]
    page = s["table"][row, position // s["case"]["page"]].long()
    return row, position, page, position % s["case"]["page"]


def _plain_append(s):
    case = s["case"]
    hk, d = case["kv_heads"], case["dim"]
    row, position, page, slot = _tokens(s, s["cu"], s["start"], s["total"])
    k = s["k"] if s["rope"] is None else _rotated(s["k"], s["rope"][position], case["interleaved"])
    # a token's scale is the one of its block, [pages, kv_heads, blocks of a page]
    blocks = case["page"] // BLOCK
    scale_at = (page[:, None] * hk + torch.arange(hk, device="cuda")) * blocks + (slot // BLOCK)[:, None]
    # where a row begins inside a block, the tokens before stay
    first = s["start"].long()
    begin_page = s["table"].gather(1, (first // case["page"])[:, None])[:, 0].long()
    begin_block = first % case["page"] // BLOCK
    before = (torch.arange(BLOCK, device="cuda") < (first % BLOCK)[:, None])[:, None, :, None]
    for x, codes, scales in ((k, s["k_pages"], s["k_scales"]), (s["v"], s["v_pages"], s["v_scales"])):
        top = torch.zeros_like(scales).view(-1)
        top.scatter_reduce_(0, scale_at.view(-1), x.abs().amax(-1).reshape(-1), "amax")
        fresh = (top * RECIPROCAL).view_as(scales)
        fresh = torch.where(fresh < LEAST_SCALE, torch.zeros_like(fresh), fresh)
        touched = torch.zeros_like(scales, dtype=torch.bool)
        touched.view(-1)[scale_at.view(-1)] = True
        blocked = codes.view(*scales.shape, BLOCK, d)
        was = scales[begin_page, :, begin_block]                      # [rows, hk]
        kept = torch.where((first % BLOCK > 0)[:, None], was, torch.zeros_like(was))
        fresh[begin_page, :, begin_block] = torch.maximum(fresh[begin_page, :, begin_block], kept)
        inverse = torch.where(fresh > 0, fresh.reciprocal(), torch.zeros_like(fresh))
        grown = fresh[begin_page, :, begin_block]
        ratio = torch.where(grown > 0, kept / grown, torch.zeros_like(kept))[..., None, None]
        old = blocked[begin_page, :, begin_block]                     # [rows, hk, 16, d]
        blocked[begin_page, :, begin_block] = torch.where(before, (old * ratio).round().to(torch.int8), old)
        new = (x * inverse.view(-1)[scale_at][..., None]).round().clamp(-127, 127)
        codes[page, :, slot] = new.to(torch.int8)
        scales.copy_(torch.where(touched, fresh, scales))
    k, v = _values(s, s["back_cu"], s["back_start"], s["back"])
    return {"k": k, "v": v, "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def _values(s, cu, start, total):
    row, position, page, slot = _tokens(s, cu, start, total)
    k, v = (codes[page, :, slot] * scales[page, :, slot // BLOCK][..., None]
            for codes, scales in ((s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"])))
    return k, v


def _plain_read(s):
    k, v = _values(s, s["cu"], s["start"], s["total"])
    return {"k": k, "v": v} if s["case"]["to"] == "f32" else {"k": k.half(), "v": v.half()}


def _plain_decode(s):
    """Sequences padded to the longest, all of them in one batched product each."""
    case, q = s["case"], s["q"]
    b, h, d = q.shape
    hk = case["kv_heads"]
    if s["rope"] is not None:
        q = _rotated(q, s["rope"][(s["lengths"] - 1).long()], case["interleaved"])
    pages = s["table"].long().clamp_min(0)
    n = pages.shape[1] * case["page"]

    def values(codes, scales):
        x = codes[pages].view(b, -1, hk, case["page"] // BLOCK, BLOCK, d) * scales[pages][..., None, None]
        return x.transpose(1, 2).reshape(b, hk, n, d)

    scores = torch.matmul(q.view(b, hk, h // hk, d), values(s["k_pages"], s["k_scales"]).transpose(-1, -2))
    scores.mul_(d ** -0.5)
    hidden = torch.arange(n, device="cuda") >= s["lengths"][:, None]
    scores.masked_fill_(hidden[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, values(s["v_pages"], s["v_scales"])) / total
    return {"out": out.reshape(b, h, d), "lse": (top + total.log()).reshape(b, h)}


# --------------------------------------------------------------------------
# From the definitions, in 64 bits
# --------------------------------------------------------------------------
def _exact_turn(x, positions, rot, interleaved):
    """Pairs as complex numbers, each multiplied by e^(i p f)."""
    x = x.double().clone()
    freq = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device="cuda") / rot)
    e = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), positions.double()[:, None] * freq)[:, None]
    i = torch.arange(rot // 2, device="cuda")
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    z = torch.complex(x[..., first], x[..., second]) * e
    x[..., first], x[..., second] = z.real, z.imag
    return x


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_turn(s["x"], s["positions"], case["rot"], case["interleaved"])
    page, d = case["page"], case["dim"]
    if case["op"] == "decode":
        out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
        q = s["q"].double()
        if case["rot"]:
            q = _exact_turn(q, s["lengths"] - 1, case["rot"], case["interleaved"])
        group = case["heads"] // case["kv_heads"]
        for b, n in enumerate(s["lengths"].tolist()):
            at = s["table"][b, :-(-n // page)].long()
            k, v = (_exact_rows(codes, scales, at, n) for codes, scales in ((s["k_pages"], s["k_scales"]),
                                                                           (s["v_pages"], s["v_scales"])))
            x = q[b].view(-1, group, d) @ k.transpose(1, 2) / math.sqrt(d)
            lse[b] = torch.logsumexp(x, -1).flatten()
            out[b] = (torch.softmax(x, -1) @ v).view(-1, d)
        return {"out": out, "lse": lse}
    names = (("k", "k_pages", "k_scales"), ("v", "v_pages", "v_scales"))
    if case["op"] == "read":
        return {name: torch.cat([_exact_rows(s[codes], s[scales], s["table"][b, :-(-n // page)].long(), n)
                                 .transpose(0, 1) for b, n in enumerate(_lengths(case))])
                for name, codes, scales in names}
    if case["seqs"] > 64:
        return None  # block by block below
    # the definition's operations are 32-bit ones: each is computed in 64 and rounded once
    def rounded(x):
        return x.float().double()

    per_step = rounded(torch.tensor(RECIPROCAL, dtype=torch.float64, device="cuda"))
    result = {}
    for name, codes, scales in names:
        x = s[name].double()
        if name == "k" and case["rot"]:
            positions = torch.cat([torch.arange(a, a + n, device="cuda") for a, n in zip(_pasts(case), _lengths(case))])
            e = s["rope"].double()[positions][:, None]
            i = torch.arange(case["rot"] // 2, device="cuda")
            first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + case["rot"] // 2)
            u, w = x[..., first], x[..., second]
            x = x.clone()
            x[..., first] = rounded(rounded(u * e[..., 0]) - rounded(w * e[..., 1]))
            x[..., second] = rounded(rounded(w * e[..., 0]) + rounded(u * e[..., 1]))
        steps, got, at = s[scales].double(), [], 0
        for b, (a, n) in enumerate(zip(_pasts(case), _lengths(case))):
            # the blocks from the one that the row's new tokens begin in, the last one filled up with zeros
            lead, first = a % BLOCK, a // BLOCK
            count = -(-(lead + n) // BLOCK)
            cols = first + torch.arange(count, device="cuda")
            pages, inner = s["table"][b].long()[cols * BLOCK // page], cols % (page // BLOCK)
            tokens = torch.zeros(case["kv_heads"], count * BLOCK, d, dtype=torch.float64, device="cuda")
            tokens[:, lead:lead + n] = x[at:at + n].transpose(0, 1)
            at += n
            tokens = tokens.view(-1, count, BLOCK, d)
            step = rounded(tokens.abs().amax((2, 3)) * per_step)
            past = s[codes].view(*steps.shape, BLOCK, d)[pages[0], :, inner[0], :lead].double()
            if lead:
                step[:, 0] = torch.maximum(step[:, 0], steps[pages[0], :, inner[0]])
            new = torch.round(rounded(tokens * rounded(1 / step)[..., None, None])).clamp(-127, 127)
            if lead:
                shrink = rounded(steps[pages[0], :, inner[0]] / step[:, 0])[:, None, None]
                new[:, 0, :lead] = torch.round(rounded(past * shrink))
            steps[pages, :, inner] = step.transpose(0, 1)
            got.append((new * step[..., None, None]).view(-1, count * BLOCK, d)[:, :lead + n].transpose(0, 1))
        result[name], result[scales] = torch.cat(got), steps
    return result


def _exact_rows(codes, scales, pages, n):
    """The first n tokens on these pages, [kv_heads, n, dim]."""
    _, hk, page, d = codes.shape
    x = codes[pages].double().view(-1, hk, page // BLOCK, BLOCK, d) * scales[pages].double()[..., None, None]
    return x.transpose(0, 1).reshape(hk, -1, d)[:, :n]
