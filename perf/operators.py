"""The attention and cache operators as measured work: inputs, plain forms, exact forms.

Three operators that stand next to the compensated projection:

* ``attn``    attention over whole prompts packed one after the other
              (comp_attn_f32 with FP32 keys and values, comp_attn_f32x16 with
              FP16 ones);
* ``decode``  one token for each sequence of a batch: its key and value go into
              the paged FP16 cache, then it attends to its sequence, whose
              leading pages the whole batch may share (comp_kv_append_f32,
              comp_attn_decode_f32x16);
* ``fork``, ``compact``, ``copy``  maintenance of the cache's pages
              (comp_kv_fork with comp_kv_free, comp_kv_compact,
              comp_kv_copy_pages).

``own`` selects the side: False computes the plain form from elementary torch
operations in 32 bits, True calls the framework.
"""
from __future__ import annotations

import math
import random

import torch

own = False


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def listed():
    return [
        # a short question alone: the smallest call, where only latency counts
        _attn("attn one question", "f32", 1, 19, 19, 16, 16, 64, True),
        # an encoder's batch of questions, packed, both directions visible, at the encoder projection's width (16 x 64)
        _attn("attn encoder batch", "f32", 9, 61, 512, 16, 16, 64, False),
        # prompts of very different lengths prefilled together, grouped heads at the 4096-wide projection (32 x 128)
        _attn("attn ragged prompts", "f16", 24, 23, 2011, 32, 8, 128, True),
        # full FP32 keys and values at the square projection's 4096 rows
        _attn("attn prompt fp32", "f32", 1, 4096, 4096, 32, 32, 128, True),
        # one long document
        _attn("attn long prompt", "f16", 1, 16384, 16384, 32, 8, 128, True),
        # a single user's next token
        _decode("decode one sequence", 1, 0, 777, 777, 16, 32, 8, 128),
        # ordinary serving: nothing shared, lengths far apart
        _decode("decode ragged batch", 48, 0, 129, 6001, 16, 32, 8, 128),
        # questions about one document: the document's pages are shared
        _decode("decode shared prefix", 64, 8192, 5, 397, 32, 16, 16, 64),
        # many samples of one long prompt
        _decode("decode shared long prefix", 256, 32768, 33, 1024, 64, 32, 8, 128),
        # four prompts sampled four times each, the samples given back later
        {"name": "fork and free", "op": "fork", "pages": 2048, "page": 16, "kv_heads": 8, "dim": 128, "parents": 4,
         "children": 16, "longest": 3001},
        # a fragmented cache moved together
        {"name": "compact cache", "op": "compact", "pages": 8192, "page": 32, "kv_heads": 8, "dim": 128, "seqs": 96,
         "live": 0.55},
        # pages duplicated to others, as many as a long prompt has
        {"name": "copy pages", "op": "copy", "pages": 1536, "page": 64, "kv_heads": 8, "dim": 64, "count": 511},
    ]


def _attn(name, kv, seqs, shortest, longest, heads, kv_heads, dim, causal):
    return {"name": name, "op": "attn", "kv": kv, "seqs": seqs, "shortest": shortest, "longest": longest,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "causal": causal}


def _decode(name, batch, shared, shortest, longest, page, heads, kv_heads, dim):
    return {"name": name, "op": "decode", "batch": batch, "shared": shared, "shortest": shortest, "longest": longest,
            "page": page, "heads": heads, "kv_heads": kv_heads, "dim": dim}


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "decode", "decode", "decode", "fork", "compact", "copy"])
    heads, kv_heads, dim = rng.choice([(16, 16, 64), (32, 8, 128), (32, 32, 128), (8, 1, 64), (12, 4, 128), (16, 2, 96),
                                       (28, 4, 128), (10, 5, 80)])
    if op == "attn":
        seqs = _log_int(rng, 1, 40)
        longest = _log_int(rng, 7, 6000 if seqs == 1 else 3000 if seqs < 12 else 1500)
        c = _attn("", rng.choice(["f32", "f16"]), seqs, max(1, longest // rng.choice([1, 2, 5, 30])), longest, heads,
                  kv_heads, dim, rng.random() < 0.7)
    elif op == "decode":
        batch = _log_int(rng, 1, 200)
        page = rng.choice([16, 32, 64, 128])
        shared = rng.choice([0, 0, 1]) * page * _log_int(rng, 1, 20000 // page)
        longest = _log_int(rng, 3, 9000 if batch < 40 else 1500)
        c = _decode("", batch, shared, max(1, longest // rng.choice([1, 2, 5, 30])), longest, page, heads, kv_heads,
                    dim)
    elif op == "fork":
        parents = rng.randint(1, 6)
        c = {"op": "fork", "pages": _log_int(rng, 1200, 6000), "page": rng.choice([16, 32, 64]), "kv_heads": kv_heads,
             "dim": dim, "parents": parents, "children": parents * _log_int(rng, 1, 12),
             "longest": _log_int(rng, 50, 3000)}
    elif op == "compact":
        c = {"op": "compact", "pages": _log_int(rng, 300, 8000), "page": rng.choice([16, 32]), "kv_heads": kv_heads,
             "dim": dim, "seqs": rng.randint(3, 90), "live": round(rng.uniform(0.1, 0.95), 3)}
    else:
        pages = _log_int(rng, 100, 3000)
        c = {"op": "copy", "pages": pages, "page": rng.choice([16, 32, 64]), "kv_heads": kv_heads, "dim": dim,
             "count": rng.randint(1, pages // 2 - 1)}
    c.pop("name", None)
    return c


def _lengths(case):
    """The lengths of a case's sequences: spread over their logarithm, the longest among them."""
    n = case["seqs"] if case["op"] == "attn" else case["batch"]
    rng = random.Random("%d %d %d" % (n, case["shortest"], case["longest"]))
    return [case["longest"]] + [_log_int(rng, case["shortest"], case["longest"]) for _ in range(n - 1)]


def _parent_lengths(case):
    rng = random.Random("%d %d" % (case["parents"], case["longest"]))
    return [case["longest"]] + [rng.randint(1, case["longest"]) for _ in range(case["parents"] - 1)]


def work(case):
    """Each input read once, each output written once; two products of 2 D operations for each visible pair."""
    if case["op"] == "attn":
        h, hk, d, size = case["heads"], case["kv_heads"], case["dim"], 2 if case["kv"] == "f16" else 4
        lens = _lengths(case)
        pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lens)
        return {"bytes": sum(lens) * (2 * 4 * h * d + 2 * size * hk * d + 4 * h), "flops": 4.0 * d * h * pairs}
    if case["op"] == "decode":
        h, hk, d = case["heads"], case["kv_heads"], case["dim"]
        lens = _lengths(case)
        rows = case["shared"] + sum(lens)
        return {"bytes": rows * 4 * hk * d + len(lens) * (2 * 4 * h * d + 8 * hk * d + 4 * h),
                "flops": 4.0 * d * h * sum(case["shared"] + n for n in lens)}
    slot = 2 * 2 * case["kv_heads"] * case["dim"]  # a token's key and value
    if case["op"] == "fork":
        lens = _parent_lengths(case)
        each = case["children"] // case["parents"]
        moved = sum(each * (n % case["page"]) for n in lens)
        listed_pages = sum((1 + 2 * each) * -(-n // case["page"]) for n in lens)
        return {"bytes": 2 * slot * moved + 4 * listed_pages + 3 * 4 * case["pages"], "flops": 0}
    if case["op"] == "compact":
        live = _live(case)
        n = sum(live)
        moved = sum(live[n:])
        return {"bytes": 2 * slot * case["page"] * moved + 4 * 5 * case["pages"], "flops": 0}
    return {"bytes": 2 * slot * case["page"] * case["count"] + 8 * case["count"], "flops": 0}


def _live(case):
    rng = random.Random("%d %g" % (case["pages"], case["live"]))
    return [rng.random() < case["live"] for _ in range(case["pages"])]


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pool(case, g):
    shape = (case["pages"], case["kv_heads"], case["page"], case["dim"])
    return [torch.randn(shape, generator=g, device="cuda", dtype=torch.float16) for _ in range(2)]


def prepare(case, seed):
    import compensated_fp32_projection_gb300 as pkg

    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    s = {"pkg": pkg, "case": case}

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda") * scale

    if case["op"] == "attn":
        lens = _lengths(case)
        total, h, hk, d = sum(lens), case["heads"], case["kv_heads"], case["dim"]
        # one fused projection's output holds q, k and v side by side; queries
        # of this size give scores with a standard deviation of 2
        qkv = normal(total, (h + 2 * hk) * d)
        s["q"] = qkv[:, :h * d].view(total, h, d).mul_(2.0)
        k, v = qkv[:, h * d:(h + hk) * d].view(total, hk, d), qkv[:, (h + hk) * d:].view(total, hk, d)
        s["k"], s["v"] = (k.half(), v.half()) if case["kv"] == "f16" else (k, v)
        s["cu"] = _ints([0] + [sum(lens[:i + 1]) for i in range(len(lens))])
        s["longest"] = max(lens)
        return s
    if case["op"] == "decode":
        lens = _lengths(case)
        b, p, h, hk, d = len(lens), case["page"], case["heads"], case["kv_heads"], case["dim"]
        shared = case["shared"] // p
        own_pages = [-(-n // p) for n in lens]
        width = shared + max(own_pages)
        case = dict(case, pages=shared + sum(own_pages) + 7)
        s["k_pages"], s["v_pages"] = _pool(case, g)
        order = list(range(case["pages"]))
        rng.shuffle(order)
        table, at = [], shared
        for n in own_pages:
            table.append(order[:shared] + order[at:at + n] + [-1] * (width - shared - n))
            at += n
        s["table"] = _ints(table)
        s["lengths"] = _ints([case["shared"] + n for n in lens])
        s["start"] = s["lengths"] - 1
        s["shared"] = shared
        s["q"] = normal(b, h, d, scale=2.0)
        s["k"], s["v"] = normal(b, hk, d), normal(b, hk, d)
        return s
    s["k_pages"], s["v_pages"] = _pool(case, g)
    if case["op"] == "fork":
        lens, p = _parent_lengths(case), case["page"]
        n_pages = [-(-n // p) for n in lens]
        order = rng.sample(range(case["pages"]), sum(n_pages))
        rows, at = [], 0
        width = max(n_pages) + 2
        for n in n_pages:
            rows.append(order[at:at + n] + [-1] * (width - n))
            at += n
        rows += [[-1] * width for _ in range(case["children"] + 3)]
        refs = [0] * case["pages"]
        for i in order:
            refs[i] = 1
        s["table"], s["refs"] = _ints(rows), _ints(refs)
        s["lengths"] = _ints(lens + [0] * (case["children"] + 3))
        s["parents"] = _ints([i % case["parents"] for i in range(case["children"])])
        s["children"] = _ints(rng.sample(range(case["parents"], len(rows)), case["children"]))
        return s
    if case["op"] == "compact":
        live = [i for i, x in enumerate(_live(case)) if x]
        rng.shuffle(live)
        n = -(-len(live) // case["seqs"])
        rows = [live[i * n:(i + 1) * n] for i in range(case["seqs"])]
        refs = [0] * case["pages"]
        for i in live:
            refs[i] = rng.choice([1, 1, 1, 2, 5])
        s["table"], s["refs"] = _ints([r + [-1] * (n + 1 - len(r)) for r in rows]), _ints(refs)
        return s
    both = rng.sample(range(case["pages"]), 2 * case["count"])
    s["src"], s["dst"] = _ints(both[:case["count"]]), _ints(both[case["count"]:])
    return s


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"attn": _plain_attn, "decode": _plain_decode, "fork": _plain_fork, "compact": _plain_compact,
                "copy": _plain_copy}[op](s)
    pkg = s["pkg"]
    if op == "attn":
        lse = torch.empty(s["q"].shape[:2], device="cuda")
        call = pkg.comp_attn_f32 if s["case"]["kv"] == "f32" else pkg.comp_attn_f32x16
        out = call(s["q"], s["k"], s["v"], s["cu"], s["cu"], causal=s["case"]["causal"], lse=lse)
        return {"out": out, "lse": lse}
    if op == "decode":
        lse = torch.empty(s["q"].shape[:2], device="cuda")
        pkg.comp_kv_append_f32(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["start"])
        out = pkg.comp_attn_decode_f32x16(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lengths"],
                                          shared=s["shared"], lse=lse)
        return {"out": out, "lse": lse, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if op == "fork":
        forked = pkg.comp_kv_fork(s["k_pages"], s["v_pages"], s["table"], s["lengths"], s["refs"], s["parents"],
                                  s["children"])
        freed = pkg.comp_kv_free(*forked[:3], s["children"])
        return {"forked": forked, "freed": freed, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if op == "compact":
        table, refs, remap, live = pkg.comp_kv_compact(s["k_pages"], s["v_pages"], s["table"], s["refs"])
        return {"table": table, "refs": refs, "remap": remap, "live": live, "k_pages": s["k_pages"],
                "v_pages": s["v_pages"]}
    pkg.comp_kv_copy_pages(s["k_pages"], s["v_pages"], s["src"], s["dst"])
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _softmax_parts(x):
    """exp(x - max), its sum and log-sum-exp over the last dimension, in place; -inf is masked."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    return x, total, (m + total.log()).squeeze(-1)


def _plain_attn(s):
    """Sequences padded to the longest, all of them in one batched product each."""
    case, q, k, v, cu, n = s["case"], s["q"], s["k"].float(), s["v"].float(), s["cu"].long(), s["longest"]
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    lens = cu[1:] - cu[:-1]
    at = torch.arange(n, device="cuda")
    inside = at < lens[:, None]
    rows = torch.where(inside, cu[:-1, None] + at, torch.zeros_like(at))
    keys = k[rows].permute(0, 2, 3, 1)                                    # [seqs, hk, d, n]
    values = v[rows].permute(0, 2, 1, 3)                                  # [seqs, hk, n, d]
    queries = q[rows].view(-1, n, hk, h // hk, d).permute(0, 2, 3, 1, 4)  # [seqs, hk, group, n, d]
    scores = torch.matmul(queries.reshape(-1, hk, (h // hk) * n, d), keys).mul_(d ** -0.5)
    scores = scores.view(-1, hk, h // hk, n, n)
    hidden = ~inside[:, None, :]
    if case["causal"]:
        hidden = hidden | (at > at[:, None])
    scores.masked_fill_(hidden[:, None, None], -math.inf)
    p, total, lse = _softmax_parts(scores)
    out = torch.matmul(p.view(-1, hk, (h // hk) * n, n), values).view(-1, hk, h // hk, n, d) / total
    out = out.permute(0, 3, 1, 2, 4).reshape(-1, n, h, d)[inside]
    return {"out": out, "lse": lse.permute(0, 3, 1, 2).reshape(-1, n, h)[inside].contiguous()}


def _plain_append(s):
    page = s["case"]["page"]
    at = s["start"].long()
    where = s["table"].long().gather(1, (at // page)[:, None])[:, 0]
    s["k_pages"][where, :, at % page] = s["k"].half()
    s["v_pages"][where, :, at % page] = s["v"].half()


def _plain_decode(s):
    """The shared pages in one product for the whole batch, the others gathered sequence by sequence."""
    _plain_append(s)
    case, q = s["case"], s["q"]
    h, hk, d, shared = case["heads"], case["kv_heads"], case["dim"], case["shared"]
    b = q.shape[0]
    queries = q.view(b, hk, h // hk, d)
    mine = s["table"][:, s["shared"]:].long().clamp_min(0)
    n = mine.shape[1] * case["page"]
    keys = s["k_pages"][mine].float().permute(0, 2, 1, 3, 4).reshape(b, hk, n, d)
    values = s["v_pages"][mine].float().permute(0, 2, 1, 3, 4).reshape(b, hk, n, d)
    scores = torch.matmul(queries, keys.transpose(-1, -2)).mul_(d ** -0.5)
    hidden = torch.arange(n, device="cuda") + shared >= s["lengths"][:, None]
    scores.masked_fill_(hidden[:, None, None], -math.inf)
    values.masked_fill_(hidden[:, None, :, None], 0.0)
    if not shared:
        p, total, lse = _softmax_parts(scores)
        out = torch.matmul(p, values) / total
    else:
        first = s["table"][0, :s["shared"]].long()
        pre_k = s["k_pages"][first].float().permute(1, 0, 2, 3).reshape(hk, shared, d)
        pre_v = s["v_pages"][first].float().permute(1, 0, 2, 3).reshape(hk, shared, d)
        rows = queries.permute(1, 0, 2, 3).reshape(hk, -1, d)
        pre = torch.matmul(rows, pre_k.transpose(-1, -2)).mul_(d ** -0.5).view(hk, b, h // hk, shared)
        every, total, lse = _softmax_parts(torch.cat([pre.permute(1, 0, 2, 3), scores], -1))
        p = every[..., :shared].permute(1, 0, 2, 3).reshape(hk, -1, shared)
        out = torch.matmul(p, pre_v).view(hk, b, h // hk, d).permute(1, 0, 2, 3)
        out = (out + torch.matmul(every[..., shared:], values)) / total
    return {"out": out.reshape(b, h, d), "lse": lse.reshape(b, h), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _count_pages(pages, n):
    """How often each of n pages is named; a name of -1 counts for none."""
    flat = torch.where(pages < 0, torch.full_like(pages, n), pages).reshape(-1)
    return torch.zeros(n + 1, dtype=torch.int32, device="cuda").index_add_(0, flat, torch.ones_like(flat, dtype=torch.int32))[:n]


def _plain_fork(s):
    page, n = s["case"]["page"], s["case"]["pages"]
    parents, children = s["parents"].long(), s["children"].long()
    length = s["lengths"][parents]
    full, rest = (length // page)[:, None], length % page
    need = rest > 0
    free = torch.argsort((s["refs"] != 0).int(), stable=True)
    new = torch.where(need, free[need.long().cumsum(0) - need.long()], torch.full_like(free[:1], -1))
    left = (s["refs"] == 0).sum() - need.sum()
    ok = left >= 0
    rows, col = s["table"][parents], torch.arange(s["table"].shape[1], device="cuda")
    old = torch.where(col < full, rows, torch.full_like(rows, -1))
    child = torch.where((col == full) & need[:, None], new[:, None].int(), old)
    table, lengths = s["table"].clone(), s["lengths"].clone()
    table[children] = torch.where(ok, child, table[children])
    lengths[children] = torch.where(ok, length, lengths[children])
    refs = torch.where(ok, s["refs"] + _count_pages(child.long(), n), s["refs"])
    which = (need & ok).nonzero()[:, 0]
    src, dst = rows.gather(1, full.long())[which, 0].long(), new[which]
    slot = (torch.arange(page, device="cuda") < rest[which][:, None])[:, None, :, None]
    s["k_pages"][dst] = torch.where(slot, s["k_pages"][src], s["k_pages"][dst])
    s["v_pages"][dst] = torch.where(slot, s["v_pages"][src], s["v_pages"][dst])
    after, empty = table.clone(), lengths.clone()
    after[children] = -1
    empty[children] = 0
    freed = (after, empty, refs - _count_pages(table[children].long(), n))
    return {"forked": (table, lengths, refs, left.int().view(1)), "freed": freed, "k_pages": s["k_pages"],
            "v_pages": s["v_pages"]}


def _plain_compact(s):
    refs, table = s["refs"], s["table"].long()
    n = refs.shape[0]
    at = torch.arange(n, device="cuda")
    live = refs > 0
    count = live.sum()
    src, dst = (live & (at >= count)).nonzero()[:, 0], (~live & (at < count)).nonzero()[:, 0]
    remap = torch.where(live, at, torch.full_like(at, -1))
    remap[src] = dst
    s["k_pages"][dst] = s["k_pages"][src]
    s["v_pages"][dst] = s["v_pages"][src]
    moved = torch.where(at < count, refs, torch.zeros_like(refs))
    moved[dst] = refs[src]
    table = torch.where(table < 0, torch.full_like(table, -1), remap[table.clamp_min(0)])
    return {"table": table.int(), "refs": moved, "remap": remap.int(), "live": count.int().view(1),
            "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    s["k_pages"][dst] = s["k_pages"][src]
    s["v_pages"][dst] = s["v_pages"][src]
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


# --------------------------------------------------------------------------
# From the definitions, in 64 bits
# --------------------------------------------------------------------------
def _exact_rows(q, k, v, visible):
    """softmax(q k^T / sqrt d) v of one head: q [n, d], k and v [m, d], visible [n, m] or None for all."""
    x = q.double() @ k.double().T / math.sqrt(q.shape[1])
    if visible is not None:
        x = x.masked_fill(~visible, -math.inf)
    lse = torch.logsumexp(x, -1)
    return torch.exp(x - lse[:, None]) @ v.double(), lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn":
        q, k, v = s["q"], s["k"], s["v"]
        out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
        lse = torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
        group = case["heads"] // case["kv_heads"]
        cu = s["cu"].tolist()
        for a, b in zip(cu, cu[1:]):
            seen = torch.ones(b - a, b - a, dtype=torch.bool, device="cuda").tril() if case["causal"] else None
            for head in range(case["heads"]):
                out[a:b, head], lse[a:b, head] = _exact_rows(q[a:b, head], k[a:b, head // group], v[a:b, head // group],
                                                             seen)
        return {"out": out, "lse": lse}
    if case["op"] == "decode":
        _plain_append(s)
        out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
        group, page = case["heads"] // case["kv_heads"], case["page"]
        for b, n in enumerate(s["lengths"].tolist()):
            pages = s["table"][b, :-(-n // page)].long()
            k = s["k_pages"][pages].permute(1, 0, 2, 3).flatten(1, 2)[:, :n].double()
            v = s["v_pages"][pages].permute(1, 0, 2, 3).flatten(1, 2)[:, :n].double()
            x = s["q"][b].double().view(-1, group, case["dim"]) @ k.transpose(1, 2) / math.sqrt(case["dim"])
            lse[b] = torch.logsumexp(x, -1).flatten()
            out[b] = (torch.softmax(x, -1) @ v).view(-1, case["dim"])
        return {"out": out, "lse": lse, "k_pages": None, "v_pages": None}
    return None  # pages are moved and numbers of pages computed: equal or wrong
