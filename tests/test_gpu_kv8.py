"""The 8-bit cache: written bit for bit as plain 32-bit loops write it, read back, attended to, its pages moved."""
import math
import random

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import kv8_check as plain  # noqa: E402


@pytest.fixture(scope="module")
def pkg():
    import __graft_entry__

    __graft_entry__.build()
    import compensated_fp32_projection_gb300 as p

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return p


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def pool(pages, heads, page, dim, seed=0, spread=0.5):
    """A cache of random codes: (k_pages, v_pages, k_scales, v_scales)."""
    g = torch.Generator().manual_seed(seed)
    codes = [torch.randint(-127, 128, (pages, heads, page, dim), generator=g, dtype=torch.int8) for _ in range(2)]
    scales = [0.02 * (spread * torch.randn(pages, heads, page // 16, generator=g)).exp() for _ in range(2)]
    return [t.cuda() for t in codes + scales]


def plain_of(cache):
    return plain.Cache(cache[0], cache[2]), plain.Cache(cache[1], cache[3])


def same(cache, k, v):
    return all(torch.equal(a.cpu().view(torch.int8 if a.dtype == torch.int8 else torch.int32),
                           b.view(torch.int8 if b.dtype == torch.int8 else torch.int32))
               for a, b in zip(cache, (k.codes, v.codes, k.scales, v.scales)))


def equal(a, b):
    a, b = a.cpu(), b.cpu()
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(0.0), b.nan_to_num(0.0))


def rows_of(lens, page, pages, seed):
    order = random.Random(seed).sample(range(pages), pages)
    table, at, width = [], 0, max(1, max(-(-n // page) for n in lens))
    for n in lens:
        need = -(-n // page)
        table.append(order[at:at + need] + [-1] * (width - need))
        at += need
    return table


SHAPES = [(1, 16, 16), (2, 32, 64), (3, 64, 80), (2, 128, 128), (5, 16, 48), (1, 32, 96), (2, 64, 112), (8, 16, 32)]


@pytest.mark.parametrize("heads,page,dim", SHAPES)
@pytest.mark.parametrize("rot,interleaved", [(0, False), (16, True), (8, False), (1, False), (1, True)],
                         ids=["as they are", "part interleaved", "part in halves", "halves", "interleaved"])
def test_append_and_read(pkg, heads, page, dim, rot, interleaved):
    rot = dim if rot == 1 else min(rot, dim)
    g = torch.Generator().manual_seed(dim + page)
    cache = pool(60, heads, page, dim, seed=dim)
    k_plain, v_plain = plain_of(cache)
    past = [0, 5, 16, 31, 100, 7, 0, 50]
    new = [40, 1, 16, 3, 0, 130, 1, 15]
    table = rows_of([a + n for a, n in zip(past, new)], page, 60, seed=1)
    cu = [sum(new[:i]) for i in range(len(new) + 1)]
    total = cu[-1] + 5                       # five tokens behind the last sequence
    kv = torch.randn(total, 2 * heads, dim + 4, generator=g) * (torch.randn(dim + 4, generator=g)).exp()
    angles = pkg.comp_rope_table(300, rot) if rot else None
    for off in (0, 3):                       # aligned and not
        x = kv.cuda()[..., off:off + dim]
        k, v = x[:, :heads], x[:, heads:]
        pkg.comp_kv8_append_f32(k, v, *cache, ints(table), ints(past), ints(cu), rope=angles, interleaved=interleaved)
        plain.append(k_plain, v_plain, k, v, table, past, cu, None if angles is None else angles.cpu(), interleaved)
        assert same(cache, k_plain, v_plain)
    # and back: from positions of its own for each row
    start, count = [0, 3, 16, 0, 20, 130, 1, 64], [40, 3, 16, 34, 80, 7, 0, 1]
    cu = [sum(count[:i]) for i in range(len(count) + 1)]
    k, v = pkg.comp_kv8_read_f32(*cache, ints(table), ints(start), ints(cu), cu[-1] + 3)
    assert equal(k, plain.read(k_plain.values(), table, start, cu, cu[-1] + 3))
    assert equal(v, plain.read(v_plain.values(), table, start, cu, cu[-1] + 3))
    wide = torch.full((2, cu[-1] + 3, heads + 1, dim + 4), 7.0, dtype=torch.float16, device="cuda")
    for first in (0, 1):                     # aligned and not
        k16, v16 = wide[0, :, :heads, first:first + dim], wide[1, :, 1:, first:first + dim]
        got = pkg.comp_kv8_read_f16(*cache, ints(table), ints(start), ints(cu), cu[-1] + 3, k=k16, v=v16)
        assert got[0] is k16 and got[1] is v16
        assert equal(k16, k.half()) and equal(v16, v.half())
        assert (wide[0, :, heads] == 7).all() and (wide[1, :, 0] == 7).all() and (wide[:, :, :, dim + 1:] == 7).all()
    assert same(cache, k_plain, v_plain)


@pytest.mark.parametrize("dim", [64, 128])
def test_one_token_at_a_time(pkg, dim):
    """A block that grows: what stands in it is rounded again where the scale grows, and is never far off."""
    g = torch.Generator().manual_seed(dim)
    heads, page, rows = 2, 16, 3
    cache = pool(8, heads, page, dim)
    k_plain, v_plain = plain_of(cache)
    table = [[4, 1], [0, 7], [3, 5]]
    xs = torch.randn(20, rows, 2 * heads, dim, generator=g)
    grown = torch.zeros(rows, 2 * heads)
    for t, x in enumerate(xs):
        before = [c.scales.abs().clone() for c in (k_plain, v_plain)]
        pkg.comp_kv8_append_f32(x[:, :heads].cuda(), x[:, heads:].cuda(), *cache, ints(table), ints([t] * rows))
        plain.append(k_plain, v_plain, x[:, :heads], x[:, heads:], table, [t] * rows)
        assert same(cache, k_plain, v_plain)
        if t < 16:
            pages = [r[0] for r in table]
            new = torch.cat([c.scales.abs()[pages, :, 0] > b[pages, :, 0] for c, b in
                             zip((k_plain, v_plain), before)], 1)
            grown = torch.where(torch.tensor(t == 0), torch.zeros_like(grown), grown + new)
    for values, cache_of, first in ((xs[:, :, :heads], k_plain, 0), (xs[:, :, heads:], v_plain, heads)):
        got = cache_of.values()
        for r, row in enumerate(table):
            for h in range(heads):
                scale = float(cache_of.scales[row[0], h, 0].abs())
                off = (got[row[0], h, :16] - values[:16, r, h]).abs().max()
                # half a step for the first rounding and for each growth, and what 32 bits add to each
                assert float(off) <= scale * (0.5 + 0.5 * float(grown[r, first + h])) * (1 + 2.0 ** -14)


def test_append_twice_is_append_once(pkg):
    x = torch.randn(30, 4, 64, generator=torch.Generator().manual_seed(0)).cuda()
    cache = pool(5, 2, 16, 64)
    call = lambda: pkg.comp_kv8_append_f32(x[:, :2], x[:, 2:], *cache, ints([[3, 0, 2]]), ints([9]),  # noqa: E731
                                           ints([0, 30]))
    call()
    once = [t.clone() for t in cache]
    call()
    assert all(torch.equal(a, b) for a, b in zip(cache, once))


def test_values_of_any_kind(pkg):
    """NaN, infinities, zeros, the smallest and the largest numbers: each costs itself at most."""
    heads, page, dim = 1, 16, 32
    cache = pool(12, heads, page, dim)
    k_plain, v_plain = plain_of(cache)
    g = torch.Generator().manual_seed(0)
    x = torch.randn(12 * 16, 2, dim, generator=g)
    x[16:32] = 0
    x[32:48] *= 1e-44
    x[48:64] *= 2.0 ** -119
    x[64:80] = x[64:80].sign() * 3.4028235e38
    x[80, 0, 3], x[81, 1, 31], x[82, 0, 0] = math.nan, math.inf, -math.inf
    x[96:112] = math.nan
    x[112:128] = 0
    x[113, :, 5] = math.inf
    x[128:144] *= 1e30
    x[129, 0, 1] = math.nan
    table, cu = [list(range(11, -1, -1))], [0, 192]
    pkg.comp_kv8_append_f32(x[:, :1].cuda(), x[:, 1:].cuda(), *cache, ints(table), ints([0]), ints(cu))
    plain.append(k_plain, v_plain, x[:, :1], x[:, 1:], table, [0], cu)
    assert same(cache, k_plain, v_plain)
    k, v = pkg.comp_kv8_read_f32(*cache, ints(table), ints([0]), ints(cu), 192)
    assert torch.equal(k.isnan().cpu(), ~x[:, :1].isfinite()) and torch.equal(v.isnan().cpu(), ~x[:, 1:].isfinite())
    for got, want in ((k.cpu(), x[:, :1]), (v.cpu(), x[:, 1:])):
        for b in range(12):
            of = slice(16 * b, 16 * b + 16)
            fine = want[of].isfinite()
            top = want[of][fine].abs().max() if fine.any() else torch.tensor(0.0)
            off = (got[of] - want[of])[fine].double().abs()
            # half a step, and 2^-21 of 127 steps for the operations; below 2^-126 of a step nothing is kept
            assert not off.numel() or float(off.max()) <= float(top) * (0.5 / 127 + 2.0 ** -20) + 127 * 2.0 ** -126
    # the block with a NaN grows: the code stays, its neighbours are rounded again
    y = torch.full((1, 2, dim), 50.0)
    for x_new, start in ((y, 9 * 16 + 3), (y * 2, 6 * 16 + 1), (y, 8 * 16 + 5)):
        pkg.comp_kv8_append_f32(x_new[:, :1].cuda(), x_new[:, 1:].cuda(), *cache, ints(table), ints([start]))
        plain.append(k_plain, v_plain, x_new[:, :1], x_new[:, 1:], table, [start])
        assert same(cache, k_plain, v_plain)


def test_a_block_that_nothing_was_written_to(pkg):
    """Tokens that begin inside a block whose scale was never set: it does not reach them."""
    for junk in (math.nan, math.inf, -math.inf):
        cache = pool(3, 2, 32, 64)
        for t in cache[2:]:
            t.fill_(junk)
        x = torch.randn(20, 4, 64, generator=torch.Generator().manual_seed(0)).cuda()
        table, start, cu = ints([[2, 1]]), ints([21]), ints([0, 20])
        pkg.comp_kv8_append_f32(x[:, :2], x[:, 2:], *cache, table, start, cu)
        k, v = pkg.comp_kv8_read_f32(*cache, table, start, cu, 20)
        for got, want, scales in ((k, x[:, :2], cache[2]), (v, x[:, 2:], cache[3])):
            step = torch.cat([scales[2, :, 1].expand(11, 2), scales[1, :, 0].expand(9, 2)]).abs()
            # half a step, and 2^-21 of 127 steps for the operations
            assert ((got - want).abs() <= step[..., None] * (0.5 + 127 * 2.0 ** -21)).all()


def test_pages_that_are_not_there(pkg):
    heads, page, dim = 2, 32, 64
    cache = pool(6, heads, page, dim)
    k_plain, v_plain = plain_of(cache)
    table = [[2, -1, 6, 0], [7, 1, -9, 3], [-1, -1, -1, -1], [5, 2 ** 31 - 1, 4, -2 ** 31]]
    start, new = [10, 20, 0, -40], [130, 90, 64, 200]     # beyond the width, before the beginning
    cu = [sum(new[:i]) for i in range(5)]
    x = torch.randn(cu[-1], 4, dim, generator=torch.Generator().manual_seed(0))
    pkg.comp_kv8_append_f32(x[:, :2].cuda(), x[:, 2:].cuda(), *cache, ints(table), ints(start), ints(cu))
    plain.append(k_plain, v_plain, x[:, :2], x[:, 2:], table, start, cu)
    assert same(cache, k_plain, v_plain)
    k, v = pkg.comp_kv8_read_f32(*cache, ints(table), ints(start), ints(cu), cu[-1])
    assert equal(k, plain.read(k_plain.values(), table, start, cu, cu[-1]))
    assert equal(v, plain.read(v_plain.values(), table, start, cu, cu[-1]))
    # the far end of positions
    for far in (2 ** 31 - 1, -2 ** 31):
        pkg.comp_kv8_append_f32(x[:4, :2].cuda(), x[:4, 2:].cuda(), *cache, ints(table), ints([far] * 4))
        k, v = pkg.comp_kv8_read_f32(*cache, ints(table), ints([far] * 4), None, 4)
        assert not k.any() and not v.any() and same(cache, k_plain, v_plain)


def test_bad_sequence_starts_stay_inside(pkg):
    """cu that does not ascend, or leaves the tokens: every access stays inside the arrays."""
    cache = pool(6, 1, 16, 32)
    x = torch.zeros(20, 1, 32, device="cuda")
    table, start = ints([[0, 1], [2, 3], [4, 5]]), ints([0, 0, 0])
    for cu in ([0, 50, 7, 20], [5, 3, 2, 1], [-7, 3, 30, 90], [20, 20, 20, 20], [0, -2 ** 31, 2 ** 31 - 1, 4]):
        pkg.comp_kv8_append_f32(x, x, *cache, table, start, ints(cu))
        k, v = pkg.comp_kv8_read_f32(*cache, table, start, ints(cu), 20)
        torch.cuda.synchronize()
        assert not k.isnan().any()


def test_many_rows(pkg):
    """More rows than a warp searches at once, empty ones among them."""
    rng = random.Random(5)
    rows = 2500
    new = [rng.choice([0, 0, 1, 1, 2, 17]) for _ in range(rows)]
    past = [rng.choice([0, 7, 15]) for _ in range(rows)]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    table = rows_of([a + n for a, n in zip(past, new)], 16, 5200, seed=2)
    cache = pool(5200, 1, 16, 16)
    k_plain, v_plain = plain_of(cache)
    x = torch.randn(cu[-1], 2, 16, generator=torch.Generator().manual_seed(0))
    pkg.comp_kv8_append_f32(x[:, :1].cuda(), x[:, 1:].cuda(), *cache, ints(table), ints(past), ints(cu))
    plain.append(k_plain, v_plain, x[:, :1], x[:, 1:], table, past, cu)
    assert same(cache, k_plain, v_plain)
    k, v = pkg.comp_kv8_read_f32(*cache, ints(table), ints(past), ints(cu), cu[-1])
    assert equal(k, plain.read(k_plain.values(), table, past, cu, cu[-1]))


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def check(pkg, q, cache, table, lengths, angles=None, interleaved=False, scale=None, **kw):
    """Decode against 64-bit sums over the cache's values."""
    lse = torch.full(q.shape[:2], 9.0, device="cuda")
    out = pkg.comp_attn_decode_f32x8(q, *cache, table, lengths, rope=angles, interleaved=interleaved, scale=scale,
                                     lse=lse, **kw)
    turned = q.cpu()
    if angles is not None:
        limit = table.shape[1] * cache[0].shape[2]
        at = (lengths.cpu().long().clamp(0, limit) - 1).clamp_min(0)
        turned = plain.rotate(turned, angles.cpu(), at, interleaved)
    k, v = (c.values(torch.float64) for c in plain_of(cache))
    plain.check_decode(out, lse, turned, k, v, table.cpu(), lengths.cpu(),
                       q.shape[2] ** -0.5 if scale is None else scale)
    return out, lse


HEADS = [(1, 1), (4, 1), (8, 2), (9, 1), (16, 1), (17, 1), (6, 3), (40, 2)]


@pytest.mark.parametrize("heads,kv_heads", HEADS)
@pytest.mark.parametrize("page,dim", [(16, 128), (32, 64), (64, 16), (128, 96), (16, 48), (32, 112)])
def test_decode(pkg, heads, kv_heads, page, dim):
    lens = [1, 0, 15, 16, 17, 33, 130, 77]
    cache = pool(60, kv_heads, page, dim, seed=heads)
    table = ints(rows_of(lens, page, 60, seed=3))
    q = torch.randn(len(lens), heads, dim, generator=torch.Generator().manual_seed(dim)).cuda()
    check(pkg, q, cache, table, ints(lens))
    wide = torch.randn(len(lens), heads + 1, dim + 3, device="cuda")
    check(pkg, wide[:, 1:, 2:-1], cache, table, ints(lens), scale=0.3)     # strided, at any address
    flat = torch.empty(len(lens) * heads * dim + 1, device="cuda")[1:]
    out, _ = check(pkg, q, cache, table, ints(lens), out=flat.view(len(lens), heads, dim))
    assert out.data_ptr() == flat.data_ptr()


@pytest.mark.parametrize("rot,interleaved", [(64, False), (64, True), (16, False), (20, False), (20, True), (2, True)])
@pytest.mark.parametrize("dim", [64, 128])
def test_decode_rotates_queries(pkg, dim, rot, interleaved):
    lens = [1, 40, 0, 133]
    cache = pool(20, 2, 32, dim)
    table = ints(rows_of(lens, 32, 20, seed=3))
    angles = pkg.comp_rope_table(133, rot, magnitude=1.1)
    q = torch.randn(4, 6, dim, generator=torch.Generator().manual_seed(dim)).cuda()
    check(pkg, q, cache, table, ints(lens), angles, interleaved)
    wide = torch.randn(4, 6, dim + 3, device="cuda")[..., 1:-2]
    check(pkg, wide, cache, table, ints(lens), angles, interleaved)
    # a position that the table does not have
    out = pkg.comp_attn_decode_f32x8(q, *cache, table, ints(lens), rope=angles[:132], interleaved=interleaved)
    assert out[3].isnan().all() and not out[:3].isnan().any()


def test_decode_lengths_and_pages_out_of_range(pkg):
    cache = pool(5, 2, 16, 64)
    table = [[0, -1, 3], [5, 2, -7], [1, 4, 2 ** 31 - 1], [2, 2, 2], [4, 3, 1], [-1, -1, -1]]
    lens = [40, 48, 48, 1000, -5, 20]
    q = torch.randn(6, 4, 64, generator=torch.Generator().manual_seed(0)).cuda()
    check(pkg, q, cache, ints(table), ints(lens))
    # no pages in the table, no rows, no batch
    out, lse = check(pkg, q, cache, torch.zeros(6, 0, dtype=torch.int32, device="cuda"), ints([3] * 6))
    assert not out.any() and torch.isneginf(lse).all()
    assert pkg.comp_attn_decode_f32x8(q[:0], *cache, ints([]).view(0, 3), ints([])).shape == (0, 4, 64)


def test_decode_scales_of_any_size(pkg):
    """Blocks of very different scales, zero ones among them."""
    cache = pool(12, 2, 32, 64, spread=6.0)
    cache[2][3, 0, 1] = cache[3][2, 1, 0] = 0.0
    cache[3].mul_(1e20)
    lens = [32 * 3, 70, 5]
    table = ints([[3, 2, 1], [2, 0, 4], [6, -1, -1]])
    q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(0)).cuda()
    check(pkg, q, cache, table, ints(lens), scale=0.02)
    cache[3].mul_(1e-30)
    check(pkg, q, cache, table, ints(lens), scale=0.02)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("heads", [4, 12])
def test_decode_what_lies_behind_the_end(pkg, heads, page):
    """Blocks that no token has been written to may hold anything, NaN for a scale too."""
    dim = 64
    cache = pool(30, 1, page, dim)
    lens = [1, 16, 17, 32, 33, 48, 49, 64, 65]
    table = rows_of(lens, page, 29, seed=1)
    table = [r + [29, 29] for r in table]
    want = pkg.comp_attn_decode_f32x8(torch.ones(9, heads, dim, device="cuda"), *cache, ints(table), ints(lens))
    for r, n in zip(table, lens):
        for block in range(-(-n // 16), len(r) * page // 16):
            p = r[block * 16 // page]
            for t in cache[2:]:
                t[p, :, block % (page // 16)] = math.nan
    got = pkg.comp_attn_decode_f32x8(torch.ones(9, heads, dim, device="cuda"), *cache, ints(table), ints(lens))
    assert torch.equal(got, want) and not got.isnan().any()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads", [4, 12])
def test_decode_with_codes_that_are_not_numbers(pkg, dim, heads):
    """They reach the rows that see them, and only those."""
    cache = pool(4, 1, 32, dim)
    table, lens = ints([[0, 1], [2, 3]]), [50, 37]
    q = torch.randn(2, heads, dim, generator=torch.Generator().manual_seed(0)).cuda()
    clean, _ = check(pkg, q, cache, table, ints(lens))
    flag = lambda scales, page, block: scales[page, 0, block].neg_()  # noqa: E731
    # behind the last token of a block that is seen in part, in keys and in values
    cache[0][1, 0, 18, 3] = cache[1][1, 0, 30, dim - 1] = cache[1][3, 0, 6, 0] = cache[0][3, 0, 5] = -128
    for scales in (cache[2], cache[3]):
        for page, block in ((1, 1), (3, 0)):
            flag(scales, page, block)
    out = pkg.comp_attn_decode_f32x8(q, *cache, table, ints(lens))
    assert torch.equal(out, clean)
    # in a value that the first row sees: that component of its outputs, no other
    cache[1][0, 0, 9, 11] = -128
    flag(cache[3], 0, 0)
    out = pkg.comp_attn_decode_f32x8(q, *cache, table, ints(lens))
    assert out[0, :, 11].isnan().all() and torch.equal(out[1], clean[1])
    rest = [d for d in range(dim) if d != 11]
    assert torch.equal(out[0][:, rest], clean[0][:, rest])
    # in a key that the second row sees
    cache[0][3, 0, 2, dim - 1] = -128
    out = pkg.comp_attn_decode_f32x8(q, *cache, table, ints(lens))
    assert out[1].isnan().all() and torch.equal(out[0][:, rest], clean[0][:, rest])


@pytest.mark.parametrize("seqs,n,heads,kv_heads,dim", [(5, 70001, 16, 8, 64), (8, 70001, 36, 4, 128),
                                                       (5, 70001, 8, 8, 128)])
def test_decode_long(pkg, seqs, n, heads, kv_heads, dim):
    """More tiles of a row than a run of sums in one piece, against 64-bit sums on the device."""
    page = 128
    lens = [n - 997 * i for i in range(seqs)]
    need = [-(-m // page) for m in lens]
    cache = pool(sum(need), kv_heads, page, dim, seed=1)
    table = ints(rows_of(lens, page, sum(need), seed=4))
    q = torch.randn(seqs, heads, dim, generator=torch.Generator().manual_seed(0)).cuda()
    lse = torch.empty(seqs, heads, device="cuda")
    out = pkg.comp_attn_decode_f32x8(q, *cache, table, ints(lens), lse=lse)
    group = heads // kv_heads
    for b in (0, seqs - 1):
        for h in (0, heads - 1):
            at = table[b, :need[b]].long()
            k, v = ((c[at, h // group].double() * s[at, h // group].double().repeat_interleave(16, 1)[..., None])
                    .flatten(0, 1)[:lens[b]] for c, s in ((cache[0], cache[2]), (cache[1], cache[3])))
            plain.check_rows(out[b, h][None].cpu(), lse[b, h][None].cpu(), q[b, h][None].cpu(), k.cpu(), v.cpu(),
                             dim ** -0.5)


@pytest.mark.parametrize("heads,kv_heads", [(4, 2), (6, 1)])
def test_decode_many_short_sequences(pkg, heads, kv_heads):
    """More sequences than lanes, most of them shorter than a tile, many empty; rows share pieces."""
    rng, dim, page, batch = random.Random(7), 64, 16, 1500
    lens = [rng.choice([0, 0, 1, 2, 15, 16, 17, 40, 64, 65, 130]) for _ in range(batch)]
    need = sum(-(-n // page) for n in lens)
    cache = pool(need, kv_heads, page, dim)
    table = ints(rows_of(lens, page, need, seed=2))
    g = torch.Generator().manual_seed(0)
    q = torch.randn(batch, heads, dim, generator=g).cuda()
    lse = torch.empty(batch, heads, device="cuda")
    out = pkg.comp_attn_decode_f32x8(q, *cache, table, ints(lens), lse=lse)
    k, v = ((c.double() * s.double().repeat_interleave(16, 2)[..., None])[table.long().clamp_min(0)]
            .transpose(1, 2).flatten(2, 3).repeat_interleave(heads // kv_heads, 1)
            for c, s in ((cache[0], cache[2]), (cache[1], cache[3])))
    seen = (torch.arange(k.shape[2], device="cuda") < ints(lens)[:, None])[:, None]
    x = (torch.einsum("bhd,bhjd->bhj", q.double(), k) / 8).masked_fill(~seen, -math.inf)
    e = 4e-6 * torch.einsum("bhd,bhjd->bhj", q.double().abs(), k.abs()).masked_fill(~seen, 0).amax(-1) / 8
    want = torch.logsumexp(x, -1)
    some = ints(lens) > 0
    assert torch.isneginf(lse[~some]).all() and not out[~some].any()
    assert ((lse - want).abs() <= e + 4e-6 * (1 + want.abs()))[some].all()
    p = torch.softmax(x, -1).nan_to_num(0.0)
    # as in attn_check, and 2^-39 of each weight (kv8_check)
    size = torch.einsum("bhj,bhjd->bhd", p, v.abs())
    tol = (2 * torch.expm1(e) + 8e-6)[..., None] * size + 2.0 ** -39 * (v.abs() * seen[..., None]).sum(2) + 1e-30
    assert ((out - torch.einsum("bhj,bhjd->bhd", p, v)).abs() <= tol)[some].all()


def test_broadcast_inputs(pkg):
    """One head's keys for all heads, one token for all rows: strides of zero are read as they are."""
    cache, other = pool(8, 3, 16, 64), pool(8, 3, 16, 64)
    x = torch.randn(1, 1, 64, device="cuda")
    table, start, t = ints([[0, 1], [2, 3], [4, 5]]), ints([3, 0, 17]), pkg.comp_rope_table(40, 64)
    k, v = x.expand(3, 3, 64), (2 * x).expand(3, 3, 64)
    pkg.comp_kv8_append_f32(k, v, *cache, table, start, rope=t)
    pkg.comp_kv8_append_f32(k.contiguous(), v.contiguous(), *other, table, start, rope=t)
    assert all(torch.equal(a, b) for a, b in zip(cache, other))
    q = x.expand(3, 6, 64)
    assert torch.equal(pkg.comp_attn_decode_f32x8(q, *cache, table, start + 1, rope=t),
                       pkg.comp_attn_decode_f32x8(q.contiguous(), *cache, table, start + 1, rope=t))
    assert torch.equal(pkg.comp_rope_f32(q, t, start), pkg.comp_rope_f32(q.contiguous(), t, start))


def test_two_streams_at_once(pkg):
    """Calls on two streams, each with a cache of its own, do not disturb each other."""
    lens = [700, 90, 1200]
    runs = []
    for seed in (1, 2):
        cache = pool(80, 2, 32, 128, seed=seed)
        table = ints(rows_of([n + 40 for n in lens], 32, 80, seed=seed))
        x = torch.randn(3, 12, 128, generator=torch.Generator().manual_seed(seed)).cuda()
        runs.append((cache, table, x, torch.cuda.Stream()))
    angles = pkg.comp_rope_table(1300, 128)

    def step(cache, table, x, n, stream=None):
        pkg.comp_kv8_append_f32(x[:, 8:10], x[:, 10:], *cache, table, n, rope=angles, stream=stream)
        return pkg.comp_attn_decode_f32x8(x[:, :8], *cache, table, n + 1, rope=angles, stream=stream)

    at = [ints([n + i for n in lens]) for i in range(31)]
    want = []
    for cache, table, x, _ in runs:
        own = [t.clone() for t in cache]
        want.append([step(own, table, x, at[i]) for i in range(30)])
    torch.cuda.synchronize()
    got = [[], []]
    for i in range(30):
        for r, (cache, table, x, s) in enumerate(runs):
            with torch.cuda.stream(s):
                got[r].append(step(cache, table, x, at[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in (0, 1) for a, b in zip(got[r], want[r]))


def test_decode_identical_keys(pkg):
    """Equal terms round the same way each time: sums of 65536 of them stay within the tolerance."""
    cache = pool(512, 1, 128, 64)
    for t in cache[:2]:
        t.copy_(t[0, 0, 0].expand_as(t))
    for t in cache[2:]:
        t.fill_(0.013)
    n = 65536
    q = torch.randn(1, 1, 64, generator=torch.Generator().manual_seed(0)).cuda()
    lse = torch.empty(1, 1, device="cuda")
    out = pkg.comp_attn_decode_f32x8(q, *cache, ints([list(range(512))]), ints([n]), lse=lse)
    k, v = (t[0, 0, 0].double().cpu() * float(s[0, 0, 0]) for t, s in ((cache[0], cache[2]), (cache[1], cache[3])))
    s = float(q[0, 0].double().cpu() @ k) / 8
    e = 4e-6 * float(q[0, 0].abs().double().cpu() @ k.abs()) / 8
    # identical scores: the weights cancel and only sums' and products' roundings are left
    assert float(((out[0, 0].cpu().double() - v).abs() / (8e-6 * v.abs() + 1e-30)).max()) <= 1
    assert abs(float(lse) - (s + math.log(n))) <= e + 4e-6 * (1 + abs(s + math.log(n)))


def test_decode_large_scores_end_at_zero(pkg):
    cache = pool(4, 1, 64, 128)
    q = 60000 * torch.randn(2, 4, 128, generator=torch.Generator().manual_seed(0)).clamp(-1, 1).cuda()
    table, lens = ints([[0, 1], [2, 3]]), ints([128, 100])
    k, v = (c.values(torch.float64) for c in plain_of(cache))
    out = pkg.comp_attn_decode_f32x8(q, *cache, table, lens).cpu().double()
    for b, pages in enumerate(([0, 1], [2, 3])):
        n = int(lens[b])
        s = k[pages, 0].flatten(0, 1)[:n] @ q[b].cpu().double().T
        top, second = s.topk(2, 0).values
        # a gap far above the scores' error: one key takes it all
        clear = (top - second) * 128 ** -0.5 > 100 + 8e-6 * float((k.abs().max() * 60000 * 128) * 128 ** -0.5)
        want = v[pages, 0].flatten(0, 1)[s.argmax(0)]
        for h in range(4):
            if clear[h]:
                assert float((out[b, h] - want[h]).abs().max()) <= 8e-6 * float(want.abs().max())


def test_decode_is_the_same_every_time(pkg):
    lens = [5000, 300, 2222, 17, 4096]
    cache = pool(400, 4, 32, 128)
    table = ints(rows_of(lens, 32, 400, seed=3))
    q = torch.randn(5, 16, 128, device="cuda")
    first = pkg.comp_attn_decode_f32x8(q, *cache, table, ints(lens))
    for _ in range(5):
        assert torch.equal(pkg.comp_attn_decode_f32x8(q, *cache, table, ints(lens)), first)
    workspace = torch.empty(64 << 20, dtype=torch.uint8, device="cuda").fill_(255)
    assert torch.equal(pkg.comp_attn_decode_f32x8(q, *cache, table, ints(lens), workspace=workspace), first)


def test_graphs_and_streams(pkg):
    """Two captured steps that share a workspace, replayed in turn, and a call on a stream of its own."""
    lens = [700, 33, 1]
    table = ints(rows_of([n + 5 for n in lens], 16, 60, seed=3))
    angles = pkg.comp_rope_table(800, 64)
    workspace = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    runs = []
    for seed in (1, 2):
        g = torch.Generator().manual_seed(seed)
        cache, n = pool(60, 2, 16, 64, seed=seed), ints(lens)
        x = torch.randn(3, 12, 64, generator=g).cuda()
        out = torch.zeros(3, 8, 64, device="cuda")
        eager = [t.clone() for t in cache]
        pkg.comp_kv8_append_f32(x[:, 8:10], x[:, 10:], *eager, table, n, rope=angles)
        want = pkg.comp_attn_decode_f32x8(x[:, :8], *eager, table, n + 1, rope=angles)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pkg.comp_kv8_append_f32(x[:, 8:10], x[:, 10:], *cache, table, n, rope=angles)
            pkg.comp_attn_decode_f32x8(x[:, :8], *cache, table, n + 1, rope=angles, out=out, workspace=workspace)
        runs.append((graph, out, want, cache, eager, x, n))  # what a graph reads stays
    for _ in range(3):
        for graph, out, want, cache, eager, *_ in runs:
            out.zero_()
            graph.replay()
            assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(cache, eager))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    cache, want = runs[0][4], runs[0][2]
    x = torch.randn(3, 12, 64, generator=torch.Generator().manual_seed(1)).cuda()
    torch.cuda.synchronize()
    got = pkg.comp_attn_decode_f32x8(x[:, :8], *cache, table, ints(lens) + 1, rope=angles, stream=s.cuda_stream)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_step_by_step_is_the_whole_prompt(pkg):
    """Rotation, pages, quantisation and decoding together, against packed attention over what is read back."""
    heads, kv_heads, dim, page, steps = 8, 2, 64, 16, 20
    g = torch.Generator().manual_seed(0)
    lens = [37, 0, 16]
    angles = pkg.comp_rope_table(100, dim, factor=2.0)
    refs = torch.zeros(40, dtype=torch.int32, device="cuda")
    table = torch.full((3, 6), -1, dtype=torch.int32, device="cuda")
    cache = pool(40, kv_heads, page, dim)
    prompt = torch.randn(sum(lens), 2 * kv_heads, dim, generator=g).cuda()
    cu = ints([0, 37, 37, 53])
    table, refs, left = pkg.comp_kv_reserve(table, ints(lens), refs, page)
    pkg.comp_kv8_append_f32(prompt[:, :kv_heads], prompt[:, kv_heads:], *cache, table, ints([0, 0, 0]), cu, rope=angles)
    at = ints(lens)
    for _ in range(steps):
        x = torch.randn(3, heads + 2 * kv_heads, dim, generator=g).cuda()
        table, refs, left = pkg.comp_kv_reserve(table, at + 1, refs, page)
        pkg.comp_kv8_append_f32(x[:, heads:heads + kv_heads], x[:, heads + kv_heads:], *cache, table, at, rope=angles)
        at = at + 1
        lse = torch.empty(3, heads, device="cuda")
        out = pkg.comp_attn_decode_f32x8(x[:, :heads], *cache, table, at, rope=angles, lse=lse)
        # each sequence's one query over its past, read back
        total = int(at.sum())
        ends = torch.cat([ints([0]), at.cumsum(0).int()])
        k, v = pkg.comp_kv8_read_f32(*cache, table, ints([0, 0, 0]), ends, total)
        q = pkg.comp_rope_f32(x[:, :heads], angles, at - 1)
        lse2 = torch.empty(3, heads, device="cuda")
        want = pkg.comp_attn_f32(q, k, v, ints([0, 1, 2, 3]), ends, lse=lse2)
        # both are within the attention tests' tolerance of the exact sums, here some 2e-5 of the output
        assert float((out - want).norm() / want.norm()) < 4e-5 and float((lse - lse2).abs().max()) < 1e-4
    assert left.item() == 40 - sum(-(-(n + steps) // page) for n in lens)


# ---------------------------------------------------------------------------
# Pages
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("heads,page,dim", [(2, 16, 64), (1, 32, 128), (3, 64, 80), (5, 128, 16)])
def test_fork(pkg, heads, page, dim):
    pages, width = 40, 4
    cache = pool(pages, heads, page, dim)
    cache[2][3, 0, 0].neg_()
    lens = [page * 2 + 5, page, 1, page * 3 + page - 1, page + 16, 20 if page > 16 else 3]
    table = rows_of(lens, page, 30, seed=1)
    table = [r + [-1] * (width - len(r)) for r in table] + [[-1] * width for _ in range(7)]
    table[4][1] = 99                                       # a page that is not there: its copy reads zeros
    refs = [0] * pages
    for r in table:
        for p in r:
            if 0 <= p < pages:
                refs[p] += 1
    want = [t.cpu().clone() for t in cache]
    free = [p for p in range(pages) if refs[p] == 0]
    parents, children = [0, 3, 4, 2, 5, 1], [7, 6, 12, 8, 10, 9]
    want_t = [list(r) for r in table]
    for a, c in zip(parents, children):
        full, rest = divmod(lens[a], page)
        want_t[c] = table[a][:full] + [-1] * (width - full)
        if rest:
            p, src = free.pop(0), table[a][full]
            want_t[c][full] = p
            blocks = -(-rest // 16)
            for t in want[:2]:
                t[p, :, :rest] = t[src, :, :rest] if src < pages else 0
            for t in want[2:]:
                t[p, :, :blocks] = t[src, :, :blocks] if src < pages else 0
    got = pkg.comp_kv8_fork(*cache, ints(table), ints(lens + [0] * 7), ints(refs), ints(parents), ints(children))
    assert got[0].tolist() == want_t and got[3].tolist() == [len(free)]
    assert all(torch.equal(a.cpu(), b) for a, b in zip(cache, want))


def test_compact_and_copy(pkg):
    for heads, page, dim, pages in ((2, 16, 64, 300), (1, 128, 128, 40), (3, 64, 16, 77)):
        cache = pool(pages, heads, page, dim, seed=pages)
        rng = random.Random(pages)
        live = sorted(rng.sample(range(pages), pages // 2))
        refs = [1 if p in live else 0 for p in range(pages)]
        rows = [live[i::3] for i in range(3)]
        table = [r + [-1] * (pages // 3 + 1 - len(r)) for r in rows]
        before = [t.clone() for t in cache]
        t2, r2, remap, count = pkg.comp_kv8_compact(*cache, ints(table), ints(refs))
        assert count.item() == len(live) and r2.tolist() == [1] * len(live) + [0] * (pages - len(live))
        for old_row, new_row in zip(table, t2.tolist()):
            for a, b in zip(old_row, new_row):
                assert (a < 0) == (b < 0) and b < len(live)
                if a >= 0:
                    assert all(torch.equal(x[a], y[b]) for x, y in zip(before, cache))
        both = rng.sample(range(pages), 20)
        before = [t.clone() for t in cache]
        pkg.comp_kv8_copy_pages(*cache, ints(both[:10] + [-1, pages]), ints(both[10:] + [0, 0]))
        for t, b in zip(cache, before):
            b[both[10:]] = b[both[:10]]
            assert torch.equal(t, b)


def test_offsets_beyond_32_bits(pkg):
    """A cache of more than 2^32 bytes a side: pages at its far end are written, read, attended to and copied."""
    heads, page, dim = 8, 128, 128
    pages = (1 << 32) // (heads * page * dim) + 40
    codes = [torch.empty(pages, heads, page, dim, dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(pages, heads, page // 16, device="cuda") for _ in range(2)]
    cache = (*codes, *scales)
    table = ints([[pages - 1, pages - 7, pages - 3]])
    x = torch.randn(300, 16, dim, generator=torch.Generator().manual_seed(0)).cuda()
    pkg.comp_kv8_append_f32(x[:, :8], x[:, 8:], *cache, table, ints([0]), ints([0, 300]))
    k, v = pkg.comp_kv8_read_f32(*cache, table, ints([0]), ints([0, 300]), 300)
    small = pool(3, heads, page, dim)
    pkg.comp_kv8_append_f32(x[:, :8], x[:, 8:], *small, ints([[0, 1, 2]]), ints([0]), ints([0, 300]))
    k2, v2 = pkg.comp_kv8_read_f32(*small, ints([[0, 1, 2]]), ints([0]), ints([0, 300]), 300)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    q = torch.randn(1, 8, dim, device="cuda")
    want = pkg.comp_attn_decode_f32x8(q, *small, ints([[0, 1, 2]]), ints([300]))
    assert torch.equal(pkg.comp_attn_decode_f32x8(q, *cache, table, ints([300])), want)
    pkg.comp_kv8_copy_pages(*cache, table[0].contiguous(), ints([pages - 20, pages - 21, pages - 22]))
    moved = ints([[pages - 20, pages - 21, pages - 22]])
    assert torch.equal(pkg.comp_attn_decode_f32x8(q, *cache, moved, ints([300])), want)


def test_refusals(pkg):
    cache = pool(4, 2, 32, 64)
    k = torch.zeros(2, 2, 64, device="cuda")
    q = torch.zeros(2, 4, 64, device="cuda")
    table, n = ints([[0, 1], [2, 3]]), ints([3, 4])
    t = pkg.comp_rope_table(8, 64)

    def refused(f):
        with pytest.raises((ValueError, TypeError, pkg.CompError)):
            f()

    bad = [[cache[0].half(), *cache[1:]], [cache[0], cache[1][:3], *cache[2:]], [*cache[:2], cache[2].half(), cache[3]],
           [*cache[:3], cache[3][..., :1]], [cache[0].cpu(), *cache[1:]], [cache[0], cache[0], *cache[2:]],
           [*cache[:2], cache[2], cache[2]], [cache[0].transpose(1, 2), *cache[1:]],
           [c[:, :, :24].contiguous() for c in cache[:2]] + cache[2:],
           [c[..., :40].contiguous() for c in cache[:2]] + cache[2:], [cache[0][0], *cache[1:]]]
    for c in bad:
        refused(lambda: pkg.comp_kv8_append_f32(k, k, *c, table, n))
        refused(lambda: pkg.comp_kv8_read_f32(*c, table, n, None, 2))
        refused(lambda: pkg.comp_attn_decode_f32x8(q, *c, table, n))
        refused(lambda: pkg.comp_kv8_copy_pages(*c, n, n))
    for args in ((k.half(), k, table, n), (k[:1], k[:1], table, n), (k, k[..., :32], table, n), (k, k, table[0], n),
                 (k, k, table, n[:1]), (k, k, table, n, n), (k, k, table.long(), n)):
        refused(lambda: pkg.comp_kv8_append_f32(*args[:2], *cache, *args[2:]))
    refused(lambda: pkg.comp_kv8_append_f32(k, k, *cache, table, n, rope=t.cpu()))
    refused(lambda: pkg.comp_kv8_append_f32(k, k, *cache, table, n, rope=pkg.comp_rope_table(8, 66)))
    refused(lambda: pkg.comp_kv8_read_f32(*cache, table, n, None, 3))
    refused(lambda: pkg.comp_kv8_read_f32(*cache, table, n, ints([0, 1, 2]), -1))
    refused(lambda: pkg.comp_kv8_read_f32(*cache, table, n, None, 2, k=k.half()))
    refused(lambda: pkg.comp_kv8_read_f16(*cache, table, n, None, 2, k=k))
    refused(lambda: pkg.comp_kv8_read_f32(*cache, table, n, None, 2, k=k, v=k))
    refused(lambda: pkg.comp_kv8_read_f32(*cache, table, n, None, 2, v=k[:1].expand(2, 2, 64)))
    for args, kw in (((q[:1], table, n), {}), ((q[:, :3], table, n), {}), ((q[..., :32], table, n), {}),
                     ((q, table, n[:1]), {}), ((q.half(), table, n), {}), ((q, table, n), dict(scale=-1.0)),
                     ((q, table, n), dict(lse=torch.zeros(2, 3, device="cuda"))), ((q, table, n), dict(out=q)),
                     ((q, table, n), dict(workspace=torch.zeros(16, device="cuda"))),
                     ((q, table, n), dict(rope=t[:, :, :1])), ((q, table, n), dict(rope=q))):
        refused(lambda: pkg.comp_attn_decode_f32x8(args[0], *cache, *args[1:], **kw))
    assert pkg.device_status()[0] == 0
