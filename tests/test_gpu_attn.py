"""Attention over packed prompts and over the paged cache, against 64-bit sums."""
import itertools
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from attn_check import check_attn, check_decode  # noqa: E402


@pytest.fixture(scope="module")
def pkg():
    import __graft_entry__

    __graft_entry__.build()
    import compensated_fp32_projection_gb300 as p

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield p
    assert p.device_status() == (0, 0)


def cu_of(lens):
    return [0] + list(itertools.accumulate(lens))


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def case(lens_q, lens_k, heads, kv_heads, dim, kv, seed=0, q_scale=2.0):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(sum(lens_q), heads, dim, generator=g) * q_scale
    k, v = (torch.randn(sum(lens_k), kv_heads, dim, generator=g) for _ in range(2))
    if kv == torch.float16:
        k, v = k.half(), v.half()
    return q.cuda(), k.cuda(), v.cuda()


def call(pkg, q, k, v, cu_q, cu_k, causal, scale=None, **more):
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    f = pkg.comp_attn_f32 if k.dtype == torch.float32 else pkg.comp_attn_f32x16
    out = f(q, k, v, ints(cu_q), ints(cu_k), causal=causal, scale=scale, lse=lse, **more)
    return out, lse


KV = [torch.float16, torch.float32]


@pytest.mark.parametrize("kv", KV, ids=["f16", "f32"])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("lens_q,lens_k", [
    ([1], [1]),
    ([1], [300]),
    ([127], [127]),
    ([128, 129], [128, 129]),
    ([0, 5, 0, 64, 1], [0, 5, 3, 64, 1]),       # sequences without tokens, and without queries
    ([9, 20], [4, 0]),                          # more queries than keys: causal rows that see nothing; no keys at all
    ([33, 2, 65], [200, 131, 257]),             # queries that continue a longer sequence
    ([257], [511]),
], ids=str)
def test_lengths(pkg, lens_q, lens_k, causal, kv):
    q, k, v = case(lens_q, lens_k, 4, 2, 64, kv)
    cu_q, cu_k = cu_of(lens_q), cu_of(lens_k)
    out, lse = call(pkg, q, k, v, cu_q, cu_k, causal)
    check_attn(out, lse, q, k, v, cu_q, cu_k, causal, 64 ** -0.5)


@pytest.mark.parametrize("kv", KV, ids=["f16", "f32"])
@pytest.mark.parametrize("heads,kv_heads,dim", [(1, 1, 1), (3, 1, 17), (2, 2, 40), (6, 2, 72), (5, 5, 80), (8, 1, 96),
                                                (4, 4, 127), (8, 2, 128), (28, 4, 128), (20, 1, 64), (7, 7, 8)])
def test_heads(pkg, heads, kv_heads, dim, kv):
    lens = [150, 1, 37]
    q, k, v = case(lens, lens, heads, kv_heads, dim, kv, seed=1)
    cu = cu_of(lens)
    out, lse = call(pkg, q, k, v, cu, cu, True)
    check_attn(out, lse, q, k, v, cu, cu, True, dim ** -0.5)


@pytest.mark.parametrize("kv", KV, ids=["f16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 60])
def test_parts_of_one_projection(pkg, kv, dim):
    """q, k and v side by side in one tensor, at an odd offset too; out strided."""
    heads, kv_heads, n = 4, 2, 141
    for pad in (0, 1, 8):
        g = torch.Generator().manual_seed(2)
        width = (heads + 2 * kv_heads) * dim + pad
        x = torch.randn(n, width, generator=g).cuda()
        at = pad
        q = x[:, at:at + heads * dim].view(n, heads, dim)
        kvx = x.to(kv)
        k = kvx[:, at + heads * dim:at + (heads + kv_heads) * dim].view(n, kv_heads, dim)
        v = kvx[:, at + (heads + kv_heads) * dim:].view(n, kv_heads, dim)
        place = torch.full((n, heads, dim + 5), 3.0, device="cuda")
        out, lse = call(pkg, q, k, v, [0, n], [0, n], True, out=place[:, :, :dim])
        check_attn(out, lse, q, k, v, [0, n], [0, n], True, dim ** -0.5)
        assert bool((place[:, :, dim:] == 3.0).all())
        head_major = torch.empty(heads, n, dim, device="cuda")
        again, _ = call(pkg, q, k, v, [0, n], [0, n], True, out=head_major.transpose(0, 1))
        assert torch.equal(again, out)


def test_one_key_head_broadcast(pkg):
    q, k, v = case([70], [70], 4, 1, 64, torch.float16, seed=3)
    out, lse = call(pkg, q, k.expand(70, 4, 64), v.expand(70, 4, 64), [0, 70], [0, 70], True)
    check_attn(out, lse, q, k, v, [0, 70], [0, 70], True, 64 ** -0.5)


@pytest.mark.parametrize("kv", KV, ids=["f16", "f32"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dim", [64, 128])
def test_hidden_values_have_no_influence(pkg, kv, bad, dim):
    """What a row may not see can hold anything: later tokens, and other sequences."""
    lens = [40, 200, 90]
    q, k, v = case(lens, lens, 4, 2, dim, kv, seed=4)
    cu = cu_of(lens)
    plain, plain_lse = call(pkg, q, k, v, cu, cu, True)
    k2, v2 = k.clone(), v.clone()
    hurt = [30, 40 + 150, 40 + 199, 240 + 13]      # a token in each sequence, and one's last
    for j, t in enumerate(hurt):
        k2[t, j % 2, 3] = bad
        v2[t, j % 2, 5 * j] = bad
    out, lse = call(pkg, q, k2, v2, cu, cu, True)
    for j, t in enumerate(hurt):
        start = max(a for a in cu if a <= t)
        first = min(x for x in hurt if x >= start)
        assert torch.equal(out[start:first], plain[start:first])
        assert torch.equal(lse[start:first], plain_lse[start:first])
        mine = slice(2 * (j % 2), 2 * (j % 2) + 2)
        assert not bool(out[t, mine].isfinite().all())     # the token itself sees it


@pytest.mark.parametrize("kv", KV, ids=["f16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
def test_only_the_value_is_not_finite(pkg, kv, dim):
    """A non-finite value reaches its own column, of the rows that see it, alone."""
    q, k, v = case([300], [300], 2, 1, dim, kv, seed=5)
    plain, plain_lse = call(pkg, q, k, v, [0, 300], [0, 300], True)
    v2 = v.clone()
    v2[170, 0, 7] = math.inf
    out, lse = call(pkg, q, k, v2, [0, 300], [0, 300], True)
    assert torch.equal(lse, plain_lse)
    assert torch.equal(out[:170], plain[:170])
    keep = [d for d in range(dim) if d != 7]
    assert torch.equal(out[:, :, keep], plain[:, :, keep])
    assert not bool(out[170:, :, 7].isfinite().any())


@pytest.mark.parametrize("kv", KV, ids=["f16", "f32"])
def test_sizes_of_scores(pkg, kv):
    """Scores from next to nothing to thousands, values over the whole range, outliers among them."""
    for q_scale, scale in ((1e-4, 0.125), (40.0, 0.125), (300.0, 1.0), (2.0, 1e-3)):
        q, k, v = case([260], [260], 2, 2, 64, kv, seed=6, q_scale=q_scale)
        v = v * torch.logspace(-4, 3, 64, device="cuda").to(v.dtype)
        k[::7] *= 8
        out, lse = call(pkg, q, k, v, [0, 260], [0, 260], True, scale=scale)
        check_attn(out, lse, q, k, v, [0, 260], [0, 260], True, scale)


def large_scores(n, dim, unit, seed):
    """Keys c_j (1, 1, ...) of shuffled multiples c_j of `unit`: a query a (1, 1, ...)
    with a > 15 gives scores that are 100 and more apart, and far beside their
    rounding, so the largest one's value is the output."""
    c = torch.randperm(n, generator=torch.Generator().manual_seed(seed)) + 400
    k = (unit * c).float()[:, None, None].expand(n, 1, dim).contiguous()
    v = torch.randn(n, 1, dim, generator=torch.Generator().manual_seed(seed + 1))
    return k, v


def check_largest(out, lse, q, k, v, seen):
    """out: what the two products round away (4e-6 of a value); lse: the score's own 4e-6."""
    s = torch.where(seen, (q[:, 0].double() @ k[:, 0].double().T) * q.shape[2] ** -0.5, -math.inf)
    top, at = s.max(1)
    assert bool(((out[:, 0] - v[at, 0]).abs() <= 4e-6 * v[at, 0].abs()).all())
    assert bool(((lse[:, 0].double() - top).abs() <= 4e-6 * top.abs()).all())


@pytest.mark.parametrize("n,dim", [(300, 64), (300, 128), (1100, 128)])
@pytest.mark.parametrize("size", [1e-5, 1e-7, 1e-9])
def test_small_values(pkg, n, dim, size):
    """A split value is off by at most 2^-22 of it or 2^-35, whichever is more: in v the
    2^-35 reach the output as they are, in q and k scores that are next to nothing."""
    from attn_check import compare, exact_rows

    q, k, v = case([n], [n], 1, 1, dim, torch.float32, seed=19)
    for q2, k2, v2 in ((q, k, v * size), (q * size, k, v), (q, k * size, v)):
        out, lse = (x.cpu()[:, 0] for x in call(pkg, q2, k2, v2, [0, n], [0, n], False))
        qc, kc, vc = (x.cpu()[:, 0] for x in (q2, k2, v2))
        x_out, x_lse, tol, ltol = exact_rows(qc, kc, vc, torch.ones(n, n, dtype=torch.bool), dim ** -0.5)
        e = 2.0 ** -35 * dim ** -0.5 * float(torch.maximum(qc.abs().sum(1).max(), kc.abs().sum(1).max()))
        compare(out, lse, x_out, x_lse, tol + 2.0 ** -35 + 2 * math.expm1(e) * float(vc.abs().max()), ltol + e)


@pytest.mark.parametrize("kv", KV, ids=["f16", "f32"])
@pytest.mark.parametrize("n,dim", [(300, 64), (300, 128), (1100, 128)])
@pytest.mark.parametrize("unit", [1, -1, 32, -32])
def test_scores_of_any_size(pkg, kv, n, dim, unit):
    """Scores from 5 10^4 to 3 10^10, in one warp's rows side by side."""
    k, v = large_scores(n, dim, unit, seed=n)
    k, v = k.to(kv), v.to(kv)
    a = 2.0 ** (4 + torch.arange(n) % 12) * 1.96875
    q = a[:, None, None].expand(n, 1, dim).contiguous()
    q[1::2] *= 0.5078125  # bits below FP16's too
    out, lse = call(pkg, q.cuda(), k.cuda(), v.cuda(), [0, n], [0, n], True)
    check_largest(out.cpu(), lse.cpu(), q, k, v.float(), torch.ones(n, n, dtype=torch.bool).tril())


@pytest.mark.parametrize("kv", KV, ids=["f16", "f32"])
@pytest.mark.parametrize("heads,kv_heads,dim,n", [(2, 1, 128, 2500), (2, 2, 64, 4100)])
def test_long(pkg, kv, heads, kv_heads, dim, n):
    q, k, v = case([n], [n], heads, kv_heads, dim, kv, seed=7)
    out, lse = call(pkg, q, k, v, [0, n], [0, n], True)
    rows = torch.arange(0, n, 97).tolist() + [n - 1]
    from attn_check import compare, exact_rows

    qc, kc, vc, oc, lc = (x.cpu() for x in (q, k, v, out, lse))
    for h in range(heads):
        g = h // (heads // kv_heads)
        seen = torch.arange(n)[None] <= torch.tensor(rows)[:, None]
        compare(oc[rows, h], lc[rows, h], *exact_rows(qc[rows, h], kc[:, g], vc[:, g], seen, dim ** -0.5))


def equal_keys(n, s1, dim, kv, queries, heads, kv_heads):
    """Keys that all score 0 but the first, which scores s1; values about 1: the
    additions of equal weights to a growing sum all round the same way."""
    q = torch.ones(queries, heads, dim)
    k = torch.zeros(n, kv_heads, dim)
    k[0] = s1 * dim ** -0.5
    v = torch.rand(n, kv_heads, dim, generator=torch.Generator().manual_seed(n)) + 0.5
    return q, k.to(kv), v.to(kv)


def compare_equal_keys(out, lse, q, k, v):
    """All rows against one in 64 bits.  lse more closely than the tests' general
    bound: sums of at most 64 equal terms (4e-6 with the exponentials' own error),
    one compensated addition a tile, the logarithm and the last rounding."""
    from attn_check import compare, exact_rows

    heads, n = q.shape[1], k.shape[0]
    group = heads // k.shape[1]
    for g in range(k.shape[1]):  # all queries are the same
        x_out, x_lse, tol, _ = exact_rows(q[:1, 0].cpu(), k[:, g], v[:, g], torch.ones(1, n, dtype=torch.bool),
                                          q.shape[2] ** -0.5)
        e = 4e-6 * q.shape[2] ** -0.5 * float((k[:, g].double().abs() @ q[0, 0].double().cpu()).max())
        ltol = e + 4e-6 + 2.0 ** -22 * x_lse.abs()
        mine = out[:, g * group:(g + 1) * group].flatten(0, 1).cpu()
        mine_lse = lse[:, g * group:(g + 1) * group].flatten().cpu()
        rows = mine.shape[0]
        compare(mine, mine_lse, x_out.expand(rows, -1), x_lse.expand(rows), tol.expand(rows, -1), ltol.expand(rows))


@pytest.mark.parametrize("kv", KV, ids=["f16", "f32"])
@pytest.mark.parametrize("queries,dim", [(3, 64), (3, 128), (600, 128)])   # the last: pairs of CTAs for FP32
@pytest.mark.parametrize("n,s1", [(16384, 0.3), (16384, 0.5), (65536, 0.7)])
def test_many_equal_keys(pkg, n, s1, queries, dim, kv):
    q, k, v = equal_keys(n, s1, dim, kv, queries, 2, 1)
    out, lse = call(pkg, q.cuda(), k.cuda(), v.cuda(), [0, queries], [0, n], False)
    compare_equal_keys(out, lse, q, k, v)


def sampled(out, lse, q, k, v, cu, causal, every):
    """check_attn on some rows of each sequence (its first and last among them)."""
    from attn_check import compare, exact_rows

    out, lse, q, k, v = (x.cpu() for x in (out, lse, q, k, v))
    group = q.shape[1] // k.shape[1]
    for a, b in zip(cu, cu[1:]):
        n = b - a
        rows = sorted({0, n // 2, n - 1, *range(0, n, every)})
        seen = torch.arange(n)[None] <= torch.tensor(rows)[:, None] if causal else torch.ones(len(rows), n,
                                                                                              dtype=torch.bool)
        at = [a + r for r in rows]
        for h in range(q.shape[1]):
            compare(out[at, h], lse[at, h], *exact_rows(q[at, h], k[a:b, h // group], v[a:b, h // group], seen,
                                                        q.shape[2] ** -0.5))


@pytest.mark.parametrize("kv", KV, ids=["f16", "f32"])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("lens,heads,kv_heads,dim", [
    ([1100, 1, 1535, 1600], 2, 2, 128),      # sequences that fill blocks of 512 rows, and ones that do not
    ([513, 700, 130], 9, 3, 72),             # three heads to a key head: blocks end inside a token
    ([2048, 511], 4, 1, 128),
    ([1030], 5, 5, 100),
], ids=str)
def test_long_packed(pkg, lens, heads, kv_heads, dim, causal, kv):
    q, k, v = case(lens, lens, heads, kv_heads, dim, kv, seed=10)
    cu = cu_of(lens)
    out, lse = call(pkg, q, k, v, cu, cu, causal)
    sampled(out, lse, q, k, v, cu, causal, 229)
    again, lse2 = call(pkg, q, k, v, cu, cu, causal)
    assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("kv", KV, ids=["f16", "f32"])
@pytest.mark.parametrize("column", [3, 100])
def test_long_hidden_values(pkg, kv, column):
    """As test_only_the_value_is_not_finite, in blocks of 512 rows; and what follows a sequence."""
    lens = [1300, 1200]
    q, k, v = case(lens, lens, 2, 2, 128, kv, seed=11)
    cu = cu_of(lens)
    plain, plain_lse = call(pkg, q, k, v, cu, cu, True)
    v2, k2 = v.clone(), k.clone()
    v2[777, 1, column] = math.nan
    v2[1300 + 600, 0, column] = math.inf
    k2[1300 + 1199, :, 5] = math.nan
    out, lse = call(pkg, q, k2, v2, cu, cu, True)
    keep = torch.ones(2500, 2, 128, dtype=torch.bool, device="cuda")
    keep[777:1300, 1, column] = False
    keep[1900:, 0, column] = False
    keep[2499] = False
    assert torch.equal(out[keep], plain[keep])
    assert not bool(out[777:1300, 1, column].isfinite().any())
    assert not bool(out[1900:, 0, column].isfinite().any())
    assert torch.equal(lse[:2499], plain_lse[:2499])


def test_reruns_side_stream_and_no_lse(pkg):
    lens = [300, 77, 1024]
    q, k, v = case(lens, lens, 8, 2, 128, torch.float16, seed=8)
    cu = cu_of(lens)
    out, lse = call(pkg, q, k, v, cu, cu, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q2 = q * 1.0
        again = pkg.comp_attn_f32x16(q2, k, v, ints(cu), ints(cu))
    side.synchronize()
    assert torch.equal(again, out)
    third = torch.empty_like(out)
    cu_t = ints(cu)
    torch.cuda.synchronize()
    pkg.comp_attn_f32x16(q, k, v, cu_t, cu_t, out=third, stream=side)
    side.synchronize()
    assert torch.equal(third, out)


def test_what_a_call_allocates_belongs_to_its_stream(pkg):
    """An output allocated for another stream must not be memory that work queued
    on the current stream, but not done yet, still writes."""
    q, k, v = case([64], [64], 4, 2, 64, torch.float32, seed=10)
    want = pkg.comp_attn_f32(q, k, v)
    kp, vp = (torch.zeros(8, 2, 16, 64, dtype=torch.float16, device="cuda") for _ in range(2))
    table, lengths = ints([[0, 1]]), ints([20])
    decoded = pkg.comp_attn_decode_f32x16(q[:1], kp, vp, table, lengths)
    refs, seqs = torch.zeros(8, dtype=torch.int32, device="cuda"), ints([5])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call_it, right in ((lambda: pkg.comp_attn_f32(q, k, v, stream=side), want),
                           (lambda: pkg.comp_attn_decode_f32x16(q[:1], kp, vp, table, lengths, stream=side), decoded),
                           (lambda: pkg.comp_kv_free(table, lengths, refs, seqs, stream=side)[0], table)):
        for queued in (right.numel() * right.element_size(), 4096, 1 << 16):
            old = torch.empty(queued, dtype=torch.uint8, device="cuda")
            torch.cuda._sleep(20_000_000)  # about 10 ms
            old.fill_(0x7f)
            del old  # the current stream may use this memory again: its work is in order
            got = call_it()
            side.synchronize()
            torch.cuda.synchronize()
            assert torch.equal(got, right)


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a device that is not the current one")
def test_tensors_that_are_not_on_the_current_device(pkg):
    q, k, v = case([64], [64], 4, 2, 64, torch.float16, seed=10)
    want = pkg.comp_attn_f32x16(q, k, v)
    kp, vp = (torch.zeros(8, 2, 16, 64, dtype=torch.float16, device="cuda:1") for _ in range(2))
    got = pkg.comp_attn_f32x16(*(x.to("cuda:1") for x in (q, k, v)))
    assert torch.cuda.current_device() == 0 and torch.equal(got.to("cuda:0"), want)
    new = k[:1].float().to("cuda:1")
    pkg.comp_kv_append_f32(new, new, kp, vp, ints([[3]]).to("cuda:1"), ints([5]).to("cuda:1"))
    pkg.comp_kv_copy_pages(kp, vp, ints([3]).to("cuda:1"), ints([6]).to("cuda:1"))
    torch.cuda.synchronize("cuda:1")
    assert torch.cuda.current_device() == 0
    assert torch.equal(kp[3, :, 5], k[0].to("cuda:1")) and torch.equal(kp[6], kp[3])


@pytest.mark.parametrize("kv", KV, ids=["f16", "f32"])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("cu,tokens,dim", [([0], 5, 64), ([0], 700, 128), ([0, 4, 9], 10, 64), ([0, 256], 777, 64),
                                           ([0, 600, 600, 1050], 2000, 128), (list(range(70)), 400, 80)], ids=str)
def test_tokens_beyond_the_last_sequence(pkg, cu, tokens, dim, causal, kv):
    """They see no key: zeros and -inf, and nothing stays unwritten."""
    q, k, v = case([tokens], [tokens], 4, 2, dim, kv, seed=14)
    out = torch.full_like(q, 7.0)
    _, lse = call(pkg, q, k, v, cu, cu, causal, out=out)
    n = cu[-1]
    assert bool((out[n:] == 0).all()) and bool(lse[n:].isneginf().all())
    check_attn(out[:n], lse[:n], q, k, v, cu, cu, causal, dim ** -0.5)


def test_no_sequence(pkg):
    """The C call with n_seq 0, with and without offsets."""
    import ctypes

    q, k, v = case([300], [300], 4, 2, 64, torch.float32, seed=14)
    lib, cu = pkg._native.load(), ints([0])
    a = pkg._native.Attn(0, 300, 300, 4, 2, 64, 1, 0.125, 256, 64, 128, 64, 128, 64, 256, 64)
    stream = torch.cuda.current_stream().cuda_stream
    for offsets in (None, cu.data_ptr()):
        out, lse = torch.full_like(q, 7.0), torch.full((300, 4), 7.0, device="cuda")
        assert lib.comp_attn_workspace_bytes(ctypes.byref(a), 4, k.data_ptr(), v.data_ptr()) == 0
        assert lib.comp_attn_f32(ctypes.byref(a), q.data_ptr(), k.data_ptr(), v.data_ptr(), offsets, offsets,
                                 out.data_ptr(), lse.data_ptr(), None, 0, stream) == 0
        assert bool((out == 0).all()) and bool(lse.isneginf().all())


def test_one_sequence_without_offsets(pkg):
    q, k, v = case([50], [80], 4, 2, 64, torch.float32, seed=9)
    out = pkg.comp_attn_f32(q, k, v)
    want, _ = call(pkg, q, k, v, [0, 50], [0, 80], True)
    assert torch.equal(out, want)


# --------------------------------------------------------------------------
# decode
# --------------------------------------------------------------------------
def cache_case(lengths, shared, page, heads, kv_heads, dim, seed=0, spare=3, hole=None):
    """Shuffled pages; what lies beyond the lengths is NaN."""
    g = torch.Generator().manual_seed(seed)
    own = [max(0, -(-n // page) - shared) for n in lengths]
    width = shared + max(own) + 1
    pages = shared + sum(own) + spare
    order = torch.randperm(pages, generator=g).tolist()
    k, v = (torch.full((pages, kv_heads, page, dim), math.nan, dtype=torch.float16) for _ in range(2))
    table, at = [], shared
    for n, o in zip(lengths, own):
        row = order[:shared] + order[at:at + o]
        at += o
        for i, p in enumerate(row):
            m = max(0, min(page, max(lengths) - i * page if i < shared else n - i * page))
            k[p, :, :m] = torch.randn(kv_heads, m, dim, generator=g).half() if i >= shared or k[p, 0, 0, 0].isnan() \
                else k[p, :, :m]
            v[p, :, :m] = torch.randn(kv_heads, m, dim, generator=g).half() if i >= shared or v[p, 0, 0, 0].isnan() \
                else v[p, :, :m]
        table.append(row + [-1] * (width - len(row)))
    q = torch.randn(len(lengths), heads, dim, generator=g) * 2
    return q.cuda(), k.cuda(), v.cuda(), ints(table), ints(lengths)


def decode(pkg, q, k, v, table, lengths, shared=0, **more):
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    return pkg.comp_attn_decode_f32x16(q, k, v, table, lengths, shared=shared, lse=lse, **more), lse


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 64), (8, 1, 128), (3, 3, 80), (20, 2, 128), (2, 2, 8),
                                                (12, 1, 96)])
def test_decode_lengths(pkg, page, heads, kv_heads, dim):
    lengths = [1, 0, page, page + 1, 5 * page - 1, 900, 2]
    q, k, v, table, n = cache_case(lengths, 0, page, heads, kv_heads, dim, seed=page)
    out, lse = decode(pkg, q, k, v, table, n)
    check_decode(out, lse, q, k, v, table, n, dim ** -0.5)


@pytest.mark.parametrize("shared,page,batch,heads,kv_heads,dim", [
    (1, 16, 3, 4, 2, 64), (8, 16, 5, 8, 2, 128), (9, 64, 40, 4, 1, 128), (3, 128, 70, 16, 2, 64), (33, 32, 2, 3, 1, 96),
    (70, 16, 260, 2, 2, 64), (2, 32, 17, 5, 5, 80), (5, 16, 9, 40, 1, 72),
])
def test_decode_shared_prefix(pkg, shared, page, batch, heads, kv_heads, dim):
    lengths = [shared * page + (7 * i * i) % 150 for i in range(batch)]
    q, k, v, table, n = cache_case(lengths, shared, page, heads, kv_heads, dim, seed=shared)
    out, lse = decode(pkg, q, k, v, table, n, shared)
    check_decode(out, lse, q, k, v, table, n, dim ** -0.5)
    apart, apart_lse = decode(pkg, q, k, v, table, n, 0)
    check_decode(apart, apart_lse, q, k, v, table, n, dim ** -0.5)


def test_decode_sequences_shorter_than_the_prefix(pkg):
    """A sequence may end inside the shared pages, or have nothing."""
    lengths = [400, 256, 255, 129, 64, 1, 0, 300, -5, 10 ** 9]
    q, k, v, table, n = cache_case([400] * 10, 8, 32, 4, 2, 64, seed=3)
    n = ints(lengths)
    k.nan_to_num_(0.25), v.nan_to_num_(0.25)
    out, lse = decode(pkg, q, k, v, table, n, 8)
    check_decode(out, lse, q, k, v, table, n, 64 ** -0.5)


@pytest.mark.parametrize("dim,swap", [(64, False), (128, False), (128, True)])
def test_decode_shared_prefix_halves_see_differently_much(pkg, dim, swap):
    """128 rows that see little of a long prefix beside 128 that see all of it: tiles
    pass that only one half of a block uses."""
    few, all_of_it = [i % 7 for i in range(128)], [1600 + i % 40 for i in range(128)]
    lengths = all_of_it + few if swap else few + all_of_it
    q, k, v, table, n = cache_case(lengths, 100, 16, 2, 2, dim, seed=dim + swap)
    out, lse = decode(pkg, q, k, v, table, n, 100)
    check_decode(out, lse, q, k, v, table, n, dim ** -0.5)


@pytest.mark.parametrize("shared,page,batch,heads,kv_heads,dim", [
    (300, 16, 5, 8, 2, 128), (64, 128, 33, 4, 2, 64), (129, 32, 16, 8, 1, 128), (129, 32, 17, 8, 1, 128),
    (40, 128, 2, 3, 3, 96), (33, 32, 128, 1, 1, 64), (72, 16, 7, 5, 1, 8),
])
def test_decode_shared_prefix_of_few_rows(pkg, shared, page, batch, heads, kv_heads, dim):
    """Long prefixes of up to 128 rows, and just above; some sequences end inside them."""
    lengths = [shared * page + 31 * i % 170 for i in range(batch)]
    lengths[1] = shared * page // 2 + 5
    q, k, v, table, n = cache_case(lengths, shared, page, heads, kv_heads, dim, seed=shared + batch)
    out, lse = decode(pkg, q, k, v, table, n, shared)
    check_decode(out, lse, q, k, v, table, n, dim ** -0.5)
    again, again_lse = decode(pkg, q, k, v, table, n, shared)
    assert torch.equal(again, out) and torch.equal(again_lse, lse)


@pytest.mark.parametrize("dim", [64, 128])
def test_decode_infinity_in_a_shared_value(pkg, dim):
    """A value that is not finite reaches the rows that see it and no others."""
    lengths = [3300, 1500, 900, 3200, 2999, 3000]
    q, k, v, table, n = cache_case([3300] * 6, 100, 32, 4, 2, dim, seed=dim)
    n = ints(lengths)
    k.nan_to_num_(0.25), v.nan_to_num_(0.25)
    plain, plain_lse = decode(pkg, q, k, v, table, n, 100)
    check_decode(plain, plain_lse, q, k, v, table, n, dim ** -0.5)
    token, head, column = 2999, 1, dim // 2 + 3
    v[int(table[0, token // 32]), head, token % 32, column] = math.inf
    out, lse = decode(pkg, q, k, v, table, n, 100)
    assert torch.equal(lse, plain_lse)
    sees = torch.tensor([x > token for x in lengths], device="cuda")
    assert bool((out[sees][:, 2:, column] == math.inf).all())
    out[sees.nonzero()[:, 0], 2:, column] = plain[sees.nonzero()[:, 0], 2:, column]
    assert torch.equal(out, plain)


@pytest.mark.parametrize("shared", [0, 4])
def test_decode_pages_that_are_not_there(pkg, shared):
    """A page number outside the cache reads as zeros."""
    q, k, v, table, n = cache_case([200, 150, 130], 4, 16, 4, 2, 64, seed=5)
    table[0, 5], table[1, 6], table[2, 7] = -1, 10 ** 8, k.shape[0]
    if shared:
        table[:, 2] = -7
    k.nan_to_num_(0.0), v.nan_to_num_(0.0)
    out, lse = decode(pkg, q, k, v, table, n, shared)
    check_decode(out, lse, q, k, v, table, n, 64 ** -0.5)


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 8, 64), (8, 8, 128), (96, 8, 64), (72, 8, 128), (8, 8, 72)])
def test_decode_many_long_rows_in_a_piece(pkg, heads, kv_heads, dim):
    """A warp's piece of the line has several rows of more than a run of tiles."""
    batch, pool, page = 1200, 48, 64
    g = torch.Generator().manual_seed(dim)
    k, v = (torch.randn(pool, kv_heads, page, dim, generator=g).half() for _ in range(2))
    table = torch.randint(0, pool, (batch, 80), generator=g, dtype=torch.int32)
    lengths = torch.randint(0, 80 * page + 1, (batch,), generator=g, dtype=torch.int32)
    q = torch.randn(batch, heads, dim, generator=g) * 2
    out, lse = decode(pkg, q.cuda(), k.cuda(), v.cuda(), table.cuda(), lengths.cuda())
    some = torch.arange(7, batch, 199)
    check_decode(out[some.cuda()], lse[some.cuda()], q[some], k, v, table[some], lengths[some], dim ** -0.5)
    again, again_lse = decode(pkg, q.cuda(), k.cuda(), v.cuda(), table.cuda(), lengths.cuda())
    assert torch.equal(again, out) and torch.equal(again_lse, lse)


def test_decode_strided_queries_and_stream(pkg):
    q, k, v, table, n = cache_case([77, 300, 5], 0, 16, 4, 2, 64, seed=6)
    wide = torch.randn(3, 9, 64, device="cuda")
    wide[:, 2:6] = q
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, lse = decode(pkg, wide[:, 2:6], k, v, table, n)
    side.synchronize()
    check_decode(out, lse, q, k, v, table, n, 64 ** -0.5)


@pytest.mark.parametrize("batch,heads,kv_heads,dim,n,s1", [
    (160, 8, 8, 64, 65536, 0.3), (160, 8, 8, 128, 65536, 0.7), (160, 96, 8, 128, 65536, 0.3),  # long pieces of the line
    (1, 2, 2, 64, 150000, 0.0), (1, 1, 1, 128, 100000, 0.0),                                   # rows in many parts
])
def test_decode_many_equal_keys(pkg, batch, heads, kv_heads, dim, n, s1):
    """Every page but each row's first is the same one; all values of a column are equal."""
    q, k, v = equal_keys(n, s1, dim, torch.float16, 1, heads, kv_heads)
    v = v[:1].expand(n, kv_heads, dim)
    kp, vp = (torch.stack([x[128:256], x[:128]]).transpose(1, 2).contiguous().cuda() for x in (k, v))
    table = torch.zeros(batch, -(-n // 128), dtype=torch.int32, device="cuda")
    table[:, 0] = 1
    q = q.expand(batch, heads, dim).contiguous()
    out, lse = decode(pkg, q.cuda(), kp, vp, table, ints([n] * batch))
    compare_equal_keys(out, lse, q, k.float(), v.float())


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("shared", [0, 16])
@pytest.mark.parametrize("unit", [1, -1, 32, -32])
def test_decode_scores_of_any_size(pkg, dim, shared, unit):
    batch, n, page = 32, 704, 32
    k, v = large_scores(n, dim, unit, seed=dim)
    kp, vp = (x.half().view(n // page, page, 1, dim).transpose(1, 2).contiguous().cuda() for x in (k, v))
    q = (2.0 ** (4 + torch.arange(batch) % 12) * 1.96875)[:, None, None].expand(batch, 1, dim).contiguous()
    lengths = [max(1, n - 21 * i) for i in range(batch)]
    table = ints([list(range(n // page))] * batch)
    out, lse = decode(pkg, q.cuda(), kp, vp, table, ints(lengths), shared)
    seen = torch.arange(n)[None] < torch.tensor(lengths)[:, None]
    check_largest(out.cpu(), lse.cpu(), q, k, v.half().float(), seen)


@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 64), (8, 1, 128), (20, 2, 40)])
@pytest.mark.parametrize("shared", [0, 5])
def test_decode_out_at_any_address(pkg, shared, heads, kv_heads, dim):
    """Rows written whole, rows joined from parts, and rows joined with a prefix's."""
    lengths = [shared * 16 + n for n in (1, 0, 16, 5000, 33, 700)]
    q, k, v, table, n = cache_case(lengths, shared, 16, heads, kv_heads, dim, seed=13)
    want, want_lse = decode(pkg, q, k, v, table, n, shared)
    check_decode(want, want_lse, q, k, v, table, n, dim ** -0.5)
    for offset in (0, 1, 2, 3, 4, 6):
        place = torch.full((want.numel() + 16,), 3.0, device="cuda")
        out = place[offset:offset + want.numel()].view(want.shape)
        got, lse = decode(pkg, q, k, v, table, n, shared, out=out)
        assert got.data_ptr() == out.data_ptr()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        assert bool((place[:offset] == 3.0).all()) and bool((place[offset + want.numel():] == 3.0).all())


def test_decode_long(pkg):
    q, k, v, table, n = cache_case([20000, 3, 9000], 0, 64, 2, 1, 128, seed=7)
    out, lse = decode(pkg, q, k, v, table, n)
    check_decode(out, lse, q, k, v, table, n, 128 ** -0.5)
    q, k, v, table, n = cache_case([20000, 19200, 19201, 19999], 300, 64, 2, 1, 128, seed=8)
    out, lse = decode(pkg, q, k, v, table, n, 300)
    check_decode(out, lse, q, k, v, table, n, 128 ** -0.5)


# --------------------------------------------------------------------------
# refusals of the torch binding (the C calls' own are tested without a GPU)
# --------------------------------------------------------------------------
def test_refusals(pkg):
    q, k, v = case([10], [10], 4, 2, 64, torch.float16)
    cu = ints([0, 10])
    for bad in (dict(q=q.half()), dict(k=k.float()), dict(q=q.cpu()), dict(q=q[0]), dict(k=k[:, :, :32]),
                dict(k=k[:5]), dict(q=q[:, :3]), dict(cu_k=None), dict(cu_q=cu.long()), dict(cu_k=ints([0, 5, 10])),
                dict(out=torch.empty(10, 4, 64)), dict(out=torch.empty(10, 4, 63, device="cuda")),
                dict(lse=torch.empty(10, device="cuda")), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))):
        a = {**dict(q=q, k=k, v=v, cu_q=cu, cu_k=cu), **bad}
        with pytest.raises((ValueError, TypeError)):
            pkg.comp_attn_f32x16(**a)
    for bad in (dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(out=q)):
        with pytest.raises(pkg.CompError):
            pkg.comp_attn_f32x16(q, k, v, cu, cu, **bad)
    with pytest.raises(pkg.CompError):  # head_dim beyond 128
        pkg.comp_attn_f32x16(*case([4], [4], 1, 1, 136, torch.float16))
    with pytest.raises(pkg.CompError):  # rows of out on top of each other
        pkg.comp_attn_f32x16(q, k, v, cu, cu, out=torch.empty(64, device="cuda").expand(10, 4, 64))
    q, k, v, table, n = cache_case([77, 300, 5], 0, 16, 4, 2, 64)
    for bad in (dict(shared=-1), dict(shared=table.shape[1] + 1), dict(scale=math.inf)):
        with pytest.raises(pkg.CompError):
            pkg.comp_attn_decode_f32x16(q, k, v, table, n, **bad)
    with pytest.raises(pkg.CompError):  # a page size that is not offered
        pkg.comp_attn_decode_f32x16(q, k[:, :, :8].contiguous(), v[:, :, :8].contiguous(), table, n)
    for bad in (dict(q=q[:2]), dict(lengths=n.long()), dict(table=table[0]), dict(k_pages=k.float())):
        with pytest.raises(ValueError):
            pkg.comp_attn_decode_f32x16(**{**dict(q=q, k_pages=k, v_pages=v, table=table, lengths=n), **bad})


def test_arguments_that_cannot_be_taken_as_they_are(pkg):
    """A truth value that raises, a number beyond 32 bits, a negation not carried out."""
    q, k, v = case([10], [10], 4, 2, 64, torch.float16)
    with pytest.raises(RuntimeError):
        pkg.comp_attn_f32x16(q, k, v, causal=torch.ones(2))
    assert torch.equal(pkg.comp_attn_f32x16(q, k, v, causal=torch.ones(1)), pkg.comp_attn_f32x16(q, k, v))
    table, refs = ints([[-1, -1]]), ints([0, 0, 0])
    for size in (2 ** 32 + 16, -2 ** 32 + 16, 2 ** 40):
        with pytest.raises(ValueError):
            pkg.comp_kv_reserve(table, ints([20]), refs, size)
    with pytest.raises(ValueError):
        pkg.comp_attn_f32x16(torch._neg_view(q), k, v)
    want = pkg.comp_attn_f32x16(-q, k, v)
    assert torch.equal(pkg.comp_attn_f32x16(torch._neg_view(q).resolve_neg(), k, v), want)


def test_nothing_to_do(pkg):
    q, k, v = case([0], [0], 4, 2, 64, torch.float16)
    assert pkg.comp_attn_f32x16(q, k, v).shape == (0, 4, 64)
    q, k, v = case([3], [0], 4, 2, 64, torch.float32)
    lse = torch.empty(3, 4, device="cuda")
    assert bool((pkg.comp_attn_f32(q, k, v, lse=lse) == 0).all()) and bool(lse.isneginf().all())


# --------------------------------------------------------------------------
# a workspace of the caller's, and the error's norm
# --------------------------------------------------------------------------
def with_workspace(need, call_it):
    """Exactly `need` bytes between guards, at a 16-byte boundary; nothing beyond them
    changes, fewer or misaligned ones are refused."""
    import compensated_fp32_projection_gb300 as p

    assert need > 0
    place = torch.full((need + 512,), 0x5a, dtype=torch.uint8, device="cuda")
    got = call_it(place[240:240 + need])
    assert bool((place[:240] == 0x5a).all()) and bool((place[240 + need:] == 0x5a).all())
    for bad in (place[240:240 + need - 1], place[244:244 + need]):
        with pytest.raises(p.CompError):
            call_it(bad)
    return got


@pytest.mark.parametrize("lens,heads,kv_heads,dim", [([1], 1, 1, 1), ([150, 37], 6, 2, 72), ([1100, 1200], 2, 1, 128),
                                                     ([513], 4, 4, 64)], ids=str)
@pytest.mark.parametrize("kv", KV, ids=["f16", "f32"])
def test_packed_workspace(pkg, lens, heads, kv_heads, dim, kv):
    import ctypes

    q, k, v = case(lens, lens, heads, kv_heads, dim, kv, seed=15)
    if kv == torch.float16:  # rows that the kernel cannot load where they are
        k, v = (torch.nn.functional.pad(x, (1, 0))[..., 1:] for x in (k, v))
    cu = cu_of(lens)
    want, want_lse = call(pkg, q, k, v, cu, cu, True)
    a = pkg._native.Attn(len(lens), q.shape[0], k.shape[0], heads, kv_heads, dim, 1, 0.5, *q.stride()[:2],
                         *k.stride()[:2], *v.stride()[:2], *want.stride()[:2])
    need = pkg._native.load().comp_attn_workspace_bytes(ctypes.byref(a), k.element_size(), k.data_ptr(), v.data_ptr())
    out, lse = with_workspace(need, lambda ws: call(pkg, q, k, v, cu, cu, True, workspace=ws))
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("shared,page,batch,heads,kv_heads,dim", [
    (0, 16, 3, 4, 2, 64), (0, 64, 9, 32, 2, 128), (5, 16, 40, 4, 2, 64), (64, 128, 33, 4, 2, 64),
    (100, 32, 3, 8, 2, 128), (9, 64, 70, 40, 1, 72), (300, 16, 128, 2, 2, 8)])
def test_decode_workspace(pkg, shared, page, batch, heads, kv_heads, dim):
    import ctypes

    lengths = [shared * page + (97 * i) % 3000 for i in range(batch)]
    q, k, v, table, n = cache_case(lengths, shared, page, heads, kv_heads, dim, seed=16)
    want, want_lse = decode(pkg, q, k, v, table, n, shared)
    c = pkg._native.KvCache(k.data_ptr(), v.data_ptr(), k.shape[0], page, kv_heads, dim)
    need = pkg._native.load().comp_attn_decode_workspace_bytes(ctypes.byref(c), batch, heads, table.shape[1], shared)
    out, lse = with_workspace(need, lambda ws: decode(pkg, q, k, v, table, n, shared, workspace=ws))
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


# The error's norm: a score loses at most 2^-22 of each product by the split of q (and of
# k) and a weight 2^-22, each with a sign of its own, and FP32 sums of up to 128 terms
# and the exponential 2^-22 each: some 1e-6 of the output's norm.  An operand without its
# lo half loses 2^-11, 3e-4 on average; 4e-6, what the projections hold, lies between.
NORM = 4e-6


@pytest.mark.parametrize("kv", KV, ids=["f16", "f32"])
@pytest.mark.parametrize("n,heads,kv_heads,dim", [(900, 4, 2, 64), (900, 4, 2, 128), (2300, 2, 1, 128)])
def test_norm_of_the_error(pkg, kv, n, heads, kv_heads, dim):
    q, k, v = case([n], [n], heads, kv_heads, dim, kv, seed=17, q_scale=1.0)
    out, _ = call(pkg, q, k, v, [0, n], [0, n], False)
    kd, vd = (x.double().repeat_interleave(heads // kv_heads, 1) for x in (k, v))
    want = torch.einsum("hnm,mhd->nhd", (torch.einsum("nhd,mhd->hnm", q.double(), kd) * dim ** -0.5).softmax(-1), vd)
    assert float((out - want).norm() / want.norm()) < NORM


@pytest.mark.parametrize("shared", [0, 20])
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 64), (16, 1, 128)])
def test_norm_of_the_error_decode(pkg, shared, heads, kv_heads, dim):
    q, k, v, table, n = cache_case([2000] * 8, shared, 64, heads, kv_heads, dim, seed=18)
    out, _ = decode(pkg, q / 2, k, v, table, n, shared)
    want = torch.empty_like(out, dtype=torch.float64)
    for b in range(8):
        kd, vd = (x[table[b, :32].long()].transpose(1, 2).flatten(0, 1)[:2000].double().repeat_interleave(
            heads // kv_heads, 1) for x in (k, v))
        p = (torch.einsum("hd,mhd->hm", q[b].double() / 2, kd) * dim ** -0.5).softmax(-1)
        want[b] = torch.einsum("hm,mhd->hd", p, vd)
    assert float((out - want).norm() / want.norm()) < NORM


# --------------------------------------------------------------------------
# offsets beyond 32 bits
# --------------------------------------------------------------------------
@pytest.mark.parametrize("kv", [torch.float16, torch.float32])
def test_packed_strides_beyond_2_31_elements(pkg, kv):
    """Tokens 2^25 elements apart, 70 of them."""
    n, apart = 70, 2 ** 25
    q, k, v = case([n], [n], 4, 2, 128, kv, seed=11)
    want = (pkg.comp_attn_f32 if kv == torch.float32 else pkg.comp_attn_f32x16)(q, k, v)

    def spread(t):
        wide = torch.empty(n, apart, dtype=t.dtype, device="cuda")
        part = wide[:, -t.shape[1] * t.shape[2]:].unflatten(1, t.shape[1:])
        part.copy_(t)
        return part

    q2, k2, v2 = spread(q), spread(k), spread(v)
    out = spread(torch.zeros_like(q))
    got = (pkg.comp_attn_f32 if kv == torch.float32 else pkg.comp_attn_f32x16)(q2, k2, v2, out=out)
    assert torch.equal(got, want)


def test_decode_pages_beyond_2_31_elements(pkg):
    """The same tokens on pages far into a cache of 2^31 elements and more."""
    lengths, shared = [700, 650, 1000, 513], 4
    q, k, v, table, n = cache_case(lengths, shared, 128, 8, 2, 128, seed=12)
    want, want_lse = decode(pkg, q, k, v, table, n, shared)
    far = 2 ** 31 // (2 * 128 * 128) + 5  # the first page's number
    big = [torch.empty(far + k.shape[0], 2, 128, 128, dtype=torch.float16, device="cuda") for _ in range(2)]
    for b, t in zip(big, (k, v)):
        b[far:] = t
    moved = torch.where(table >= 0, table + far, table)
    out, lse = decode(pkg, q, *big, moved, n, shared)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
