"""The 8-bit cache over its ranges: values up to the largest numbers, every plan of the decode kernel with
rotated queries, sequence starts that do not ascend."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import kv8_check as plain  # noqa: E402
from test_gpu_kv8 import check, ints, pkg, plain_of, pool, rows_of  # noqa: E402,F401

# Query heads on a key head: up to four, up to eight, up to sixteen, and more.
GROUPS = [(4, 1), (6, 2), (5, 1), (8, 1), (14, 2), (16, 1), (40, 2)]


def largest(cache):
    return max(float((c.abs().amax((2, 3)).float()[..., None] * s.abs()).max()) for c, s in
               ((cache[0], cache[2]), (cache[1], cache[3])))


@pytest.mark.parametrize("heads,kv_heads", GROUPS)
@pytest.mark.parametrize("page,dim", [(16, 128), (64, 64), (32, 48)])
def test_decode_large_values(pkg, heads, kv_heads, page, dim):  # noqa: F811
    """Values up to the largest numbers: sums of many of them leave 32 bits, means do not."""
    lens = [1, 16, 0, 17, 300, 2500]
    pages = sum(-(-n // page) for n in lens)
    table = ints(rows_of(lens, page, pages, seed=3))
    q = torch.randn(len(lens), heads, dim, generator=torch.Generator().manual_seed(dim)).cuda()
    for size in (2.0 ** 75, 2.0 ** 82, 2.0 ** 110, 2.0 ** 127):
        cache = pool(pages, kv_heads, page, dim, seed=heads)
        cache[3].mul_(size / (128 * cache[3].max()))
        out, _ = check(pkg, q, cache, table, ints(lens))
        assert out.isfinite().all()
        # one key: its value; its weight is off by 2^-22 as it enters, and four operations round
        value = plain_of(cache)[1].values(torch.float64)[int(table[0, 0]), :, 0].cuda().repeat_interleave(
            heads // kv_heads, 0)
        assert ((out[0].double() - value).abs() <= 2.0 ** -21 * value.abs()).all()


@pytest.mark.parametrize("heads,kv_heads", GROUPS)
def test_decode_equal_largest_values(pkg, heads, kv_heads):  # noqa: F811
    """The worst of it: the largest number a code and a scale make, for every key and with either sign."""
    dim, n = 64, 6000
    cache = pool(-(-n // 64), kv_heads, 64, dim)
    cache[1].fill_(127)
    cache[3].fill_(2.0 ** 121 * (1 - 2.0 ** -7))
    cache[1][..., 1::2].neg_()
    lens = ints([n])
    table = ints([list(range(len(cache[0])))])
    q = torch.randn(1, heads, dim, generator=torch.Generator().manual_seed(0)).cuda()
    out, _ = check(pkg, q, cache, table, lens)
    assert out.isfinite().all() and (out[..., ::2] > 0).all() and (out[..., 1::2] < 0).all()
    # signs that alternate over the keys
    cache[1][:, :, ::2].neg_()
    out, _ = check(pkg, q, cache, table, lens)
    assert out.isfinite().all()


@pytest.mark.parametrize("heads,kv_heads", GROUPS)
@pytest.mark.parametrize("dim", [64, 128])
def test_decode_large_beside_small_values(pkg, heads, kv_heads, dim):  # noqa: F811
    """Blocks of all sizes from 1e-20 to 1e36, in one sequence and one after the other."""
    page, lens = 32, [1500, 90, 33, 700]
    pages = sum(-(-n // page) for n in lens)
    table = ints(rows_of(lens, page, pages, seed=5))
    q = torch.randn(4, heads, dim, generator=torch.Generator().manual_seed(dim)).cuda()
    for seed in range(3):
        cache = pool(pages, kv_heads, page, dim, seed=seed)
        g = torch.Generator().manual_seed(seed)
        power = torch.randint(-20, 36, cache[3].shape, generator=g).double()
        if seed == 2:                        # every other sequence's values are small
            power.fill_(-20)
            for row in (0, 2):
                at = [p for p in table[row].tolist() if p >= 0]
                power[at] = torch.randint(20, 36, power[at].shape, generator=g).double()
        cache[3].copy_((cache[3].double().cpu() * 10 ** power).float())
        cache[3][0, :, 0] = 0.0
        check(pkg, q, cache, table, ints(lens), scale=0.02)
    # a dimension in which the large blocks have a code of 0 keeps its small values
    cache = pool(pages, kv_heads, page, dim)
    cache[3][::2] *= 1e30
    cache[3][1::2] *= 1e-20
    cache[1][::2, ..., 3] = 0
    out, _ = check(pkg, q, cache, table, ints(lens))
    assert (out[0, :, 3] != 0).all()


@pytest.mark.parametrize("seqs,n,heads,kv_heads,dim", [(5, 70001, 16, 8, 64), (8, 70001, 32, 4, 128),
                                                       (8, 70001, 36, 4, 128), (5, 70001, 8, 8, 128),
                                                       (10, 70001, 32, 4, 64)])
@pytest.mark.parametrize("size", [1.0, 2.0 ** 80, 2.0 ** 121])
def test_decode_long_at_any_size(pkg, seqs, n, heads, kv_heads, dim, size):  # noqa: F811
    """Pieces of several runs of sums, against 64-bit sums; at 2^80 one block in seventy has a scale beyond 2^76."""
    page = 128
    lens = [n - 997 * i for i in range(seqs)]
    need = [-(-m // page) for m in lens]
    cache = pool(sum(need), kv_heads, page, dim, seed=1)
    cache[3].mul_(size)
    assert largest(cache) < 3.4e38
    table = ints(rows_of(lens, page, sum(need), seed=4))
    q = torch.randn(seqs, heads, dim, generator=torch.Generator().manual_seed(0)).cuda()
    lse = torch.empty(seqs, heads, device="cuda")
    out = pkg.comp_attn_decode_f32x8(q, *cache, table, ints(lens), lse=lse)
    assert out.isfinite().all()
    group = heads // kv_heads
    for b, h in ((0, 0), (seqs // 2, group), (seqs - 1, heads - 1)):
        at = table[b, :need[b]].long()
        k, v = ((c[at, h // group].double() * s[at, h // group].double().repeat_interleave(16, 1)[..., None])
                .flatten(0, 1)[:lens[b]] for c, s in ((cache[0], cache[2]), (cache[1], cache[3])))
        plain.check_rows(out[b, h][None].cpu(), lse[b, h][None].cpu(), q[b, h][None].cpu(), k.cpu(), v.cpu(),
                         dim ** -0.5)


@pytest.mark.parametrize("heads,kv_heads", GROUPS)
@pytest.mark.parametrize("dim", [64, 112])
def test_decode_large_values_beside_nan(pkg, heads, kv_heads, dim):  # noqa: F811
    """A code that is not a number costs its own dimension, whatever the others' size; outputs at any address."""
    page, lens = 16, [1500, 40, 1100]
    pages = sum(-(-n // page) for n in lens)
    table = ints(rows_of(lens, page, pages, seed=5))
    q = torch.randn(3, heads, dim, generator=torch.Generator().manual_seed(dim)).cuda()
    cache = pool(pages, kv_heads, page, dim)
    cache[3].mul_(1e36)
    at = int(table[0, 70])
    cache[1][at, :, 3, 7] = -128
    cache[3][at, :, 0].neg_()
    clean = [t.clone() for t in cache]
    clean[1][at, :, 3, 7] = 0
    flat = torch.full((3 * heads * dim + 2,), 5.0, device="cuda")
    out = pkg.comp_attn_decode_f32x8(q, *cache, table, ints(lens), out=flat[1:-1].view(3, heads, dim))
    want, _ = check(pkg, q, clean, table, ints(lens))
    rest = [d for d in range(dim) if d != 7]
    assert torch.equal(out[..., rest], want[..., rest]) and torch.equal(out[1:], want[1:])
    assert out[0, :, 7].isnan().all() and out[0][:, rest].isfinite().all() and flat[0] == 5 and flat[-1] == 5


def test_decode_large_values_in_a_graph(pkg):  # noqa: F811
    """Large and ordinary values in turn, the same workspace, of exactly its size."""
    import ctypes

    from compensated_fp32_projection_gb300 import _native

    lens = [2000, 3, 777]
    cache = pool(200, 2, 16, 64)
    table = ints(rows_of(lens, 16, 200, seed=3))
    q = torch.randn(3, 16, 64, generator=torch.Generator().manual_seed(0)).cuda()
    out = torch.zeros(3, 16, 64, device="cuda")
    c = _native.Kv8Cache(*(t.data_ptr() for t in cache), 200, 16, 2, 64)
    size = _native.load().comp_attn_decode_f32x8_workspace_bytes(ctypes.byref(c), 3, 16, table.shape[1])
    workspace = torch.full((size + 64,), 255, dtype=torch.uint8, device="cuda")
    graph, n = torch.cuda.CUDAGraph(), ints(lens)
    want = pkg.comp_attn_decode_f32x8(q, *cache, table, n)
    with torch.cuda.graph(graph):
        pkg.comp_attn_decode_f32x8(q, *cache, table, n, out=out, workspace=workspace[:size])
    scales = cache[3].clone()
    for power in (0, 123, 0, 110, 123):
        cache[3].copy_(scales * 2.0 ** power)
        graph.replay()
        # powers of two change no bits of the sums
        assert torch.equal(out, want * 2.0 ** power)
    assert (workspace[size:] == 255).all()


@pytest.mark.parametrize("heads,kv_heads", [(5, 1), (7, 1), (8, 1), (14, 2), (64, 8)])
@pytest.mark.parametrize("page,dim", [(16, 128), (32, 64), (64, 112), (128, 80), (16, 16)])
def test_decode_five_to_eight_heads(pkg, heads, kv_heads, page, dim):  # noqa: F811
    lens = [1, 0, 15, 16, 17, 33, 130, 77, 1200]
    pages = sum(-(-n // page) for n in lens)
    cache = pool(pages, kv_heads, page, dim, seed=heads)
    table = ints(rows_of(lens, page, pages, seed=3))
    q = torch.randn(len(lens), heads, dim, generator=torch.Generator().manual_seed(dim)).cuda()
    check(pkg, q, cache, table, ints(lens))
    wide = torch.randn(len(lens), heads + 1, dim + 3, generator=torch.Generator().manual_seed(1)).cuda()
    check(pkg, wide[:, 1:, 2:-1], cache, table, ints(lens), scale=0.3)


@pytest.mark.parametrize("heads,kv_heads", GROUPS)
@pytest.mark.parametrize("dim,rot,interleaved", [(128, 128, False), (128, 128, True), (64, 64, False), (64, 64, True),
                                                 (128, 64, False), (128, 20, True), (96, 96, False), (80, 20, False),
                                                 (48, 48, True), (112, 4, False)])
def test_decode_rotates_queries_of_any_group(pkg, heads, kv_heads, dim, rot, interleaved):  # noqa: F811
    """Queries and angles at any address, against a rotation and sums of their own."""
    lens = [1, 40, 0, 133, 600]
    cache = pool(60, kv_heads, 16, dim)
    table = ints(rows_of(lens, 16, 60, seed=3))
    angles = pkg.comp_rope_table(640, rot, magnitude=0.9)
    q = torch.randn(5, heads, dim, generator=torch.Generator().manual_seed(dim)).cuda()
    check(pkg, q, cache, table, ints(lens), angles, interleaved)
    off = torch.empty(angles.numel() + 2, device="cuda")[2:].view(angles.shape).copy_(angles)  # on 8 bytes, not on 16
    check(pkg, q, cache, table, ints(lens), off, interleaved)
    wide = torch.randn(5, heads, dim + 3, generator=torch.Generator().manual_seed(1)).cuda()[..., 1:-2]
    check(pkg, wide, cache, table, ints(lens), angles, interleaved)
    # a length beyond the pages' table ends where that does, and so does the position
    limit = table.shape[1] * 16
    call = lambda n: pkg.comp_attn_decode_f32x8(q, *cache, table, ints(lens[:4] + [n]), rope=angles,  # noqa: E731
                                                interleaved=interleaved)
    assert torch.equal(call(10000), call(limit)) and call(limit).isfinite().all()
    # a position that the table does not have
    out = pkg.comp_attn_decode_f32x8(q, *cache, table, ints(lens), rope=angles[:599].contiguous(),
                                     interleaved=interleaved)
    assert out[4].isnan().all() and not out[:4].isnan().any()


def test_bad_sequence_starts_write_nothing_else(pkg):  # noqa: F811
    """cu that does not ascend, or leaves the tokens: what stands around the cache and the outputs stays."""
    around = [torch.full((8, 1, 16, 32), 77, dtype=torch.int8, device="cuda") for _ in range(2)]
    around += [torch.full((8, 1, 1), 5.0, device="cuda") for _ in range(2)]
    cache = [t[1:-1] for t in around]
    x = torch.randn(20, 1, 32, generator=torch.Generator().manual_seed(0)).cuda()
    table, start = ints([[0, 1], [2, 3], [4, 5]]), ints([0, 0, 0])
    for cu in ([0, 50, 7, 20], [5, 3, 2, 1], [-7, 3, 30, 90], [20, 20, 20, 20], [0, -2 ** 31, 2 ** 31 - 1, 4]):
        pkg.comp_kv8_append_f32(x, x, *cache, table, start, ints(cu))
        out = torch.full((2, 24, 1, 32), 9.0, device="cuda")
        pkg.comp_kv8_read_f32(*cache, table, start, ints(cu), 20, k=out[0, 2:22], v=out[1, 2:22])
        for t, was in zip(around, (77, 77, 5.0, 5.0)):
            assert (t[0] == was).all() and (t[-1] == was).all()
        assert (out[:, :2] == 9).all() and (out[:, 22:] == 9).all() and out.isfinite().all()
    # ascending, but not from 0: the tokens before belong to no sequence, and those behind read zeros
    out = torch.full((2, 20, 1, 32), 9.0, device="cuda")
    pkg.comp_kv8_append_f32(x, x, *cache, table, start, ints([3, 3, 9, 17]))
    pkg.comp_kv8_read_f32(*cache, table, start, ints([3, 3, 9, 17]), 20, k=out[0], v=out[1])
    k, v = plain_of(cache)
    want = plain.read(k.values(), table.tolist(), [0, 0, 0], [3, 3, 9, 17], 20)
    assert torch.equal(out[0, 3:].cpu(), want[3:]) and torch.equal(out[1, 3:], out[0, 3:])
    # half a step of the largest possible scale, and 2^-21 of 127 steps for the operations
    assert float((out[0, 3:17] - x[3:17]).abs().max()) <= float(x.abs().max()) / 127 * (0.5 + 127 * 2.0 ** -21)
