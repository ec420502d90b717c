"""The paged cache's bookkeeping and data movement, against plain loops."""
import math
import random

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from attn_check import check_decode  # noqa: E402


@pytest.fixture(scope="module")
def pkg():
    import __graft_entry__

    __graft_entry__.build()
    import compensated_fp32_projection_gb300 as p

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return p


def ints(values, shape=None):
    t = torch.tensor(values, dtype=torch.int32, device="cuda")
    return t if shape is None else t.view(shape)


def pool(pages, heads, page, dim, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(pages, heads, page, dim, generator=g).half().cuda() for _ in range(2)]


def bits(t):
    return t.cpu().view(torch.int16)


def random_tables(pages, rows, width, page, seed):
    """Rows of random lengths on distinct pages; refs count them."""
    rng = random.Random(seed)
    order = rng.sample(range(pages), pages)
    table, lengths, refs, at = [], [], [0] * pages, 0
    for _ in range(rows):
        n = rng.choice([0, 1, page, width * page, rng.randint(0, width * page)])
        need = -(-n // page)
        if at + need > pages * 2 // 3:
            n = need = 0
        mine = order[at:at + need]
        at += need
        for p in mine:
            refs[p] += 1
        table.append(mine + [-1] * (width - need))
        lengths.append(n)
    return table, lengths, refs


@pytest.mark.parametrize("heads,page,dim", [(2, 16, 64), (1, 32, 128), (3, 64, 80), (5, 128, 8)])
@pytest.mark.parametrize("in_place", [False, True])
def test_fork_and_free(pkg, heads, page, dim, in_place):
    pages, rows, width = 300, 12, 9
    table, lengths, refs = random_tables(pages, rows, width, page, seed=dim)
    k, v = pool(pages, heads, page, dim)
    empty = [r for r in range(rows) if lengths[r] == 0]
    table += [[-1] * width for _ in range(20)]
    lengths += [0] * 20
    children = [rows + i for i in (7, 3, 19, 0, 12, 5)]
    parents = [r for r in range(rows) if lengths[r] > 0][:5] + empty[:1]
    parents = (parents * 6)[:6]
    kx, vx = k.cpu().clone(), v.cpu().clone()
    want_t, want_l, want_r = [list(r) for r in table], list(lengths), list(refs)
    free = [p for p in range(pages) if refs[p] == 0]
    for a, c in zip(parents, children):
        full, rest = divmod(lengths[a], page)
        want_t[c] = table[a][:full] + [-1] * (width - full)
        for p in table[a][:full]:
            want_r[p] += 1
        if rest:
            p = free.pop(0)
            want_t[c][full] = p
            want_r[p] = 1
            kx[p, :, :rest] = kx[table[a][full], :, :rest]
            vx[p, :, :rest] = vx[table[a][full], :, :rest]
        want_l[c] = lengths[a]
    t, n, r = ints(table), ints(lengths), ints(refs)
    outs = dict(table_out=t, lengths_out=n, refs_out=r) if in_place else {}
    before = [x.clone() for x in (t, n, r)]
    t2, n2, r2, left = pkg.comp_kv_fork(k, v, t, n, r, ints(parents), ints(children), **outs)
    assert t2.tolist() == want_t and n2.tolist() == want_l and r2.tolist() == want_r
    assert left.tolist() == [len(free)]
    assert torch.equal(bits(k), bits(kx)) and torch.equal(bits(v), bits(vx))
    if not in_place:
        assert all(torch.equal(a, b) for a, b in zip((t, n, r), before))
    outs = dict(table_out=t2, lengths_out=n2, refs_out=r2) if in_place else {}
    t3, n3, r3 = pkg.comp_kv_free(t2, n2, r2, ints(children + children[:2]), **outs)  # named twice: given back once
    assert t3.tolist() == table and n3.tolist() == lengths and r3.tolist() == refs
    # everything given back: nothing is referenced
    _, n4, r4 = pkg.comp_kv_free(t3, n3, r3, ints(list(range(rows))))
    assert r4.tolist() == [0] * pages and n4.tolist() == [0] * len(lengths)


@pytest.mark.parametrize("in_place", [False, True])
def test_fork_without_enough_pages_changes_nothing(pkg, in_place):
    page, width = 16, 4
    k, v = pool(4, 2, page, 64)
    kx, vx = k.clone(), v.clone()
    t = ints([[0, 1, -1, -1]] + [[-1] * width] * 3)
    n, r = ints([20, 0, 0, 0]), ints([1, 1, 0, 0])
    want = [x.tolist() for x in (t, n, r)]
    outs = dict(table_out=t, lengths_out=n, refs_out=r) if in_place else {}
    t2, n2, r2, left = pkg.comp_kv_fork(k, v, t, n, r, ints([0, 0, 0]), ints([1, 2, 3]), **outs)
    assert left.tolist() == [-1]
    assert [x.tolist() for x in (t2, n2, r2)] == want
    assert torch.equal(bits(k), bits(kx)) and torch.equal(bits(v), bits(vx))


def test_numbers_out_of_range_are_not_followed(pkg):
    page, width = 16, 3
    k, v = pool(5, 1, page, 64)
    kx = k.clone()
    t = ints([[99, -3, 7], [-1] * width, [-1] * width])
    n, r = ints([10 ** 9, -4, 0]), ints([0, 0, 0, 0, 0])
    t2, n2, r2, left = pkg.comp_kv_fork(k, v, t, n, r, ints([0, 1, -1, 50]), ints([1, 2, 2, 1000]))
    assert left.tolist() == [5] and r2.tolist() == [0] * 5 and torch.equal(bits(k), bits(kx))
    t3, n3, r3 = pkg.comp_kv_free(t, n, r, ints([0, 77, -1]))
    assert r3.tolist() == [0] * 5 and t3.tolist()[0] == [-1] * 3
    pkg.comp_kv_copy_pages(k, v, ints([0, 9, -1, 1]), ints([-2, 2, 3, 5]))
    assert torch.equal(bits(k), bits(kx))
    x = torch.randn(3, 1, 64, device="cuda")
    pkg.comp_kv_append_f32(x, x, k, v, t, ints([0, 5, 10 ** 9]))
    assert torch.equal(bits(k), bits(kx))
    t4, _, _, live = pkg.comp_kv_compact(k, v, t, r)
    assert t4.tolist() == [[-1] * 3] * 3 and live.tolist() == [0]


@pytest.mark.parametrize("gone", [-1, 77])
def test_fork_of_a_page_that_is_not_there(pkg, gone):
    """Such a page reads as zeros; the child's own copy of it must too."""
    page, rest = 32, 9
    k, v = pool(6, 2, page, 64)
    t, n, r = ints([[4, gone], [-1, -1]]), ints([page + rest, 0]), ints([0, 0, 0, 0, 1, 0])
    kx, vx = k.clone(), v.clone()
    kx[0, :, :rest] = 0
    vx[0, :, :rest] = 0
    q = torch.randn(2, 4, 64, device="cuda")
    q[1] = q[0]
    t2, n2, r2, left = pkg.comp_kv_fork(k, v, t, n, r, ints([0]), ints([1]))
    assert t2.tolist() == [[4, gone], [4, 0]] and r2.tolist() == [1, 0, 0, 0, 2, 0] and left.tolist() == [4]
    assert torch.equal(bits(k), bits(kx)) and torch.equal(bits(v), bits(vx))
    lse = torch.empty(2, 4, device="cuda")
    out = pkg.comp_attn_decode_f32x16(q, k, v, t2, n2, lse=lse)
    check_decode(out, lse, q, kx, vx, t2, n2, 64 ** -0.5)


@pytest.mark.parametrize("pages", [1, 7, 300, 2048, 5000, 20011])
@pytest.mark.parametrize("share", [0.0, 0.03, 0.5, 0.97, 1.0])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(pkg, pages, share, in_place):
    rng = random.Random(pages + int(100 * share))
    refs = [rng.choice([1, 2, 9]) if rng.random() < share else 0 for _ in range(pages)]
    live = [p for p in range(pages) if refs[p]]
    table = [rng.sample(live, len(live)) + [-1, pages + 3], [p if refs[p] else -1 for p in live] + [-1, -1]]
    k, v = pool(pages, 1, 16, 16, seed=pages)
    kx, vx = k.cpu().clone(), v.cpu().clone()
    n = len(live)
    holes, movers = [p for p in range(n) if not refs[p]], [p for p in range(n, pages) if refs[p]]
    remap = [p if refs[p] else -1 for p in range(pages)]
    want_r = [r if p < n else 0 for p, r in enumerate(refs)]
    for a, b in zip(movers, holes):
        remap[a] = b
        want_r[b] = refs[a]
    if movers:
        kx[holes], vx[holes] = kx[movers], vx[movers]
    t, r = ints(table), ints(refs)
    outs = dict(table_out=t, refs_out=r) if in_place else {}
    t2, r2, m2, l2 = pkg.comp_kv_compact(k, v, t, r, **outs)
    assert l2.tolist() == [n] and m2.tolist() == remap and r2.tolist() == want_r
    assert t2.tolist() == [[remap[p] if 0 <= p < pages else -1 for p in row] for row in table]
    assert torch.equal(bits(k), bits(kx)) and torch.equal(bits(v), bits(vx))


def test_calls_of_different_size_from_two_threads(pkg):
    """The plan kernels' shared memory grows with the call: a smaller call must not
    take it from a larger one that is about to be launched (C calls: ctypes lets
    the threads run)."""
    import ctypes
    import threading

    lib = pkg._native.load()
    k, v = pool(4, 1, 16, 64)
    c = pkg._native.KvCache(k.data_ptr(), v.data_ptr(), 4, 16, 1, 64)
    torch.cuda.synchronize()
    states = []

    def work(rows, n):
        table, refs, want = (torch.full((m,), x, dtype=torch.int32, device="cuda")
                             for m, x in ((rows, -1), (4, 0), (rows, 0)))
        lens, parents, left = (torch.full((m,), x, dtype=torch.int32, device="cuda")
                               for m, x in ((rows, 0), (n, -1), (1, 7)))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        t, r, w, m, p, f = (x.data_ptr() for x in (table, refs, want, lens, parents, left))
        for _ in range(400):
            states.append(lib.comp_kv_reserve(4, 16, t, r, rows, 1, w, t, r, f, side.cuda_stream))
            states.append(lib.comp_kv_fork(ctypes.byref(c), t, m, r, rows, 1, p, p, n, t, m, r, f, side.cuda_stream))
        side.synchronize()
        assert left.tolist() == [4]

    threads = [threading.Thread(target=work, args=a) for a in ((16384, 32768), (6200, 12400), (7000, 14000))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(states) == 2400 and set(states) == {0}


@pytest.mark.parametrize("in_place", [False, True])
def test_reserve(pkg, in_place):
    pages, width, page = 3000, 40, 16
    rng = random.Random(1)
    order = rng.sample(range(pages), pages)
    table, refs, want, at = [], [0] * pages, [], 0
    for i in range(70):
        n = rng.randint(0, 12)
        mine = order[at:at + n]
        at += n
        for p in mine:
            refs[p] = rng.choice([1, 3])
        table.append(mine + [-1] * (width - n))
        want.append(rng.choice([0, -3, 1, n * page, n * page + 1, rng.randint(0, 600), 10 ** 6]))
    free = iter([p for p in range(pages) if not refs[p]])
    want_t, want_r = [list(x) for x in table], list(refs)
    for row, w in zip(want_t, want):
        have = sum(p >= 0 for p in row)
        for c in range(have, min(width, -(-max(w, 0) // page))):
            row[c] = next(free)
            want_r[row[c]] = 1
    t, r = ints(table), ints(refs)
    outs = dict(table_out=t, refs_out=r) if in_place else {}
    t2, r2, left = pkg.comp_kv_reserve(t, ints(want), r, page, **outs)
    assert t2.tolist() == want_t and r2.tolist() == want_r and left.tolist() == [len(list(free))]
    # more than there are
    t3, r3, left = pkg.comp_kv_reserve(t2, ints([10 ** 9] * 70), r2, page)
    missing = sum(width - sum(p >= 0 for p in row) for row in want_t) - sum(x == 0 for x in want_r)
    if missing > 0:
        assert left.tolist() == [-missing] and torch.equal(t3, t2) and torch.equal(r3, r2)


@pytest.mark.parametrize("heads,page,dim", [(2, 16, 64), (1, 128, 8), (8, 64, 128)])
def test_copy_pages(pkg, heads, page, dim):
    k, v = pool(41, heads, page, dim)
    kx, vx = k.clone(), v.clone()
    both = random.Random(2).sample(range(41), 38)
    src, dst = both[:19], both[19:]
    pkg.comp_kv_copy_pages(k, v, ints(src), ints(dst))
    kx[dst], vx[dst] = kx[src], vx[src]
    assert torch.equal(bits(k), bits(kx)) and torch.equal(bits(v), bits(vx))
    pkg.comp_kv_copy_pages(k, v, ints([]), ints([]))
    assert torch.equal(bits(k), bits(kx))


@pytest.mark.parametrize("lens", [None, [3, 0, 40, 1]])
@pytest.mark.parametrize("pad", [0, 3])
def test_append(pkg, lens, pad):
    heads, page, dim = 3, 16, 40
    k, v = pool(20, heads, page, dim)
    kx, vx = k.cpu().clone(), v.cpu().clone()
    table = [[4, 9, 2, -1], [0, 1, 3, 5], [19, 7, 8, 6], [10, -1, -1, -1]]
    start = [30, 0, 5, 15]
    n = lens or [1] * 4
    x = torch.randn(sum(n), 2 * heads, dim + pad, generator=torch.Generator().manual_seed(3)) * 100
    x[0, 0, :4] = torch.tensor([65519.0, 65520.0, math.nan, 1e-8])
    knew, vnew = x.cuda()[:, :heads, pad:], x.cuda()[:, heads:, pad:]
    t = 0
    for r in range(4):
        for i in range(n[r]):
            page_, slot = table[r][(start[r] + i) // page], (start[r] + i) % page
            kx[page_, :, slot], vx[page_, :, slot] = knew[t].cpu().half(), vnew[t].cpu().half()
            t += 1
    cu = None if lens is None else ints([0] + [sum(n[:i + 1]) for i in range(4)])
    pkg.comp_kv_append_f32(knew, vnew, k, v, ints(table), ints(start), cu)
    for got, want in ((k, kx), (v, vx)):
        got = got.cpu()
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(7.0, 8.0, 9.0), want.nan_to_num(7.0, 8.0, 9.0))


def test_refusals(pkg):
    k, v = pool(8, 2, 16, 64)
    t, n, r = ints([[0, -1], [-1, -1]]), ints([5, 0]), ints([1] + [0] * 7)
    one = ints([0])
    with pytest.raises(ValueError):
        pkg.comp_kv_fork(k, v, t, n, r[:5], one, ints([1]))
    with pytest.raises(ValueError):
        pkg.comp_kv_fork(k, v, t, n, r, one, ints([1, 1]))
    with pytest.raises(ValueError):
        pkg.comp_kv_free(t.long(), n, r, one)
    with pytest.raises(pkg.CompError):  # the output on top of another input
        pkg.comp_kv_fork(k, v, t, n, r, one, ints([1]), lengths_out=t.view(-1)[:2])
    with pytest.raises(pkg.CompError):
        pkg.comp_kv_compact(k, k, t, r)
    with pytest.raises(pkg.CompError):
        pkg.comp_kv_reserve(t, n, r, 24)
    with pytest.raises(ValueError):
        pkg.comp_kv_append_f32(torch.zeros(2, 2, 32, device="cuda"), torch.zeros(2, 2, 32, device="cuda"), k, v, t, n)
    with pytest.raises(ValueError):
        pkg.comp_kv_append_f32(torch.zeros(3, 2, 64, device="cuda"), torch.zeros(3, 2, 64, device="cuda"), k, v, t, n)
    with pytest.raises(ValueError):
        pkg.comp_kv_copy_pages(k, v, one, ints([1, 2]))


def test_pages_beyond_2_31_elements(pkg):
    """New tokens, copies, a fork and a compaction at the far end of a large cache."""
    far = 2 ** 31 // (2 * 128 * 128) + 3
    k, v = (torch.zeros(far + 4, 2, 128, 128, dtype=torch.float16, device="cuda") for _ in range(2))
    new = [torch.randn(130, 2, 128, device="cuda") for _ in range(2)]
    table, start = ints([[far, far + 3, -1], [-1, -1, -1]]), ints([0, 0])
    pkg.comp_kv_append_f32(*new, k, v, table, start, ints([0, 130, 130]))
    for t, x in ((k, new[0]), (v, new[1])):
        assert torch.equal(t[far].transpose(0, 1), x[:128].half())
        assert torch.equal(t[far + 3, :, :2].transpose(0, 1), x[128:].half())
    pkg.comp_kv_copy_pages(k, v, ints([far + 3]), ints([far + 1]))
    assert torch.equal(k[far + 1], k[far + 3]) and torch.equal(v[far + 1], v[far + 3])
    k[far + 1] = 0
    # all pages before are taken, so that the fork's copy goes to the next free one
    refs = torch.ones(far + 4, dtype=torch.int32, device="cuda")
    refs[far + 1:far + 3] = 0
    table, lengths, refs, left = pkg.comp_kv_fork(k, v, table, ints([130, 0]), refs, ints([0]), ints([1]))
    assert left.item() == 1 and table.tolist() == [[far, far + 3, -1], [far, far + 1, -1]]
    assert lengths.tolist() == [130, 130] and refs[far:].tolist() == [2, 1, 0, 1]
    assert torch.equal(k[far + 1, :, :2], k[far + 3, :, :2]) and not k[far + 1, :, 2:].any()
    # only those three are in use then: they move to the front
    kept = [t[p].clone() for t in (k, v) for p in (far, far + 1, far + 3)]
    refs[:far] = 0
    table, refs, remap, live = pkg.comp_kv_compact(k, v, table, refs)
    assert live.item() == 3 and table.tolist() == [[0, 2, -1], [0, 1, -1]] and refs[:4].tolist() == [2, 1, 1, 0]
    assert remap[far:].tolist() == [0, 1, -1, 2] and int((remap >= 0).sum()) == 3
    assert all(torch.equal(a, b) for a, b in zip(kept, [t[p] for t in (k, v) for p in (0, 1, 2)]))
