"""Rotary positions against the formulas in 64 bits and, bit for bit, against 32-bit operations one at a time."""
import math

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


def equal(a, b):
    """The same bits, any NaN for any NaN."""
    a, b = a.cpu(), b.cpu()
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(0.0), b.nan_to_num(0.0))


@pytest.mark.parametrize("rot", [2, 20, 64, 128])
@pytest.mark.parametrize("scaling", [dict(), dict(factor=4.0), dict(base=5e5, factor=8.0, context=8192.0, low=1.0,
                                                                    high=4.0, magnitude=1.2),
                                     dict(base=1e4, factor=0.5, context=300.0, low=-3.0, high=90.0, first=100000)],
                         ids=["plain", "interpolated", "by parts", "far"])
def test_table(pkg, rot, scaling):
    positions = 777
    got = pkg.comp_rope_table(positions, rot, **scaling).cpu().double()
    want, angle = plain.table(positions, rot, **scaling)
    # half a step of 32 bits on values of up to the magnitude; the angle is off by some 2^-52 of itself for
    # each of the power, the blend and the product, on both sides: 16 of them
    tol = scaling.get("magnitude", 1.0) * (2.0 ** -24 + 16 * 2.0 ** -52 * (1 + angle.abs()))[..., None]
    assert got.shape == (positions, rot // 2, 2)
    assert float(((got - want).abs() / tol).max()) <= 1


def test_table_given(pkg):
    t = torch.zeros(5, 8, 2, device="cuda")
    assert pkg.comp_rope_table(5, 16, table=t) is t
    assert torch.equal(t, pkg.comp_rope_table(9, 16)[:5])
    assert torch.equal(pkg.comp_rope_table(4, 16, first=5, device="cuda:0"), pkg.comp_rope_table(9, 16)[5:])
    assert pkg.comp_rope_table(0, 16).shape == (0, 8, 2)


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,dim,rot", [(1, 1, 2, 2), (1, 40, 128, 128), (7, 5, 64, 32), (33, 3, 96, 96),
                                                  (130, 2, 80, 20), (19, 7, 50, 26), (3, 300, 16, 16), (2, 6, 36, 4),
                                                  (5, 2, 300, 256), (4, 33, 1000, 1000), (6, 3, 51, 26),
                                                  (2, 2, 3, 2)])
def test_rotation(pkg, tokens, heads, dim, rot, interleaved, inverse):
    g = torch.Generator().manual_seed(dim + rot)
    angles = pkg.comp_rope_table(500, rot, magnitude=1.1)
    positions = torch.randint(0, 500, (tokens,), generator=g, dtype=torch.int32)
    wide = torch.randn(tokens, heads + 2, dim + 8, generator=g)
    for x in (wide[:, :heads, :dim].contiguous(), wide[:, 1:-1, 4:-4], wide[:, 1:-1, 3:-5],
              wide[:, :heads, :dim].transpose(0, 1).contiguous().transpose(0, 1)):
        want = plain.rotate(x, angles.cpu(), positions.long(), interleaved, inverse)
        # on the device with the same strides
        y = torch.empty(wide.numel() + 64, device="cuda")[1 if x.storage_offset() % 4 else 0:]
        y = torch.as_strided(y, x.shape, x.stride()).copy_(x)
        got = pkg.comp_rope_f32(y, angles, positions.cuda(), interleaved=interleaved, inverse=inverse)
        assert equal(got, want) and equal(y, x)
        assert pkg.comp_rope_f32(y, angles, positions.cuda(), interleaved=interleaved, inverse=inverse, out=y) is y
        assert equal(y, want)


def test_positions_that_are_left_out_or_not_there(pkg):
    angles = pkg.comp_rope_table(10, 32)
    x = torch.randn(12, 3, 48, generator=torch.Generator().manual_seed(0))
    got = pkg.comp_rope_f32(x.cuda(), angles)
    assert equal(got, plain.rotate(x, angles.cpu(), torch.arange(12), False))
    assert got[10:, :, :32].isnan().all() and not got[10:, :, 32:].isnan().any() and not got[:10].isnan().any()
    at = [0, -1, 9, 10, 2 ** 31 - 1, -2 ** 31, 3, 3, 3, 3, 3, 3]
    for interleaved in (False, True):
        got = pkg.comp_rope_f32(x.cuda(), angles, ints(at), interleaved=interleaved)
        assert equal(got, plain.rotate(x, angles.cpu(), torch.tensor(at), interleaved))
    assert pkg.comp_rope_f32(x.cuda(), pkg.comp_rope_table(0, 32))[..., :32].isnan().all()
    assert pkg.comp_rope_f32(x.cuda()[:0], angles).shape == (0, 3, 48)


def test_values_of_any_kind(pkg):
    angles = pkg.comp_rope_table(4, 16)
    x = torch.randn(4, 1, 16, generator=torch.Generator().manual_seed(0))
    x[0, 0, 3], x[1, 0, 9], x[2, 0, 0], x[3] = math.inf, math.nan, 3e38, 1e-42
    got = pkg.comp_rope_f32(x.cuda(), angles)
    assert equal(got, plain.rotate(x, angles.cpu(), torch.arange(4), False))
    assert not got[1, 0, [0, 2, 8, 15]].isnan().any()   # a NaN reaches its pair only


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient(pkg, interleaved):
    """inverse is the gradient: against the formula's transposed matrix, and against differences."""
    g = torch.Generator().manual_seed(3)
    angles = pkg.comp_rope_table(50, 24, magnitude=1.3)
    x, up = torch.randn(6, 2, 40, generator=g), torch.randn(6, 2, 40, generator=g)
    at = torch.randint(0, 50, (6,), generator=g, dtype=torch.int32)
    grad = pkg.comp_rope_f32(up.cuda(), angles, at.cuda(), interleaved=interleaved, inverse=True).cpu().double()
    leaf = x.double().requires_grad_()
    y = plain.rotate(leaf.detach(), angles.cpu().double(), at.long(), interleaved)
    i = torch.arange(12)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + 12)
    c, s = (angles.cpu().double()[at.long()][:, None, :, e] for e in (0, 1))
    y = leaf.clone()
    a, b = leaf[..., one], leaf[..., two]
    y = y.index_copy(2, one, a * c - b * s).index_copy(2, two, b * c + a * s)
    (want,) = torch.autograd.grad((y * up.double()).sum(), leaf)
    # two products and a sum, each off by 2^-24 of values of up to magnitude times the pair's
    assert float((grad - want).abs().max()) <= 4 * 2.0 ** -24 * 1.3 * 2 * float(up.abs().max())
    # the call is linear: a step of 1 in one value changes the sum by that value's gradient
    base = (pkg.comp_rope_f32(x.cuda(), angles, at.cuda(), interleaved=interleaved).cpu().double() * up.double()).sum()
    for t, h, d in ((0, 0, 0), (2, 1, 13), (5, 0, 23), (4, 1, 39)):
        z = x.clone()
        z[t, h, d] += 1
        moved = pkg.comp_rope_f32(z.cuda(), angles, at.cuda(), interleaved=interleaved).cpu().double()
        step = float((z[t, h, d].double() - x[t, h, d].double()))
        # each of the two values that move is rounded, on either side of the difference, thrice
        tol = 12 * 2.0 ** -24 * 1.3 * 8 * float(up.abs().max())
        assert abs(float((moved * up.double()).sum() - base) - step * float(grad[t, h, d])) <= tol


def test_rotated_scores_depend_on_distance(pkg):
    """q at p + n and k at p give the same score for any p."""
    g = torch.Generator().manual_seed(1)
    angles = pkg.comp_rope_table(100000, 64)
    q, k = (torch.randn(1, 1, 64, generator=g).expand(4, 1, 64).contiguous().cuda() for _ in range(2))
    p = ints([0, 17, 5000, 99900])
    s = (pkg.comp_rope_f32(q, angles, p + 99).double() * pkg.comp_rope_f32(k, angles, p).double()).sum((1, 2))
    # each rotated value is off by 2^-24 of the pair for the table and each of three operations: 4 a side
    assert float((s - s[0]).abs().max()) <= 16 * 2.0 ** -24 * float(q[0].norm() * k[0].norm())


def test_refusals(pkg):
    x, t = torch.zeros(4, 2, 16, device="cuda"), torch.zeros(8, 8, 2, device="cuda")
    for bad in (x.half(), x.cpu(), x[0], x.transpose(1, 2), x[..., :14], x[:, :0]):
        with pytest.raises((ValueError, pkg.CompError)):
            pkg.comp_rope_f32(bad, t)
    for bad in (t.double(), t[0], t[..., :1], t.transpose(0, 1), t.cpu(), t[:, :0],
                torch.zeros(8, 9, 2, device="cuda")):
        with pytest.raises(ValueError):
            pkg.comp_rope_f32(x, bad)
    with pytest.raises(TypeError):
        pkg.comp_rope_f32(x, None)
    for at in (ints([0, 1, 2]), ints([0, 1, 2, 3]).long(), ints([[0], [1], [2], [3]])):
        with pytest.raises(ValueError):
            pkg.comp_rope_f32(x, t, at)
    for out in (x[:2], x.half(), torch.zeros(1, 2, 16, device="cuda").expand(4, 2, 16)):
        with pytest.raises((ValueError, pkg.CompError)):
            pkg.comp_rope_f32(x, t, out=out)
    for args, kw in (((4, 3), {}), ((-1, 4), {}), ((4, 4), dict(base=0.0)), ((4, 4), dict(factor=-1.0)),
                     ((4, 4), dict(context=10.0, low=2.0, high=2.0)), ((4, 4), dict(first=-1)),
                     ((4, 4), dict(device="cpu")), ((4, 4), dict(table=t))):
        with pytest.raises((ValueError, pkg.CompError)):
            pkg.comp_rope_table(*args, **kw)
    assert pkg.device_status()[0] == 0


def test_captured_on_another_stream(pkg):
    x = torch.randn(30, 4, 64, device="cuda")
    t = pkg.comp_rope_table(64, 64)
    want = pkg.comp_rope_f32(x, t)
    out = torch.zeros_like(x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    pkg.comp_rope_f32(x, t, out=out, stream=s)
    s.synchronize()
    assert equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.comp_rope_f32(x, t, out=out)
    x.mul_(2)
    graph.replay()
    assert equal(out, 2 * want)
