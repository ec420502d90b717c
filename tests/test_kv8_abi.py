"""Refusals of the rotary and 8-bit cache calls, before any device work (no GPU needed)."""
import ctypes

import pytest

INVALID = 1
P = ctypes.c_void_p
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from compensated_fp32_projection_gb300 import _native, build

    build.build()
    return _native.load()


def rope(**change):
    from compensated_fp32_projection_gb300 import _native

    f = dict(table=32 * MB, positions=100, rot=64, interleaved=0)
    f.update(change)
    return ctypes.byref(_native.Rope(**f))


def cache(**change):
    from compensated_fp32_projection_gb300 import _native

    f = dict(k=64 * MB, v=65 * MB, k_scale=66 * MB, v_scale=67 * MB, pages=8, page_size=32, kv_heads=2, head_dim=64)
    f.update(change)
    return ctypes.byref(_native.Kv8Cache(**f))


BAD_CACHES = [dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(k=64 * MB + 8),
              dict(v=64 * MB + 4096), dict(k_scale=64 * MB + 64), dict(v_scale=66 * MB + 4), dict(v_scale=67 * MB + 2),
              dict(pages=-1), dict(page_size=8), dict(page_size=24), dict(page_size=256), dict(kv_heads=0),
              dict(kv_heads=70000), dict(head_dim=0), dict(head_dim=8), dict(head_dim=72), dict(head_dim=144),
              dict(pages=1 << 40)]

BAD_ROPES = [dict(table=None), dict(table=32 * MB + 4), dict(positions=-1), dict(rot=0), dict(rot=-2), dict(rot=63),
             dict(rot=66), dict(positions=1 << 60)]


def decode(lib, c=None, heads=4, scale=0.1, table=2 * MB, batch=2, width=4, lengths=3 * MB, r=None, out=4 * MB,
           lse=None, q=MB, q_token=256, ws=128 * MB, ws_bytes=32 * MB):
    return lib.comp_attn_decode_f32x8(c or cache(), P(q), q_token, 64, heads, scale, P(table), batch, width,
                                      P(lengths), r, P(out), P(lse), P(ws), ws_bytes, None)


def append(lib, c=None, total=2, rows=2, width=4, cu=None, start=4 * MB, k=MB, k_token=128, table=3 * MB, r=None):
    return lib.comp_kv8_append_f32(c or cache(), P(k), P(2 * MB), k_token, 64, 128, 64, total, P(table), rows, width,
                                   P(cu), P(start), r, None)


def read(lib, c=None, f16=False, total=2, rows=2, width=4, cu=None, start=4 * MB, k=MB, v=2 * MB, k_token=128,
         v_head=64, table=3 * MB):
    f = lib.comp_kv8_read_f16 if f16 else lib.comp_kv8_read_f32
    return f(c or cache(), P(k), P(v), k_token, 64, 128, v_head, total, P(table), rows, width, P(cu), P(start), None)


@pytest.mark.parametrize("change", BAD_CACHES, ids=str)
def test_cache_descriptor(lib, change):
    c = cache(**change)
    assert decode(lib, c) == INVALID
    assert lib.comp_attn_decode_f32x8_workspace_bytes(c, 2, 4, 4) == 0
    assert append(lib, c) == INVALID
    assert read(lib, c) == INVALID and read(lib, c, f16=True) == INVALID
    assert lib.comp_kv8_fork(c, P(MB), P(2 * MB), P(3 * MB), 2, 4, P(4 * MB), P(5 * MB), 1, P(6 * MB), P(7 * MB),
                             P(8 * MB), P(9 * MB), None) == INVALID
    assert lib.comp_kv8_compact(c, P(MB), P(2 * MB), 2, 4, P(3 * MB), P(4 * MB), P(5 * MB), P(6 * MB), None) == INVALID
    assert lib.comp_kv8_copy_pages(c, P(MB), P(2 * MB), 3, None) == INVALID


@pytest.mark.parametrize("change", BAD_ROPES, ids=str)
def test_rope_descriptor(lib, change):
    r = rope(**change)
    assert append(lib, r=r) == INVALID
    assert decode(lib, r=r) == INVALID
    assert rotate(lib, r=r) == INVALID


def test_decode_arguments(lib):
    need = lib.comp_attn_decode_f32x8_workspace_bytes(cache(), 2, 4, 4)
    assert 0 < need <= 32 * MB
    for bad in (dict(heads=3), dict(heads=0), dict(heads=1 << 17), dict(scale=0.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(table=None), dict(batch=-1), dict(width=-1), dict(lengths=None),
                dict(out=None), dict(q=None), dict(q_token=-1), dict(out=MB), dict(out=64 * MB), dict(out=66 * MB),
                dict(lse=4 * MB), dict(lse=67 * MB), dict(ws_bytes=-1), dict(ws=4 * MB), dict(ws=None),
                dict(ws=128 * MB + 8), dict(ws_bytes=need - 1), dict(r=rope(table=4 * MB)),
                dict(batch=1 << 20, width=1 << 12), dict(c=cache(pages=0, k=None, v=None))):
        assert decode(lib, **bad) == INVALID, bad
    assert decode(lib, batch=0) == 0


def test_append_and_read_arguments(lib):
    for bad in (dict(total=-1), dict(total=3), dict(start=None), dict(k=None), dict(k=64 * MB), dict(k=66 * MB),
                dict(k_token=-1), dict(rows=-1), dict(width=-1), dict(table=None), dict(total=1 << 40)):
        assert append(lib, **bad) == INVALID, bad
        assert read(lib, **bad) == INVALID, bad
    assert append(lib, r=rope(table=64 * MB)) == INVALID
    for bad in (dict(v=MB), dict(k_token=0), dict(v_head=32), dict(k=3 * MB), dict(v=None), dict(v=67 * MB),
                dict(cu=MB, total=9)):
        assert read(lib, **bad) == INVALID, bad
    assert append(lib, total=0, rows=0) == 0 and read(lib, total=0, rows=0) == 0
    assert append(lib, c=cache(pages=0)) == 0   # nowhere to write to


def test_sizes_that_a_grid_does_not_have(lib):
    far = 1 << 44
    for f in (append, read):
        assert f(lib, total=1 << 20, rows=(1 << 30) - 1, width=0 if f is read else 1, cu=far, start=2 * far,
                 table=3 * far) == INVALID
    assert read(lib, f16=True, total=(1 << 31) - 1, rows=(1 << 30) - 100, width=1, cu=far, start=2 * far,
                table=3 * far) == INVALID


def rotate(lib, r=None, x=MB, x_token=256, x_head=64, tokens=10, heads=4, dim=64, positions=None, out=4 * MB,
           out_token=256, out_head=64):
    return lib.comp_rope_f32(r or rope(), P(x), x_token, x_head, tokens, heads, dim, P(positions), 0, P(out),
                             out_token, out_head, None)


def test_rotation_arguments(lib):
    for bad in (dict(x=None), dict(out=None), dict(tokens=-1), dict(heads=0), dict(heads=70000), dict(dim=62),
                dict(dim=0), dict(dim=70000), dict(x_token=-1), dict(out_token=64), dict(out_head=0),
                dict(out=MB, x_token=512), dict(out=MB + 4), dict(out=32 * MB), dict(positions=4 * MB),
                dict(tokens=1 << 40)):
        assert rotate(lib, **bad) == INVALID, bad
    assert lib.comp_rope_f32(None, P(MB), 256, 64, 10, 4, 64, None, 0, P(4 * MB), 256, 64, None) == INVALID
    assert rotate(lib, tokens=0) == 0


def test_table_arguments(lib):
    from compensated_fp32_projection_gb300 import _native

    def make(rot=64, first=0, positions=10, out=MB, **change):
        f = dict(base=1e4, factor=1.0, context=0.0, low=1.0, high=32.0, magnitude=1.0)
        f.update(change)
        return lib.comp_rope_table(ctypes.byref(_native.RopeAngles(**f)), rot, first, positions, P(out), None)

    nan, inf = float("nan"), float("inf")
    for bad in (dict(rot=0), dict(rot=7), dict(rot=-2), dict(rot=1 << 20), dict(first=-1), dict(positions=-1),
                dict(positions=1 << 31), dict(first=1 << 31), dict(out=None), dict(out=MB + 4), dict(base=0.0),
                dict(base=-1.0), dict(base=nan), dict(factor=0.0), dict(factor=inf), dict(magnitude=nan),
                dict(context=-1.0), dict(context=nan), dict(context=100.0, low=4.0, high=4.0),
                dict(context=100.0, low=nan), dict(context=100.0, high=inf)):
        assert make(**bad) == INVALID, bad
    assert lib.comp_rope_table(None, 64, 0, 10, P(MB), None) == INVALID
    assert make(positions=0, out=None) == 0


def test_page_arguments(lib):
    fork = lambda n=1, rows=2, out=6 * MB, refs_out=8 * MB, left=9 * MB: lib.comp_kv8_fork(  # noqa: E731
        cache(), P(MB), P(2 * MB), P(3 * MB), rows, 4, P(4 * MB), P(5 * MB), n, P(out), P(7 * MB), P(refs_out), P(left),
        None)
    for bad in (dict(n=-1), dict(n=40000), dict(rows=-1), dict(out=None), dict(left=None), dict(out=2 * MB),
                dict(left=66 * MB), dict(refs_out=64 * MB), dict(out=67 * MB)):
        assert fork(**bad) == INVALID, bad
    assert lib.comp_kv8_copy_pages(cache(), P(66 * MB), P(2 * MB), 3, None) == INVALID
    assert lib.comp_kv8_copy_pages(cache(), None, P(2 * MB), 3, None) == INVALID
    assert lib.comp_kv8_copy_pages(cache(), None, None, 0, None) == 0


def test_calls_are_offered():
    import compensated_fp32_projection_gb300 as pkg

    for name in ("comp_rope_table", "comp_rope_f32", "comp_kv8_append_f32", "comp_kv8_read_f32", "comp_kv8_read_f16",
                 "comp_attn_decode_f32x8", "comp_kv8_fork", "comp_kv8_compact", "comp_kv8_copy_pages"):
        assert name in pkg.__all__ and callable(getattr(pkg, name))
