"""Refusals of the attention and cache calls, before any device work (no GPU needed)."""
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


def attn(**change):
    from compensated_fp32_projection_gb300 import _native

    f = dict(n_seq=1, total_q=10, total_k=12, heads=4, kv_heads=2, head_dim=64, causal=1, scale=0.125, q_token=256,
             q_head=64, k_token=128, k_head=64, v_token=128, v_head=64, out_token=256, out_head=64)
    f.update(change)
    return ctypes.byref(_native.Attn(**f))


def call(lib, a, q=MB, k=2 * MB, v=3 * MB, cu_q=None, cu_k=None, out=4 * MB, lse=None, ws=8 * MB, ws_bytes=4 * MB,
         f32=False):
    f = lib.comp_attn_f32 if f32 else lib.comp_attn_f32x16
    return f(a, P(q), P(k), P(v), P(cu_q), P(cu_k), P(out), P(lse), P(ws), ws_bytes, None)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("change", [dict(n_seq=-1), dict(total_q=-1), dict(total_k=-1), dict(heads=0), dict(kv_heads=0),
                                    dict(heads=3), dict(head_dim=0), dict(head_dim=129), dict(scale=0.0),
                                    dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                                    dict(q_token=-1), dict(k_head=-64), dict(v_token=-5), dict(out_token=255),
                                    dict(out_head=0), dict(n_seq=2), dict(total_q=1 << 40), dict(q_token=1 << 62)],
                         ids=str)
def test_attn_descriptor(lib, change, f32):
    assert call(lib, attn(**change), f32=f32) == INVALID


def test_attn_pointers(lib):
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(cu_q=5 * MB), dict(cu_k=5 * MB),
                dict(out=MB + 64), dict(out=2 * MB), dict(out=3 * MB), dict(lse=4 * MB + 16), dict(lse=MB),
                dict(ws=4 * MB), dict(ws_bytes=-1)):
        assert call(lib, attn(), **bad) == INVALID, bad
    assert call(lib, None) == INVALID
    assert call(lib, attn(total_q=0)) == 0   # nothing to do


def test_attn_workspace(lib):
    need = lambda a, size, k=MB, v=2 * MB: lib.comp_attn_workspace_bytes(a, size, P(k), P(v))  # noqa: E731
    assert need(attn(head_dim=500), 4) == 0 and need(attn(), 3) == 0   # bad arguments
    planes = 12 * 2 * 64 * 2
    assert need(attn(), 2) == 0
    assert need(attn(), 2, k=MB + 2) == need(attn(k_token=129), 2) == need(attn(v_head=0), 2) == 2 * planes
    assert need(attn(), 4) == 4 * planes
    assert call(lib, attn(), f32=True, ws_bytes=4 * planes - 1) == INVALID
    assert call(lib, attn(), f32=True, ws=8 * MB + 8) == INVALID
    assert call(lib, attn(), f32=True, ws=None, ws_bytes=0) == INVALID


def cache(**change):
    from compensated_fp32_projection_gb300 import _native

    f = dict(k=64 * MB, v=65 * MB, pages=8, page_size=16, kv_heads=2, head_dim=64)
    f.update(change)
    return ctypes.byref(_native.KvCache(**f))


BAD_CACHES = [dict(k=None), dict(v=None), dict(k=64 * MB + 8), dict(v=64 * MB + 4096), dict(pages=-1),
              dict(page_size=8), dict(page_size=24), dict(page_size=256), dict(kv_heads=0), dict(head_dim=60),
              dict(head_dim=136), dict(pages=1 << 40)]


@pytest.mark.parametrize("change", BAD_CACHES, ids=str)
def test_cache_descriptor(lib, change):
    c = cache(**change)
    assert lib.comp_attn_decode_f32x16(c, P(MB), 256, 64, 4, 0.1, P(2 * MB), 2, 4, P(3 * MB), 0, P(4 * MB), None,
                                       P(8 * MB), MB, None) == INVALID
    assert lib.comp_kv_append_f32(c, P(MB), P(2 * MB), 128, 64, 128, 64, 2, P(3 * MB), 2, 4, None, P(4 * MB),
                                  None) == INVALID
    assert lib.comp_kv_fork(c, P(MB), P(2 * MB), P(3 * MB), 2, 4, P(4 * MB), P(5 * MB), 1, P(6 * MB), P(7 * MB),
                            P(8 * MB), P(9 * MB), None) == INVALID
    assert lib.comp_kv_compact(c, P(MB), P(2 * MB), 2, 4, P(3 * MB), P(4 * MB), P(5 * MB), P(6 * MB), None) == INVALID
    assert lib.comp_kv_copy_pages(c, P(MB), P(2 * MB), 3, None) == INVALID


def test_decode_arguments(lib):
    def go(heads=4, scale=0.1, table=2 * MB, batch=2, width=4, lengths=3 * MB, shared=0, out=4 * MB, lse=None, q=MB,
           q_token=256, ws=8 * MB, ws_bytes=MB):
        return lib.comp_attn_decode_f32x16(cache(), P(q), q_token, 64, heads, scale, P(table), batch, width,
                                           P(lengths), shared, P(out), P(lse), P(ws), ws_bytes, None)

    for bad in (dict(heads=3), dict(heads=0), dict(scale=0.0), dict(scale=float("nan")), dict(table=None),
                dict(batch=-1), dict(width=-1), dict(lengths=None), dict(shared=-1), dict(shared=5), dict(out=None),
                dict(q=None), dict(q_token=-1), dict(out=MB), dict(out=64 * MB), dict(lse=4 * MB), dict(ws_bytes=-1),
                dict(ws=4 * MB)):
        assert go(**bad) == INVALID, bad
    assert go(batch=0) == 0


def test_sizes_that_cannot_be_counted(lib):
    """Refused as arguments, before a device is asked for or anything is enqueued."""
    far = [i << 44 for i in range(1, 9)]
    for shared in (0, 2):
        for pages_of, heads, want in ((cache(), 4, INVALID), (cache(kv_heads=1), 40, INVALID)):
            assert lib.comp_attn_decode_workspace_bytes(pages_of, 1 << 20, heads, 1 << 12, shared) == 0
            assert lib.comp_attn_decode_f32x16(pages_of, P(far[0]), 64 * heads, 64, heads, 0.1, P(far[1]), 1 << 20,
                                               1 << 12, P(far[2]), shared, P(far[3]), None, P(far[4]), 1 << 40,
                                               None) == want
    assert lib.comp_attn_decode_workspace_bytes(cache(), 1 << 10, 4, 1 << 12, 2) > 0
    for f32 in (False, True):
        assert call(lib, attn(n_seq=(1 << 28) + 1), q=far[0], k=far[1], v=far[2], cu_q=far[3], cu_k=far[4],
                    out=far[5], ws=far[6], f32=f32) == INVALID
        # a tile's last key must be an int
        for keys in (2 ** 31 - 255, 2 ** 31 - 1, 2 ** 31):
            assert call(lib, attn(total_k=keys), q=far[0], k=far[1], v=far[2], out=far[5], ws=far[6],
                        ws_bytes=1 << 42, f32=f32) == INVALID
    assert lib.comp_attn_workspace_bytes(attn(total_k=2 ** 31 - 256), 4, P(far[0]), P(far[1])) > 0


def test_page_arguments(lib):
    fork = lambda n=1, rows=2, width=4, out=6 * MB, lengths_out=7 * MB, refs_out=8 * MB, left=9 * MB, par=4 * MB: \
        lib.comp_kv_fork(cache(), P(MB), P(2 * MB), P(3 * MB), rows, width, P(par), P(5 * MB), n, P(out),
                         P(lengths_out), P(refs_out), P(left), None)  # noqa: E731
    for bad in (dict(n=-1), dict(n=40000), dict(rows=-1), dict(width=-1), dict(out=None), dict(left=None),
                dict(out=MB + 4), dict(out=2 * MB), dict(lengths_out=MB), dict(refs_out=7 * MB), dict(par=None),
                dict(left=6 * MB + 8), dict(refs_out=64 * MB)):
        assert fork(**bad) == INVALID, bad
    free = lambda pages=8, n=1, out=6 * MB, seqs=4 * MB: lib.comp_kv_free(  # noqa: E731
        pages, P(MB), P(2 * MB), P(3 * MB), 2, 4, P(seqs), n, P(out), P(7 * MB), P(8 * MB), None)
    for bad in (dict(pages=-1), dict(n=-1), dict(out=None), dict(out=2 * MB), dict(seqs=None), dict(seqs=6 * MB)):
        assert free(**bad) == INVALID, bad
    reserve = lambda pages=8, size=16, rows=2, want=4 * MB, out=6 * MB: lib.comp_kv_reserve(  # noqa: E731
        pages, size, P(MB), P(3 * MB), rows, 4, P(want), P(out), P(7 * MB), P(8 * MB), None)
    for bad in (dict(pages=-1), dict(size=20), dict(rows=20000), dict(want=None), dict(want=6 * MB), dict(out=3 * MB)):
        assert reserve(**bad) == INVALID, bad
    assert lib.comp_kv_copy_pages(cache(), P(MB), P(2 * MB), -1, None) == INVALID
    assert lib.comp_kv_copy_pages(cache(), None, P(2 * MB), 3, None) == INVALID
    assert lib.comp_kv_copy_pages(cache(), P(64 * MB), P(2 * MB), 3, None) == INVALID
    assert lib.comp_kv_copy_pages(cache(), None, None, 0, None) == 0
    append = lambda total=2, rows=2, cu=None, start=4 * MB, k=MB, k_token=128: lib.comp_kv_append_f32(  # noqa: E731
        cache(), P(k), P(2 * MB), k_token, 64, 128, 64, total, P(3 * MB), rows, 4, P(cu), P(start), None)
    for bad in (dict(total=-1), dict(total=3), dict(start=None), dict(k=None), dict(k=64 * MB), dict(k_token=-1)):
        assert append(**bad) == INVALID, bad
    assert append(total=0, rows=0) == 0
