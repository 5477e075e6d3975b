"""CPU checks of include/dash_cache.h: symbols, and arguments rejected before any launch."""
import ctypes
import subprocess

import pytest

import adaptive_sparse_hierarchical_b200 as D
from adaptive_sparse_hierarchical_b200 import _lib as L
from adaptive_sparse_hierarchical_b200.build import LIB, build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def test_symbols():
    syms = L.header_symbols(L.CACHE_HEADER)
    assert set(syms) == {"dash_append_q4", "dash_load_q4", "dash_decode_q4", "dash_q4_workspace_size",
                         "dash_pages_workspace_size", "dash_pages_copy", "dash_pages_reserve", "dash_pages_fork",
                         "dash_pages_free", "dash_pages_compact"}
    out = subprocess.run(["nm", "-D", "--defined-only", LIB], capture_output=True, text=True).stdout
    assert set(syms) <= {ln.split()[-1] for ln in out.splitlines() if " T " in ln}


def _p(**kw):
    base = dict(batch=2, seqlen=1024, h_q=8, h_kv=2, d_h=128, chunk=64, alpha=1.5, gamma=2.0, dtype=L.DASH_BF16,
                k_strides=(1024 * 256, 256, 128), v_strides=(1024 * 256, 256, 128))
    base.update(kw)
    return L.params(**base)


def _kv(**kw):
    base = dict(k_codes=4096, k_scales=4096, v_codes=4096, v_scales=4096, k_code_page=2 * 128 * 64,
                k_scale_page=2 * 128 * 4, v_code_page=2 * 128 * 64, v_scale_page=2 * 128 * 4, page_table=4096,
                max_pages=8, page_size=128, num_pages=20, k_exp=0, v_exp=0)
    base.update(kw)
    return L.dash_q4_kv(**base)


def _all(p, kv):
    lib, ws = D.load(), 1 << 40
    return {lib.dash_append_q4(p, kv, 256, 256, 3, 256, 256, 256, 256, 256, None),
            lib.dash_load_q4(p, kv, 256, 0, 3, 256, 256, 256, None),
            lib.dash_decode_q4(p, kv, 256, 256, 256, 256, None, 256, ws, None)}


@pytest.mark.parametrize("kw,code", [
    (dict(h_q=6, h_kv=4), L.DASH_EINVAL), (dict(alpha=1.0), L.DASH_EINVAL), (dict(gamma=-1.0), L.DASH_EINVAL),
    (dict(batch=0), L.DASH_EINVAL), (dict(seqlen=1025), L.DASH_EINVAL),     # 8 pages of 128 do not hold it
    (dict(d_h=96), L.DASH_EUNSUPPORTED), (dict(chunk=48), L.DASH_EUNSUPPORTED), (dict(chunk=1), L.DASH_EUNSUPPORTED),
    (dict(dtype=L.DASH_F32), L.DASH_EUNSUPPORTED), (dict(h_q=6, h_kv=2), L.DASH_EUNSUPPORTED),
])
def test_bad_params(kw, code):
    assert _all(_p(**kw), _kv()) == {code}


@pytest.mark.parametrize("kw,code", [
    (dict(k_codes=None), L.DASH_EINVAL), (dict(v_scales=None), L.DASH_EINVAL), (dict(page_table=None), L.DASH_EINVAL),
    (dict(page_size=0), L.DASH_EINVAL), (dict(num_pages=0), L.DASH_EINVAL), (dict(max_pages=7), L.DASH_EINVAL),
    (dict(k_exp=33), L.DASH_EINVAL), (dict(v_exp=-33), L.DASH_EINVAL), (dict(k_code_page=2 * 128 * 64 - 16), L.DASH_EINVAL),
    (dict(v_scale_page=16), L.DASH_EINVAL), (dict(page_size=160), L.DASH_EUNSUPPORTED),   # not a multiple of the chunk
    (dict(k_code_page=2 * 128 * 64 + 8), L.DASH_EALIGN), (dict(v_codes=4104), L.DASH_EALIGN),
    (dict(k_scales=4100), L.DASH_EALIGN), (dict(page_table=4098), L.DASH_EALIGN),
])
def test_bad_pools(kw, code):
    assert _all(_p(), _kv(**kw)) == {code}


def test_bad_calls():
    lib, p, kv = D.load(), _p(), _kv()
    ws = L.dash_q4_workspace_size(p)
    assert ws > 0 and L.dash_q4_workspace_size(_p(alpha=3.0)) == 0
    append = lambda **a: lib.dash_append_q4(*{**dict(p=p, kv=kv, k=256, v=256, n=3, c=256, qb=256, kb=256, st=256,   # noqa: E731
                                                     sl=256, s=None), **a}.values())
    for name in ("k", "v", "qb", "kb", "st", "sl"):
        assert append(**{name: None}) == L.DASH_EINVAL
    assert append(n=-1) == L.DASH_EINVAL
    assert append(k=264) == L.DASH_EALIGN
    assert append(c=258) == L.DASH_EALIGN
    assert append(p=_p(k_strides=(1024 * 256, 250, 128))) == L.DASH_EALIGN
    assert append(n=0) == L.DASH_OK
    load = lambda **a: lib.dash_load_q4(*{**dict(p=p, kv=kv, st=256, o=0, n=3, sl=256, k=256, v=256, s=None), **a}.values())   # noqa: E731
    for name in ("k", "v", "sl"):
        assert load(**{name: None}) == L.DASH_EINVAL
    assert load(p=_p(k_strides=(1024 * 256, 0, 128))) == L.DASH_EINVAL        # every token in one place
    assert load(p=_p(v_strides=(0, 256, 128))) == L.DASH_EINVAL
    assert load(n=-1) == L.DASH_EINVAL and load(v=260) == L.DASH_EALIGN and load(n=0) == L.DASH_OK
    dec = lambda **a: lib.dash_decode_q4(*{**dict(p=p, kv=kv, q=256, kb=256, sl=256, o=256, r=None, w=256, n=ws, s=None),   # noqa: E731
                                           **a}.values())
    for name in ("q", "kb", "sl", "o"):
        assert dec(**{name: None}) == L.DASH_EINVAL
    assert dec(w=None) == L.DASH_EWORKSPACE and dec(n=ws - 1) == L.DASH_EWORKSPACE
    assert dec(w=384) == L.DASH_EALIGN and dec(q=264) == L.DASH_EALIGN
    assert dec(p=_p(batch=2000), n=1 << 50) == L.DASH_EUNSUPPORTED       # 4000 pairs
    # routing 16 heads of 32768 chunks fits neither way of doing it; dense decoding needs no routing, so only the
    # workspace is missed here, as with 16384 chunks
    big = dict(h_q=32, seqlen=524288, chunk=16)
    assert dec(p=_p(**big), kv=_kv(max_pages=4096), n=1 << 50) == L.DASH_EUNSUPPORTED
    assert dec(p=_p(**big, gamma=0.0), kv=_kv(max_pages=4096), kb=None, n=16) == L.DASH_EWORKSPACE
    big["seqlen"] = 262144
    assert dec(p=_p(**big), kv=_kv(max_pages=4096), n=16) == L.DASH_EWORKSPACE
    assert dec(p=_p(gamma=0.0), kb=None, r=L.route_out(256), n=1 << 50) == L.DASH_EINVAL   # routes asked for
    # more granules than 32 bits number: 2048 pairs of 2^25 tokens
    huge = _p(batch=1024, seqlen=1 << 25, chunk=128, gamma=0.0)
    assert dec(p=huge, kv=_kv(max_pages=1 << 18), kb=None, n=1 << 60) == L.DASH_EUNSUPPORTED
    # a cache shorter than a chunk has no summaries to point to: only the workspace is missed here
    short = dict(p=_p(seqlen=63), kb=None)
    assert dec(**short, n=16) == L.DASH_EWORKSPACE
    assert append(**short, n=0) == L.DASH_OK
    assert append(p=_p(seqlen=64), kb=None, n=0) == L.DASH_EINVAL


def _pg(arrays=(), rows=(), **kw):
    a, r = (L.dash_page_array * len(arrays))(*arrays), (L.dash_row_array * len(rows))(*rows)
    base = dict(batch=4, max_pages=8, page_size=64, num_pages=20, page_table=256, refs=256, seqlens=256, arrays=a, rows=r,
                num_arrays=len(arrays), num_rows=len(rows))
    base.update(kw)
    return L.dash_pages(**base)


A, W = L.dash_page_array, L.dash_row_array


@pytest.mark.parametrize("pg,code", [
    (_pg(batch=0), L.DASH_EINVAL), (_pg(num_pages=0), L.DASH_EINVAL), (_pg(page_size=0), L.DASH_EINVAL),
    (_pg(max_pages=0), L.DASH_EINVAL), (_pg(refs=None), L.DASH_EINVAL), (_pg(page_table=258), L.DASH_EALIGN),
    (_pg(max_pages=1 << 20, page_size=1 << 20), L.DASH_EINVAL), (_pg(num_arrays=-1), L.DASH_EINVAL),
    (_pg([A(None, 64, 64)]), L.DASH_EINVAL), (_pg([A(256, 64, 48)]), L.DASH_EINVAL), (_pg([A(256, 56, 64)]), L.DASH_EALIGN),
    (_pg([A(264, 64, 64)]), L.DASH_EALIGN), (_pg([A(256, 64, 72)]), L.DASH_EALIGN),
    (_pg(rows=[W(None, 64, 16, 16, 2, 1, 0, 0)]), L.DASH_EINVAL), (_pg(rows=[W(256, 62, 16, 16, 2, 1, 0, 0)]), L.DASH_EALIGN),
    (_pg(rows=[W(256, 64, 16, 16, 2, 2, 0, 0)]), L.DASH_EINVAL),    # runs overlap
    (_pg(rows=[W(256, 32, 32, 16, 2, 2, 32, 0)]), L.DASH_EINVAL),   # rows overlap
    (_pg(rows=[W(256, 64, 16, 16, -1, 1, 0, 0)]), L.DASH_EINVAL), (_pg(rows=[W(256, 64, 16, 16, 2, 1, 0, 3)]), L.DASH_EINVAL),
    # sizes whose pieces or slots 32 bits do not number
    (_pg([A(256, 1 << 37, 1 << 37)]), L.DASH_EUNSUPPORTED), (_pg(batch=1 << 20, max_pages=1 << 11), L.DASH_EUNSUPPORTED),
    (_pg(batch=1, max_pages=1 << 26, page_size=16), L.DASH_EUNSUPPORTED),
    (_pg(rows=[W(256, 1 << 50, 1 << 50, 1 << 40, 1, 8, 0, 0)]), L.DASH_EUNSUPPORTED),
    (_pg(rows=[W(256, 1 << 62, 1 << 61, 64, 4, 1, 0, 0)]), L.DASH_EUNSUPPORTED),
])
def test_bad_pages(pg, code):
    lib, ws = D.load(), 1 << 40
    assert lib.dash_pages_workspace_size(pg) == 0
    assert {lib.dash_pages_copy(pg, 256, 256, 1, 256, 256, ws, None), lib.dash_pages_reserve(pg, 256, 0, 256, 256, ws, None),
            lib.dash_pages_fork(pg, 256, 256, 1, 256, 256, ws, None), lib.dash_pages_free(pg, 256, 1, 256, None),
            lib.dash_pages_compact(pg, 256, 256, ws, None)} == {code}


def test_bad_page_calls():
    lib, pg = D.load(), _pg([A(256, 64, 64)])
    ws = lib.dash_pages_workspace_size(pg)
    assert ws > 0
    assert lib.dash_pages_copy(pg, 256, 256, 21, 256, 256, ws, None) == L.DASH_EINVAL     # more than there are pages
    assert lib.dash_pages_copy(pg, None, 256, 2, 256, 256, ws, None) == L.DASH_EINVAL
    assert lib.dash_pages_copy(pg, 256, 256, -1, 256, 256, ws, None) == L.DASH_EINVAL
    assert lib.dash_pages_fork(pg, 256, 256, 5, 256, 256, ws, None) == L.DASH_EINVAL      # more than there are rows
    many = _pg(batch=2000)
    ws2 = lib.dash_pages_workspace_size(many)
    assert lib.dash_pages_fork(many, 256, 256, 1025, 256, 256, ws2, None) == L.DASH_EUNSUPPORTED
    assert lib.dash_pages_free(pg, None, 1, 256, None) == L.DASH_EINVAL
    assert lib.dash_pages_free(pg, 258, 1, 256, None) == L.DASH_EALIGN
    assert lib.dash_pages_copy(pg, 256, 256, 1, 256, 256, ws - 1, None) == L.DASH_EWORKSPACE
    assert lib.dash_pages_compact(pg, 256, None, ws, None) == L.DASH_EWORKSPACE
    assert lib.dash_pages_reserve(pg, 256, 0, 256, 384, ws, None) == L.DASH_EALIGN
    assert lib.dash_pages_copy(pg, 256, 256, 0, 256, 256, ws, None) == L.DASH_OK
    assert lib.dash_pages_free(pg, None, 0, 256, None) == L.DASH_OK
