"""Refusals of the serving-step calls (host validation, no GPU)."""
import ctypes as C

import pytest

EINVAL, ESHAPE, ECAPACITY, EUNSUPPORTED, EALIGN, ECUDA, EWORKSPACE = 1, 2, 3, 4, 5, 6, 7
P = 1 << 20
STEP = 1 << 24                                           # buffers that do not meet


@pytest.fixture(scope="module")
def L():
    import __graft_entry__ as g
    from sub_byte_quantized_gb300 import _lib
    try:
        return _lib.lib()
    except RuntimeError:
        g.build()
        return _lib.lib()


def _cache(layout=0, D=128, cap=64, n_recent=0, ptr=P, batch=1, heads=2):
    from sub_byte_quantized_gb300._lib import KvqCache
    r = ptr if n_recent else None
    return KvqCache(layout, batch, heads, D, cap, n_recent, ptr, ptr, ptr, ptr, ptr, ptr, r, r)


def _paged(layout=0, D=128, n_recent=0, page=64, pages=4, batch=1, heads=2):
    from sub_byte_quantized_gb300._lib import KvqPagedCache
    r = P if n_recent else None
    return KvqPagedCache(layout, batch, heads, D, page, pages, pages, n_recent, P, P, P, P, P, P, r, r, P)


NAMES = ("seq_lens", "new_lens", "table", "free", "n_free", "lens_out", "granted", "n_free_out", "cu_new", "slots", "positions")


def _plan(L, batch=4, page=64, per=8, pool=100, tokens=50, **at):
    p = {n: (i + 1) * STEP for i, n in enumerate(NAMES)} | at
    return L.kvq_page_plan(batch, page, per, p["seq_lens"], p["new_lens"], p["table"], p["free"], pool, p["n_free"], tokens,
                           p["lens_out"], p["granted"], p["n_free_out"], p["cu_new"], p["slots"], p["positions"], None)


def test_plan_refusals(L):
    assert _plan(L, batch=0) == EINVAL and _plan(L, batch=(1 << 20) + 1) == EINVAL
    assert _plan(L, per=0) == EINVAL and _plan(L, pool=0) == EINVAL
    assert _plan(L, tokens=-1) == EINVAL and _plan(L, tokens=(1 << 30) + 1) == EINVAL
    for page in (0, 32, 96, 1 << 21):
        assert _plan(L, page=page) == ESHAPE
    assert _plan(L, page=1 << 20, per=1 << 11) == ECAPACITY
    for n in NAMES:
        assert _plan(L, **{n: None}) == EINVAL
        assert _plan(L, **{n: 50 * STEP + 4}) == EALIGN
    # nothing to map: no map (the launch itself fails here for want of a GPU)
    assert _plan(L, tokens=0, slots=None, positions=None) in (0, ECUDA)


def test_plan_refuses_overlaps_but_in_place(L):
    at = {n: (i + 1) * STEP for i, n in enumerate(NAMES)}
    in_place = {("lens_out", "seq_lens"), ("granted", "new_lens"), ("n_free_out", "n_free")}
    for o in ("table", "free", "lens_out", "granted", "n_free_out", "cu_new", "slots", "positions"):
        for n in NAMES:
            if n == o:
                continue
            got = _plan(L, **{o: at[n]})
            if (o, n) in in_place:
                assert got in (0, ECUDA)
            else:
                assert got == EINVAL, (o, n)
    assert _plan(L, batch=8, lens_out=at["seq_lens"] + 16) == EINVAL               # in part


def _store(L, cache=None, k=(P, 0, 128, 256), v=(P, 0, 128, 256), dtype=1, n=3, slots=P):
    from sub_byte_quantized_gb300._lib import KvqRows
    c = cache if cache is not None else _paged()
    return L.kvq_paged_store_slots(C.byref(c), C.byref(KvqRows(*k)) if k else None, C.byref(KvqRows(*v)) if v else None, dtype, n, slots, None)


def test_store_slots_refusals(L):
    assert _store(L, n=0, k=None, v=None, slots=None) == 0
    assert _store(L, n=-1) == EINVAL and _store(L, dtype=3) == EINVAL and _store(L, k=None) == EINVAL and _store(L, v=None) == EINVAL
    assert _store(L, slots=None) == EINVAL and _store(L, slots=P + 8) == EALIGN
    assert _store(L, k=(P + 8, 0, 128, 256)) == EALIGN and _store(L, v=(P, 0, 128, 252)) == EALIGN and _store(L, k=(P, 0, -128, 256)) == EINVAL
    assert _store(L, cache=_paged(2, n_recent=32)) == EUNSUPPORTED and _store(L, cache=_paged(page=96)) == ESHAPE
    assert _store(L, cache=_paged(heads=1 << 10), n=2 ** 31 - 1) == ESHAPE


@pytest.mark.parametrize("layout", [6, 7])
def test_block_layout_sizes_and_refusals(L, layout):
    from sub_byte_quantized_gb300._lib import KvqCache, KvqRope, KvqRows, mixed
    assert L.kvq_row_bytes(layout, 128) == 128 and L.kvq_row_bytes(layout, 256) == 256 and L.kvq_row_bytes(8, 128) == 0
    out = (C.c_size_t * 4)()
    assert L.kvq_cache_bytes(layout, 2, 3, 128, 192, 0, out) == 0 and list(out) == [2 * 3 * 192 * 128, 2 * 3 * 3 * 4, 0, 0]
    assert L.kvq_cache_bytes(layout, 2, 3, 128, 100, 0, out) == ESHAPE
    assert L.kvq_paged_cache_bytes(layout, 5, 3, 256, 128, 2, 0, out) == 0 and list(out) == [5 * 3 * 128 * 256, 5 * 3 * 2 * 4, 0, 0]
    assert L.kvq_paged_cache_bytes(layout, 5, 3, 256, 32, 2, 0, out) == ESHAPE
    p = C.byref
    store = lambda c: L.kvq_store(p(c), 16, 16, 1, 1, 0, None)                     # noqa: E731
    assert store(_cache(layout, cap=100)) == ESHAPE and store(_cache(layout, D=64)) == ESHAPE
    for bad in (mixed(layout, 4), mixed(0, layout), mixed(6, 7), mixed(7, 6), mixed(2, layout)):
        assert store(_cache(bad)) == EINVAL
    assert store(_cache(layout, n_recent=32)) == EUNSUPPORTED
    c, pg = _cache(layout), _paged(layout)
    r, k = KvqRope(P, 64, 128, 0, None), KvqRows(P, 512, 256, 128)
    assert L.kvq_rope_store(p(c), p(r), p(k), p(k), None, 1, 0, 1, 0, None, None) == EUNSUPPORTED
    assert L.kvq_paged_rope_store(p(pg), p(r), p(k), p(k), None, 1, 0, 1, P, None, None) == EUNSUPPORTED
    assert L.kvq_decode_attend_weights(p(c), P, 1, 2, 1, 10, 0, 0, 0.1, 0, P, P, P, 64, 1.0, P, 1 << 40, None) == EUNSUPPORTED
    assert L.kvq_paged_decode_attend_weights(p(pg), P, 1, 2, 1, P, 10, 0, 0.1, 0, P, P, P, 64, 1.0, P, 1 << 40, None) == EUNSUPPORTED
    assert L.kvq_evict_compact(p(c), None, P, 20, 60, None, 0, None, 0, None) == EUNSUPPORTED
    assert L.kvq_paged_evict_compact(p(pg), P, 20, P, 60, None, 0, None) == EUNSUPPORTED
    assert L.kvq_debug_scores_i32(p(c), P, 1, 2, 1, 10, P, P, None) == EUNSUPPORTED
    ws = L.kvq_attend_workspace_bytes(p(c), 2, 1, 60, 64)
    assert ws > 0 and L.kvq_decode_attend(p(c), 16, 1, 2, 1, 60, 0, 0, 1.0, 64, 16, 256, ws - 1, None) == EWORKSPACE
    assert L.kvq_attend_chunk(p(c), 2, 1, 60, 0) % 64 == 0
    for name in ("kvq_store_q8_0", "kvq_store_q4_0"):
        assert getattr(L, name)(p(c), 16, 16, 1, 1, 0, None) == EUNSUPPORTED
    assert KvqCache is not None


def _bounds(codes=P, scale=P):
    from sub_byte_quantized_gb300._lib import KvqBlockBounds
    return KvqBlockBounds(codes, scale)


BIG = 1 << 40


def _sel(L, paged=False, cache=None, bounds=None, q=P, qdt=1, hq=2, nq=1, lens=P, kv=60, causal=0, q0=0, n=4, sink=1, recent=1, sel=P):
    c = cache if cache is not None else (_paged() if paged else _cache())
    b = C.byref(bounds if bounds is not None else _bounds())
    if paged:
        return L.kvq_paged_block_select(C.byref(c), b, q, qdt, hq, nq, lens, kv, causal, n, sink, recent, sel, None)
    return L.kvq_block_select(C.byref(c), b, q, qdt, hq, nq, kv, causal, q0, n, sink, recent, sel, None)


def _sparse(L, paged=False, cache=None, q=P, qdt=1, hq=2, nq=1, lens=P, kv=60, causal=0, q0=0, scale=0.1, sel=P, n=4, chunk=0, out=P, ws=P, wsb=BIG):
    c = cache if cache is not None else (_paged() if paged else _cache())
    if paged:
        return L.kvq_paged_sparse_attend(C.byref(c), q, qdt, hq, nq, lens, kv, causal, scale, sel, n, chunk, out, ws, wsb, None)
    return L.kvq_sparse_attend(C.byref(c), q, qdt, hq, nq, kv, causal, q0, scale, sel, n, chunk, out, ws, wsb, None)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("f", [_sel, _sparse])
def test_block_calls_refusals(L, f, paged):
    call = lambda **kw: f(L, paged, **kw)                                          # noqa: E731
    assert call(q=None) == EINVAL and call(sel=None) == EINVAL and call(q=P + 4) == EALIGN and call(sel=P + 4) == EALIGN
    assert call(qdt=3) == EINVAL and call(hq=0) == EINVAL and call(nq=0) == EINVAL and call(hq=3) == ESHAPE
    assert call(n=0) == EINVAL and call(kv=0) == EINVAL and call(kv=65 if not paged else 257) == ECAPACITY
    assert call(nq=40000) == ESHAPE                                                # batch * heads * n_q
    cache = _paged if paged else _cache
    assert call(cache=cache(2, n_recent=32)) == EUNSUPPORTED
    if paged:
        assert call(lens=None) == EINVAL and call(lens=P + 4) == EALIGN
    else:
        assert call(causal=1, q0=60) == EINVAL and call(causal=1, q0=-1) == EINVAL and call(cache=_cache(cap=100)) == ESHAPE
    if f is _sel:
        assert call(sink=-1) == EINVAL and call(recent=-1) == EINVAL and call(sink=3, recent=2) == EINVAL and call(sink=2 ** 31 - 1, recent=2 ** 31 - 1) == EINVAL
        assert call(bounds=_bounds(None)) == EINVAL and call(bounds=_bounds(P, None)) == EINVAL and call(bounds=_bounds(P + 8)) == EALIGN
        big = _paged(page=1 << 20, pages=17) if paged else _cache(cap=(1 << 24) + 64)
        assert call(cache=big, kv=(1 << 24) + 1) == ECAPACITY
    else:
        assert call(ws=None) == EINVAL and call(ws=P + 16) == EALIGN and call(wsb=0) == EWORKSPACE
        assert call(scale=float("nan")) == EINVAL and call(chunk=100) == ESHAPE and call(out=None) == EINVAL and call(n=1 << 25) == EINVAL


def test_block_workspaces(L):
    c, pg = _cache(cap=640), _paged(pages=10)
    need = L.kvq_sparse_attend_workspace_bytes(C.byref(c), 4, 3, 5, 64)
    assert need > 0 and L.kvq_sparse_attend_workspace_bytes(C.byref(c), 3, 3, 5, 64) == 0
    assert _sparse(L, cache=c, hq=4, nq=3, n=5, chunk=64, kv=640, wsb=need - 1) == EWORKSPACE
    assert L.kvq_paged_sparse_attend_workspace_bytes(C.byref(pg), 4, 3, 5, 64) == need
    assert L.kvq_sparse_attend_workspace_bytes(C.byref(_cache(cap=100)), 4, 3, 5, 64) == 0


def test_bounds_refusals(L):
    c, pg, b = _cache(), _paged(), _bounds()
    f = lambda first=0, kv=60, cache=c, bounds=b: L.kvq_block_bounds_update(C.byref(cache), C.byref(bounds), first, kv, None)     # noqa: E731
    assert f(60, 60) == 0 and f(-1) == EINVAL and f(61) == EINVAL and f(kv=65) == ECAPACITY
    assert f(bounds=_bounds(None)) == EINVAL and f(bounds=_bounds(P, P + 4)) == EALIGN and f(cache=_cache(cap=100)) == ESHAPE
    assert f(cache=_cache(5, n_recent=16)) == EUNSUPPORTED
    g = lambda lens=P, n=3, bounds=b: L.kvq_paged_block_bounds_update(C.byref(pg), C.byref(bounds), lens, n, None)                # noqa: E731
    assert g(n=0) == 0 and g(n=-1) == EINVAL and g(lens=None) == EINVAL and g(lens=P + 4) == EALIGN and g(bounds=_bounds(P, None)) == EINVAL


@pytest.mark.parametrize("layout", [6, 7])
@pytest.mark.parametrize("n_q", [1, 40, 64])
def test_block_layouts_have_a_balanced_chunk(L, layout, n_q):
    import numpy as np
    c = _paged(layout, pages=16, batch=3)
    lens = np.array([0, 5, 1000], np.int32)
    ch = L.kvq_paged_attend_plan_chunk(C.byref(c), 2, n_q, 1, lens.ctypes.data_as(C.c_void_p))
    assert ch >= 64 and ch % 64 == 0
    zero = np.zeros(3, np.int32)
    assert L.kvq_paged_attend_plan_chunk(C.byref(c), 2, n_q, 1, zero.ctypes.data_as(C.c_void_p)) >= 64
