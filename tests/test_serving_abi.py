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
