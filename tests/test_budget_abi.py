"""Host-side checks of the rotary and cache-budget entry points: frequencies against the oracle, and every
refusal, through the C ABI and without a device (a refused call enqueues nothing)."""
import ctypes as C
import math
import os

import numpy as np
import pytest

from oracle import rope as OR

EINVAL, ESHAPE, ECAPACITY, EUNSUPPORTED, EALIGN, ECUDA, EWORKSPACE = 1, 2, 3, 4, 5, 6, 7
P = 4096                                                   # a 256-byte aligned address nothing reads


@pytest.fixture(scope="module")
def L():
    from sub_byte_quantized_gb300 import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from sub_byte_quantized_gb300.build import build_library
        build_library()
    return _lib.lib()


def _freqs(L, rot, base=10000.0, scaling=0, factor=1.0, length=0.0, low=1.0, high=4.0):
    from sub_byte_quantized_gb300._lib import KvqRopeConfig
    cfg = KvqRopeConfig(rot, scaling, base, factor, length, low, high)
    out, mag = (C.c_double * 256)(), C.c_float()
    return L.kvq_rope_frequencies(C.byref(cfg), out, C.byref(mag)), np.array(out[:rot // 2 if rot > 0 else 0]), mag.value


@pytest.mark.parametrize("rot", [16, 48, 128, 256])
@pytest.mark.parametrize("name,kind", [("none", 0), ("linear", 1), ("ntk", 2), ("banded", 3), ("yarn", 4)])
def test_frequencies_match_the_oracle(L, rot, name, kind):
    for base, factor, length, low, high in ((10000.0, 1.0, 4096.0, 1.0, 4.0), (500000.0, 8.0, 8192.0, 1.0, 4.0),
                                            (1e6, 4.0, 32768.0, 1.0, 32.0)):
        st, got, mag = _freqs(L, rot, base, kind, factor, length, low, high)
        want, m = OR.frequencies(rot, base, name, factor, length, low, high)
        assert st == 0
        # pow in double is off by an ulp or so; the ramps repeat a handful of operations
        assert np.allclose(got, want, rtol=1e-14, atol=0) and abs(mag - m) <= 2.0 ** -24 * m


def test_frequency_refusals(L):
    for rot in (0, 8, 24, 272, -16):
        assert _freqs(L, rot)[0] == ESHAPE
    assert _freqs(L, 64, scaling=5)[0] == EINVAL and _freqs(L, 64, scaling=-1)[0] == EINVAL
    for base in (1.0, 0.0, -2.0, math.inf, math.nan):
        assert _freqs(L, 64, base=base)[0] == EINVAL
    for factor in (0.0, -1.0, math.inf, math.nan):
        assert _freqs(L, 64, scaling=1, factor=factor)[0] == EINVAL
        assert _freqs(L, 64, scaling=0, factor=factor)[0] == 0                 # unused there
    for kind in (3, 4):
        assert _freqs(L, 64, scaling=kind, factor=2.0, length=0.0)[0] == EINVAL
        assert _freqs(L, 64, scaling=kind, factor=2.0, length=4096.0, low=4.0, high=4.0)[0] == EINVAL
        assert _freqs(L, 64, scaling=kind, factor=2.0, length=math.nan)[0] == EINVAL
    assert L.kvq_rope_frequencies(None, None, None) == EINVAL


def test_table_refusals(L):
    f = (C.c_double * 32)(*([0.5] * 32))
    bad = (C.c_double * 32)(*([0.5] * 31 + [math.nan]))
    neg = (C.c_double * 32)(*([0.5] * 31 + [-1.0]))
    assert L.kvq_rope_table(f, 64, 0, 0, 1.0, None, None) == 0                  # nothing to write
    assert L.kvq_rope_table(f, 60, 0, 4, 1.0, P, None) == ESHAPE
    assert L.kvq_rope_table(f, 64, -1, 4, 1.0, P, None) == EINVAL
    assert L.kvq_rope_table(f, 64, 0, -1, 1.0, P, None) == EINVAL
    assert L.kvq_rope_table(f, 64, 2 ** 31 - 4, 4, 1.0, P, None) == EINVAL      # past INT32_MAX
    assert L.kvq_rope_table(f, 64, 0, 4, math.inf, P, None) == EINVAL
    assert L.kvq_rope_table(f, 64, 0, 4, 1.0, None, None) == EINVAL
    assert L.kvq_rope_table(None, 64, 0, 4, 1.0, P, None) == EINVAL
    assert L.kvq_rope_table(f, 64, 0, 4, 1.0, P + 4, None) == EALIGN
    assert L.kvq_rope_table(bad, 64, 0, 4, 1.0, P, None) == EINVAL and L.kvq_rope_table(neg, 64, 0, 4, 1.0, P, None) == EINVAL


def _cache(layout=0, D=128, cap=64, n_recent=0, ptr=P, batch=1, heads=2):
    from sub_byte_quantized_gb300._lib import KvqCache
    r = ptr if n_recent else None
    return KvqCache(layout, batch, heads, D, cap, n_recent, ptr, ptr, ptr, ptr, ptr, ptr, r, r)


def _paged(layout=0, D=128, n_recent=0, page=64, pages=4):
    from sub_byte_quantized_gb300._lib import KvqPagedCache
    r = P if n_recent else None
    return KvqPagedCache(layout, 1, 2, D, page, pages, pages, n_recent, P, P, P, P, P, P, r, r, P)


def _rope_call(L, paged=False, rope=(P, 64, 128, 0, None), k=(P, 512, 256, 128), q=(P, 512, 256, 128), dtype=1, hq=2, n=1,
               at=0, q_out=P, cache=None, null_k=False):
    from sub_byte_quantized_gb300._lib import KvqRope, KvqRows
    r, kr = KvqRope(*rope), KvqRows(*k)
    qr = C.byref(KvqRows(*q)) if q else None
    c = cache if cache is not None else (_paged() if paged else _cache())
    fn = L.kvq_paged_rope_store if paged else L.kvq_rope_store
    return fn(C.byref(c), C.byref(r), None if null_k else C.byref(kr), C.byref(kr), qr, dtype, hq, n, at, q_out, None)


@pytest.mark.parametrize("paged", [False, True])
def test_rope_store_refusals(L, paged):
    at = P if paged else 0
    def call(**kw):
        return _rope_call(L, paged, at=kw.pop("at", at), **kw)
    assert call(n=0) == 0 and call(n=0, null_k=True) == 0                        # nothing to append
    assert call(n=0, q=None, hq=0, q_out=None) == 0
    for rot in (0, 8, 100, 144):                                                 # 144 > head_dim
        assert call(rope=(P, 64, rot, 0, None)) == ESHAPE
    assert call(rope=(None, 64, 128, 0, None)) == EINVAL and call(rope=(P, 0, 128, 0, None)) == EINVAL
    assert call(rope=(P + 8, 64, 128, 0, None)) == EALIGN and call(rope=(P, 64, 128, 0, P + 4)) == EALIGN
    assert call(dtype=3) == EINVAL and call(dtype=-1) == EINVAL and call(n=-1) == EINVAL
    assert call(null_k=True) == EINVAL and call(k=(None, 0, 0, 0)) == EINVAL
    assert call(k=(P + 2, 512, 256, 128)) == EALIGN and call(k=(P, 512, 256, 132)) == EALIGN
    assert call(k=(P, -512, 256, 128)) == EINVAL
    assert call(q=(P + 4, 0, 0, 0)) == EALIGN and call(q=(P, 4, 0, 0)) == EALIGN
    assert call(q=None) == EINVAL and call(hq=0) == EINVAL and call(hq=-2) == EINVAL   # q and its heads go together
    assert call(hq=3) == ESHAPE
    assert call(q_out=None) == EINVAL and call(q_out=P + 4) == EALIGN
    assert call(n=65 if not paged else 257) == ECAPACITY
    if paged:
        assert call(at=None) == EINVAL and call(at=P + 4) == EALIGN
        assert call(cache=_paged(page=48)) == ESHAPE
    else:
        assert call(at=-1) == EINVAL and call(at=64) == ECAPACITY
        assert call(cache=_cache(D=96)) == ESHAPE


def test_rope_store_refuses_more_rows_than_a_grid_holds(L):
    c = _cache(cap=2 ** 31 - 1, batch=2 ** 16)
    assert _rope_call(L, cache=c, n=2 ** 31 - 1) == ESHAPE


def _weights(L, paged=False, cache=None, q=P, qdt=1, hq=2, nq=1, kv=10, lens=P, causal=0, q0=0, scale=0.1, chunk=0, out=P, si=P,
             so=P, stride=64, decay=1.0, ws=P, wsb=1 << 40):
    c = cache if cache is not None else (_paged() if paged else _cache())
    if paged:
        return L.kvq_paged_decode_attend_weights(C.byref(c), q, qdt, hq, nq, lens, kv, causal, scale, chunk, out, si, so, stride,
                                                 decay, ws, wsb, None)
    return L.kvq_decode_attend_weights(C.byref(c), q, qdt, hq, nq, kv, causal, q0, scale, chunk, out, si, so, stride, decay, ws, wsb,
                                       None)


@pytest.mark.parametrize("paged", [False, True])
def test_weights_refusals(L, paged):
    def call(**kw):
        return _weights(L, paged, **kw)
    assert call(q=None) == EINVAL and call(out=None) == EINVAL and call(ws=None) == EINVAL and call(so=None) == EINVAL
    assert call(si=P + 4) == EALIGN and call(so=P + 4) == EALIGN and call(ws=P + 16) == EALIGN
    assert call(stride=9) == ESHAPE and call(hq=3) == ESHAPE and call(chunk=100) == ESHAPE
    assert call(decay=math.nan) == EINVAL and call(decay=math.inf) == EINVAL and call(scale=math.nan) == EINVAL
    assert call(kv=0) == EINVAL and call(kv=65 if not paged else 257, stride=1000) == ECAPACITY
    assert call(qdt=3) == EINVAL and call(hq=0) == EINVAL and call(nq=0) == EINVAL
    fn = L.kvq_paged_attend_weights_workspace_bytes if paged else L.kvq_attend_weights_workspace_bytes
    plain = L.kvq_paged_attend_workspace_bytes if paged else L.kvq_attend_workspace_bytes
    c = _paged() if paged else _cache()
    need = fn(C.byref(c), 2, 1, 10, 64)
    assert need >= plain(C.byref(c), 2, 1, 10, 64) + 8 and fn(C.byref(c), 3, 1, 10, 64) == 0 and fn(None, 2, 1, 10, 64) == 0
    assert call(chunk=64, wsb=need - 1) == EWORKSPACE
    if paged:
        assert call(lens=None) == EINVAL and call(lens=P + 4) == EALIGN
    else:
        assert call(causal=1, q0=10) == EINVAL


def _select(L, scores=P, B=1, H=2, stride=64, kv=60, lens=None, keep_n=20, sink=0, recent=0, keep=P, new=None):
    return L.kvq_evict_select(scores, B, H, stride, kv, lens, keep_n, sink, recent, keep, new, None)


def test_select_refusals(L):
    call = lambda **kw: _select(L, **kw)                                          # noqa: E731
    assert call(scores=None) == EINVAL and call(keep=None) == EINVAL
    assert call(scores=P + 4) == EALIGN and call(keep=P + 4) == EALIGN and call(lens=P + 4) == EALIGN and call(new=P + 4) == EALIGN
    assert call(keep_n=0) == EINVAL and call(sink=-1) == EINVAL and call(recent=-1) == EINVAL
    assert call(sink=10, recent=11) == EINVAL and call(sink=2 ** 31 - 1, recent=2 ** 31 - 1) == EINVAL
    assert call(kv=0) == EINVAL and call(kv=65) == ESHAPE and call(kv=2 ** 27 + 1, stride=2 ** 28) == ECAPACITY
    assert call(B=0) == EINVAL and call(H=0) == EINVAL and call(B=2 ** 13, H=2 ** 13) == ESHAPE
    assert call(lens=P, new=P) == EINVAL


def test_compact_refusals(L):
    def call(cache=None, dst=None, keep=P, n=20, kv=60, s=P, ss=64, so=None, os_=0):
        return L.kvq_evict_compact(C.byref(cache if cache is not None else _cache()), C.byref(dst) if dst is not None else None, keep, n,
                                   kv, s, ss, so, os_, None)
    assert call(keep=None) == EINVAL and call(keep=P + 4) == EALIGN and call(n=0) == EINVAL
    assert call(kv=0) == EINVAL and call(kv=65) == ECAPACITY
    assert call(ss=59) == ESHAPE and call(s=P + 4) == EALIGN
    assert call(so=2 * P) == EINVAL                                               # in place: the scores too
    assert call(cache=_cache(2, n_recent=32), n=20) == EINVAL                     # the window's tokens stay
    other = dict(ptr=2 * P)
    assert call(dst=_cache(1, **other)) == ESHAPE and call(dst=_cache(D=256, **other)) == ESHAPE
    assert call(dst=_cache(heads=4, **other)) == ESHAPE and call(dst=_cache(batch=2, **other)) == ESHAPE
    assert call(cache=_cache(2, n_recent=8), dst=_cache(2, n_recent=4, **other)) == ESHAPE
    assert call(dst=_cache(cap=19, **other), so=3 * P, os_=64) == ECAPACITY
    assert call(dst=_cache(**other), so=None) == EINVAL and call(dst=_cache(**other), so=P, os_=64) == EINVAL
    assert call(dst=_cache(**other), so=3 * P, os_=19) == ESHAPE
    assert call(dst=_cache(cap=32)) == EINVAL                                     # the same planes, another capacity
    half = _cache(**other)
    half.k_payload = P
    assert call(dst=half, so=3 * P, os_=64) == EINVAL                             # one plane shared
    c = _paged()
    pc = lambda lens=P, keep=P, n=20, kv=60, s=P, ss=64: L.kvq_paged_evict_compact(C.byref(c), keep, n, lens, kv, s, ss, None)  # noqa: E731
    assert pc(lens=None) == EINVAL and pc(lens=P + 4) == EALIGN and pc(keep=None) == EINVAL and pc(kv=257, ss=300) == ECAPACITY
    assert pc(ss=19) == ESHAPE and pc(n=0) == EINVAL
