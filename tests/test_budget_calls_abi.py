"""More of the rotary and cache-budget entry points through the C ABI, without a device: calls with nothing to do,
and calls whose buffers overlap. Every call here is a no-op or refused: its addresses are not memory."""
import ctypes as C

import pytest

from tests.test_budget_abi import P, L, _rope_call  # noqa: F401


@pytest.mark.parametrize("paged", [False, True])
def test_an_append_of_no_rows_with_queries_is_a_no_op(L, paged):
    """Buffers of no rows have no address: NULL inputs and a NULL q_out are fine."""
    at = P if paged else 0
    for null in (False, True):
        rows = (None, 0, 0, 0) if null else (P, 512, 256, 128)
        assert _rope_call(L, paged, at=at, n=0, k=rows, q=rows, q_out=None) == 0, L.kvq_last_error()
        assert _rope_call(L, paged, at=at, n=0, k=rows, q=rows, q_out=P + 4) == 0


F = 1 << 20                                                # another address nothing reads, far from P


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("dtype,size", [(0, 4), (1, 2)])
def test_rope_store_refuses_a_q_out_that_overlaps_an_input(L, paged, dtype, size):
    """Rows of 2 heads of 128 dims and 3 tokens, in views of one projection of 6 heads."""
    import tests.test_budget_abi as A
    from sub_byte_quantized_gb300._lib import KvqRope, KvqRows
    fn = L.kvq_paged_rope_store if paged else L.kvq_rope_store
    c, rope = (A._paged() if paged else A._cache()), KvqRope(P, 64, 128, 0, None)
    token, head, n = 6 * 128, 128, 3
    q, k, v = (KvqRows(F + i * 2 * head * size, n * token, head, token) for i in range(3))
    end = F + (2 * token + 6 * head) * size                 # behind the projection
    rows = 2 * n * 128 * size                               # bytes of q_out

    def call(q_out):
        return fn(C.byref(c), C.byref(rope), C.byref(k), C.byref(v), C.byref(q), dtype, 2, n, P if paged else 0, q_out, None)
    for at in (F, F + 2 * head * size, F + 4 * head * size, F + token * size, F - 16, F - rows + 16, end - 16):
        assert call(at) == A.EINVAL and b"overlaps" in L.kvq_last_error(), at - F


@pytest.mark.parametrize("paged", [False, True])
def test_weights_refuse_scores_that_overlap_in_part(L, paged):
    import tests.test_budget_abi as A
    kv, stride, rows = 10, 64, 2

    need = (L.kvq_paged_attend_weights_workspace_bytes if paged else L.kvq_attend_weights_workspace_bytes)(
        C.byref(A._paged() if paged else A._cache()), 2, 1, kv, 64)

    def call(d, **kw):                                      # (a workspace one byte short is what is refused after it)
        st = A._weights(L, paged, kv=kv, stride=stride, si=F, so=F + 4 * d, chunk=64, wsb=need - 1, **kw)
        assert st in (A.EINVAL, A.EWORKSPACE)
        return st == A.EINVAL and b"overlap" in L.kvq_last_error()
    for d in range(-4 * stride, 4 * stride + 1, 4):
        meet = d != 0 and any(abs(d - k * stride) < kv for k in range(-(rows - 1), rows))
        assert call(d) == meet, d
    assert not call(4, decay=0.0)                          # scores_in is not read


def test_select_and_compact_refuse_overlaps(L):
    import tests.test_budget_abi as A
    for d in (-16, 0, 16):                                  # lengths of eight sequences: 32 bytes
        assert A._select(L, B=8, keep=F, lens=P, new=P + d) == A.EINVAL
    for d in (-(2 * 20 * 4 - 16), 0, (64 + 60) * 4 - 16 & ~15):   # 2 lists of 20, scores to entry 60 of the second row
        assert A._select(L, scores=F, keep=F + d) == A.EINVAL and b"overlap" in L.kvq_last_error()
    other = A._cache(ptr=2 * P)
    for d in (-16, 16, 64 * 4):
        assert L.kvq_evict_compact(C.byref(A._cache()), C.byref(other), P, 20, 60, F, 64, F + d, 32, None) == A.EINVAL
        assert b"overlap" in L.kvq_last_error()


def test_compact_refuses_a_scores_out_without_scores(L):
    """It would have been left unwritten, in place and into another cache."""
    import tests.test_budget_abi as A
    other = A._cache(ptr=2 * P)
    for dst in (None, C.byref(other)):
        assert L.kvq_evict_compact(C.byref(A._cache()), dst, P, 20, 60, None, 0, F, 32, None) == A.EINVAL
        assert b"scores" in L.kvq_last_error()


@pytest.mark.parametrize("layout", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("paged", [False, True])
def test_the_workspace_of_a_scoring_call_stays_near_the_attentions(L, layout, paged):
    """Long prompts under wide observation windows: the partials of the automatic chunk follow the grid, not rows
    times tokens (512 rows per kv head over 131072 tokens: 68 MB, not 1091). Allowed beside the attention's own
    chunks: four waves of two CTAs of 64 rows on 152 SMs, 4 * 304 * 64 rows of 130 floats, or chunks of 1536 tokens
    of up to 128 rows in a paged pool that the sequences do not fill."""
    import tests.test_budget_abi as A
    for nq in (4, 16, 64, 128, 256):
        for kv in (8000, 131072, 1 << 20):
            if paged:
                c = A._paged(layout, page=1 << 16, pages=16)
                c.n_kv_heads = 8
                plain = L.kvq_paged_attend_workspace_bytes(C.byref(c), 32, nq, kv, 0)
                need = L.kvq_paged_attend_weights_workspace_bytes(C.byref(c), 32, nq, kv, 0)
            else:
                c = A._cache(layout, cap=kv, heads=8)
                plain = L.kvq_attend_workspace_bytes(C.byref(c), 32, nq, kv, 0)
                need = L.kvq_attend_weights_workspace_bytes(C.byref(c), 32, nq, kv, 0)
            longest = 32 * nq * (kv // 8192 + 1) * 130 * 4
            few = 32 * nq * (kv // 1536 + 1) * 130 * 4 if paged and 4 * nq <= 128 else 0
            assert 0 < need <= max(plain, longest, few) + 4 * 304 * 64 * 130 * 4 + (1 << 20), (nq, kv, need, plain)
