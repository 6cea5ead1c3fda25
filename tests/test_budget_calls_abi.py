"""More of the rotary and cache-budget entry points through the C ABI, without a device: calls with nothing to do,
and calls whose buffers overlap."""
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
