"""A row of attention over the 8-bit block layouts whose sum is not a number comes back as NaN, never as the zeros of a row
that sees nothing. The failure is put in as a key scale of NaN, which leaves the sums as a wait that gave up leaves them."""
import pytest
import torch

import sub_byte_quantized_gb300 as kvq

pytestmark = pytest.mark.gpu
LAYOUTS = ["int8_b64", "e4m3_b64"]
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
# 1 to 160 rows of a kv head (groups of 8 and of 128), and enough rows for the join by one warp each
SHAPES = [(1, 2, 1, BF16), (2, 8, 2, F16), (1, 8, 10, BF16), (1, 8, 20, BF16), (2, 4, 80, F32), (160, 16, 1, BF16), (10, 8, 40, BF16)]


def _cache(layout, B, H, D, S, page):
    g = torch.Generator("cuda").manual_seed(B + D)
    k, v = (torch.randn((B, H, S, D), device="cuda", generator=g) for _ in range(2))
    cap = (S + 63) // 64 * 64
    if not page:
        c = kvq.KVCache(layout, B, H, D, cap)
        kvq.store(c, k, v, 0)
        return c, c.planes["k"]["scale"]
    per = cap // page + 1
    c = kvq.PagedKVCache(layout, B, H, D, page, B * per, per)
    c.set_block_table(torch.randperm(B * per).reshape(B, per))
    kvq.paged_store(c, k, v, torch.zeros(B, dtype=torch.int32, device="cuda"))
    return c, c.planes["k"]["scale"]


def _set_scale(c, scale, page, b, h, blk):
    if page:
        scale[int(c.block_table[b, blk * 64 // page]), h, blk % (page // 64)] = float("nan")
    else:
        scale[b, h, blk] = float("nan")


def _attend(c, q, S, page, causal, chunk):
    if page:
        lens = torch.full((c.batch,), S, dtype=torch.int32, device="cuda")
        return kvq.paged_decode_attend(c, q, lens, S, causal=causal, chunk=chunk)
    return kvq.decode_attend(c, q, S, causal=causal, q_pos0=S - q.shape[2] if causal else 0, chunk=chunk)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("page", [0, 64, 128])
@pytest.mark.parametrize("B,Hq,nq,dtype", SHAPES)
def test_a_failed_row_is_nan(layout, D, page, B, Hq, nq, dtype):
    """The first block of one head of one sequence: every row of that head, and no other."""
    S, H = 300, 2
    c, scale = _cache(layout, B, H, D, S, page)
    q = torch.randn((B, Hq, nq, D), device="cuda", generator=torch.Generator("cuda").manual_seed(Hq)).to(dtype)
    want = {chunk: _attend(c, q, S, page, nq > 1, chunk).clone() for chunk in (0, 64, 192)}
    _set_scale(c, scale, page, B - 1, 1, 0)
    for chunk, ref in want.items():
        got = _attend(c, q, S, page, nq > 1, chunk)
        assert torch.isfinite(ref).all()
        assert torch.isnan(got[-1, Hq // 2:]).all(), chunk
        assert torch.equal(got[:-1], ref[:-1]) and torch.equal(got[-1, :Hq // 2], ref[-1, :Hq // 2]), chunk


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("Hq,nq", [(2, 5), (4, 80), (16, 80)])
def test_rows_that_do_not_see_the_failure_keep_their_result(layout, D, page, Hq, nq):
    """The last block: causal rows that end in front of it keep their bits, the others are NaN."""
    S, H = 256 + nq // 2, 2
    c, scale = _cache(layout, 1, H, D, S, page)
    q = torch.randn((1, Hq, nq, D), device="cuda", generator=torch.Generator("cuda").manual_seed(Hq)).to(BF16)
    want = {chunk: _attend(c, q, S, page, True, chunk).clone() for chunk in (0, 64)}
    _set_scale(c, scale, page, 0, 1, 4)
    before = 256 - (S - nq)                                # rows whose last token is at most 255
    assert 0 < before < nq
    for chunk, ref in want.items():
        got = _attend(c, q, S, page, True, chunk)
        assert torch.equal(got[:, :Hq // 2], ref[:, :Hq // 2])
        assert torch.equal(got[:, Hq // 2:, :before], ref[:, Hq // 2:, :before])
        assert torch.isnan(got[:, Hq // 2:, before:]).all()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("D,nq", [(128, 1), (128, 6), (128, 80), (256, 6)])
def test_a_query_that_is_not_a_number(layout, D, nq):
    """One row's query: that row, and no other, is NaN."""
    S, H, Hq = 300, 2, 4
    c, _ = _cache(layout, 1, H, D, S, 0)
    q = torch.randn((1, Hq, nq, D), device="cuda", generator=torch.Generator("cuda").manual_seed(3)).to(BF16)
    ref = _attend(c, q, S, 0, False, 0).clone()
    q[0, 1, nq // 2, 17] = float("nan")
    got = _attend(c, q, S, 0, False, 0)
    assert torch.isnan(got[0, 1, nq // 2]).all()
    ref[0, 1, nq // 2] = got[0, 1, nq // 2] = 0
    # a row's reference maximum may follow another row's: the same result to float32
    assert (got - ref).norm() <= 1e-5 * ref.norm() and torch.isfinite(got).all()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("Hq,nq", [(2, 1), (8, 3), (96, 2)])
def test_failed_rows_of_sparse_attention(layout, Hq, nq):
    """Rows whose list names the failed block are NaN, the others keep their bits."""
    S, H, D = 640, 2, 128
    c, scale = _cache(layout, 1, H, D, S, 64)
    q = torch.randn((1, Hq, nq, D), device="cuda", generator=torch.Generator("cuda").manual_seed(Hq)).to(BF16)
    lens = torch.tensor([S], dtype=torch.int32, device="cuda")
    sel = torch.tensor([1, 4, 7], dtype=torch.int32, device="cuda").repeat(1, H, nq, 1)
    sel[0, 1, 0] = torch.tensor([2, 3, 5])
    ref = kvq.paged_sparse_attend(c, q, sel, lens, S).clone()
    _set_scale(c, scale, 64, 0, 1, 3)
    got = kvq.paged_sparse_attend(c, q, sel, lens, S)
    assert torch.isnan(got[0, Hq // 2:, 0]).all()
    assert torch.equal(got[0, :Hq // 2], ref[0, :Hq // 2]) and torch.equal(got[0, Hq // 2:, 1:], ref[0, Hq // 2:, 1:])
