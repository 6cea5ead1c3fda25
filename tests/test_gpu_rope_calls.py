"""Rotary appends at the ends of what they are documented for."""
import pytest
import torch

import sub_byte_quantized_gb300 as kvq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("queries", [False, True])
@pytest.mark.parametrize("layout", ["q4_0", "had_int4", "q4_0+q8_0"])
def test_an_append_of_no_rows(layout, queries, paged):
    B, H, D, cap = 2, 2, 128, 128
    n_recent = 16 if layout.startswith("had") else 0
    x = torch.randn((B, H, 3, D), device="cuda").bfloat16()
    f, _ = kvq.rope_frequencies(D)
    table = kvq.rope_table(f, cap)
    if paged:
        c = kvq.PagedKVCache(layout, B, H, D, 64, 4, 2, n_recent=n_recent)
        c.set_block_table(torch.arange(4).view(2, 2))
        at, call = torch.tensor([5, 9], dtype=torch.int32, device="cuda"), kvq.paged_rope_store
    else:
        c, at, call = kvq.KVCache(layout, B, H, D, cap, n_recent=n_recent), cap, kvq.rope_store
    for p in c.planes.values():
        for t in p.values():
            t.copy_(torch.randint(0, 100, t.shape, device="cuda"))
    before = {(k, n): t.clone() for k, p in c.planes.items() for n, t in p.items()}
    none = x[:, :, :0]
    got = call(c, table, none, none, at, q=none if queries else None,
               positions=torch.empty((B, 0), dtype=torch.int32, device="cuda"))
    assert got.shape == (B, H, 0, D) if queries else got is None
    torch.cuda.synchronize()
    for (k, n), t in before.items():
        assert torch.equal(c.planes[k][n], t)


def test_rotated_queries_beside_the_projection_in_one_buffer():
    """q_out right before and right behind the inputs' memory is no overlap; anywhere inside it is refused."""
    B, n, Hq, H, D = 2, 3, 4, 2, 128
    size, out = B * n * (Hq + 2 * H) * D, B * Hq * n * D
    buf = torch.randn(size + 2 * out, device="cuda").bfloat16()
    x = buf[out:out + size].view(B, n, Hq + 2 * H, D).transpose(1, 2)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    f, _ = kvq.rope_frequencies(D)
    table = kvq.rope_table(f, 16)
    c = kvq.KVCache("q4_0", B, H, D, 16)
    want = kvq.rope_store(c, table, k, v, 2, q=q)
    first = {(t, m): y.clone() for t, p in c.planes.items() for m, y in p.items()}
    for at in (0, out + size):
        got = buf[at:at + out].view(B, Hq, n, D)
        assert kvq.rope_store(c, table, k, v, 2, q=q, q_out=got) is got and torch.equal(got, want)
        for (t, m), y in first.items():
            assert torch.equal(c.planes[t][m], y)
    for at in (8, out, out + 8 * D, size + out - 8):
        with pytest.raises(kvq.KvqError, match="overlaps"):
            kvq.rope_store(c, table, k, v, 2, q=q, q_out=buf[at:at + out].view(B, Hq, n, D))
    same = q[:1, :, :1]
    with pytest.raises(kvq.KvqError, match="overlaps"):
        kvq.rope_store(kvq.KVCache("q4_0", 1, H, D, 16), table, k[:1, :, :1], v[:1, :, :1], 2, q=same, q_out=same)
