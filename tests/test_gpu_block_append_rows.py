"""append_decode_attend over the 8-bit block layouts with many query rows: the append's growing scales lie next to scales that other
CTAs of the attention, which begin before the append has ended, read."""
import pytest
import torch

import sub_byte_quantized_gb300 as kvq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["int8_b64", "e4m3_b64"])
@pytest.mark.parametrize("chunk", [0, 64])
@pytest.mark.parametrize("paged", [False, True])
def test_one_call_equals_its_parts(layout, chunk, paged):
    B, H, Hq, D, new, n0 = 2, 8, 16, 128, 30, 1500
    g = torch.Generator("cuda").manual_seed(4)
    rnd = lambda h, n, s=1.0: (s * torch.randn((B, h, n, D), device="cuda", generator=g)).to(torch.bfloat16)     # noqa: E731
    cap = 2048
    if paged:
        caches = [kvq.PagedKVCache(layout, B, H, D, 128, B * 16, 16) for _ in range(2)]
        table = torch.randperm(B * 16).reshape(B, 16)
        for c in caches:
            c.set_block_table(table)
    else:
        caches = [kvq.KVCache(layout, B, H, D, cap) for _ in range(2)]
    k, v = rnd(H, n0), rnd(H, n0)
    for c in caches:
        if paged:
            kvq.paged_store(c, k, v, torch.zeros(B, dtype=torch.int32, device="cuda"))
        else:
            kvq.store(c, k, v, 0)
    n = n0
    for step in range(16):
        k, v, q = rnd(H, new, 1.5 ** step), rnd(H, new, 1.5 ** step), rnd(Hq, new)
        n += new
        if paged:
            lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
            kvq.paged_store(caches[0], k, v, lens - new)
            want = kvq.paged_decode_attend(caches[0], q, lens, n, causal=True, chunk=chunk)
            got = kvq.paged_append_decode_attend(caches[1], k, v, q, lens, n, causal=True, chunk=chunk)
        else:
            kvq.store(caches[0], k, v, n - new)
            want = kvq.decode_attend(caches[0], q, n, causal=True, q_pos0=n - new, chunk=chunk)
            got = kvq.append_decode_attend(caches[1], k, v, n - new, q, n, causal=True, q_pos0=n - new, chunk=chunk)
        assert torch.equal(got, want), step
