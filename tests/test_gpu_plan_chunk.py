"""Attention with the balanced chunk of a batch whose query rows take more CTAs than the GPU holds."""
import pytest
import torch

import sub_byte_quantized_gb300 as kvq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout,D,n_q", [("int8_b64", 256, 512), ("e4m3_b64", 128, 4096), ("q6_0", 256, 512)])
def test_attention_with_the_balanced_chunk(layout, D, n_q):
    B, H, Hq, S, page = 2, 1, 8, 700, 64
    g = torch.Generator("cuda").manual_seed(1)
    c = kvq.PagedKVCache(layout, B, H, D, page, B * 11, 11)
    c.set_block_table(torch.randperm(B * 11).reshape(B, 11))
    k, v = (torch.randn((B, H, S, D), device="cuda", generator=g) for _ in range(2))
    kvq.paged_store(c, k, v, torch.zeros(B, dtype=torch.int32, device="cuda"))
    q = torch.randn((B, Hq, n_q, D), device="cuda", generator=g).to(torch.bfloat16)
    lens = [S, 130]
    d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    chunk = kvq.paged_attend_plan_chunk(c, Hq, n_q, lens)
    got = kvq.paged_decode_attend(c, q, d, S, chunk=chunk)
    want = kvq.paged_decode_attend(c, q, d, S)
    # two splits of one sum, each within 1e-5 of it (Q6_0's probabilities have f16's subnormals: 4e-5)
    assert (got - want).norm() <= (8e-5 if layout == "q6_0" else 2e-5) * want.norm()
