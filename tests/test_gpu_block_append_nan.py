"""A value that is not a number among the rows of an append to the 8-bit block layouts has an unspecified code of its own; the
other values of its block are stored as if it were 0."""
import numpy as np
import pytest
import torch

import sub_byte_quantized_gb300 as kvq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["int8_b64", "e4m3_b64"])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n", [1, 3, 8, 20, 64])
@pytest.mark.parametrize("slots", [False, True])
def test_the_other_values_of_the_block(layout, D, dtype, n, slots):
    H, first = 3, 64 if n == 64 else 67                    # behind three rows, whose scale grows
    g = torch.Generator("cuda").manual_seed(n)
    lead = torch.randn((1, H, 67, D), device="cuda", generator=g).to(dtype)
    x = (10 * torch.randn((1, H, n, D), device="cuda", generator=g)).to(dtype)
    x[0, 0, n - 1, 8:16] = 200.0                           # the block's largest, of one thread
    x[0, 1, 0, D - 3] = -300.0
    bad = torch.zeros(x.shape, dtype=torch.bool, device="cuda")
    bad[0, 0, n - 1, 11] = bad[0, 1, 0, D - 1] = bad[0, 1, n - 1, 0] = True
    bad[0, 2, 0] = True                                    # a whole row
    caches = []
    for y in (x.masked_fill(bad, 0.0), x.masked_fill(bad, float("nan"))):
        c = kvq.PagedKVCache(layout, 1, H, D, 64, 4, 4)
        c.set_block_table(torch.tensor([[2, 0, 3, 1]]))
        kvq.paged_store(c, lead, lead, torch.zeros(1, dtype=torch.int32, device="cuda"))
        if slots:
            kvq.paged_store_slots(c, y[0].transpose(0, 1), y[0].transpose(0, 1), torch.arange(first - 64, first - 64 + n, device="cuda"))
        else:
            kvq.paged_store(c, y, y, torch.tensor([first], dtype=torch.int32, device="cuda"))
        caches.append(c)
    want, got = caches
    for t in ("k", "v"):
        assert torch.equal(got.planes[t]["scale"], want.planes[t]["scale"])
        at = np.arange(first, first + n)
        pages = torch.as_tensor([[2, 0, 3, 1][p // 64] for p in at], device="cuda")
        rows = torch.as_tensor(at % 64, device="cuda")
        for c in caches:                                   # the codes of the values that are none
            p = c.planes[t]["payload"]
            new = p[pages, :, rows].transpose(0, 1)
            p[pages, :, rows] = new.masked_fill(bad[0], 0).transpose(0, 1)
        assert torch.equal(got.planes[t]["payload"], want.planes[t]["payload"])
