"""Selection at the longest caches: 2^18 blocks, which fill the shared memory of a cluster of eight CTAs, and the counts around
which the CTAs of a list change."""
import numpy as np
import pytest
import torch

import sub_byte_quantized_gb300 as kvq
from oracle import quant as Q, serving as OV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_blocks,n_sel,n_q", [(1 << 18, 1000, 1), (1 << 18, 1, 2), (65537, 64, 1), (65536, 64, 3), (8193, 5000, 1)])
@pytest.mark.parametrize("layout", ["had_int2", "q8_0"])
def test_selection_of_the_longest_lists(layout, n_blocks, n_sel, n_q):
    """One kv head, bounds given. The table names few pages again and again, so that many scores are equal and ties decide."""
    D, page, n_pages, heads = 128, 64, 5000, 3
    c = kvq.PagedKVCache(layout, 1, 1, D, page, n_pages, n_blocks)
    rng = np.random.default_rng(n_blocks + n_sel)
    table = rng.integers(0, n_pages, n_blocks)
    c.set_block_table(torch.from_numpy(table)[None])
    b = kvq.BlockBounds(c)
    g = torch.Generator("cuda").manual_seed(7)
    b.codes.copy_(torch.randint(-127, 128, b.codes.shape, device="cuda", generator=g))
    b.scale.copy_(torch.rand(b.scale.shape, device="cuda", generator=g))
    q = torch.randn((1, heads, n_q, D), device="cuda", generator=g).to(torch.bfloat16)
    length = 64 * n_blocks - 3
    sink, recent = (0, 0) if n_sel == 1 else (2, 3)
    sel = kvq.paged_block_select(c, b, q, torch.tensor([length], dtype=torch.int32, device="cuda"), 64 * n_blocks, n_sel, sink, recent)
    qn = q.float().cpu().numpy()
    qr = (Q.rotate(qn) if layout.startswith("had") else qn)[0]
    codes, scale = b.codes[:, 0, 0].cpu().numpy()[table], b.scale[:, 0, 0].cpu().numpy()[table]
    want = OV.select(codes, scale, qr, [length - 1] * n_q, n_sel, sink, recent)
    assert np.array_equal(sel[0, 0].cpu().numpy(), want)
