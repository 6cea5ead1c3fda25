"""The cache-budget operators at the ends of their integer arguments."""
import pytest
import torch

import sub_byte_quantized_gb300 as kvq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_keep", [2 ** 31 - 1, 2 ** 31 - 4097, 2 ** 30 + 3])
def test_a_list_far_longer_than_the_cache(n_keep):
    """Everything stays, -1 fills the list to its end, and nothing is written in front of it."""
    n, pad = 10, 64
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of device memory")
    buf = torch.full((pad + n_keep,), 7, dtype=torch.int32, device="cuda")
    keep = buf[pad:].view(1, 1, n_keep)
    scores = torch.rand((1, 1, n + 2), device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.evict_select(scores, n, n_keep, n_sink=2, n_recent=2 ** 30, keep=keep, new_lens=lens)
    assert lens.item() == n and (buf[:pad] == 7).all()
    assert torch.equal(buf[pad:pad + n], torch.arange(n, dtype=torch.int32, device="cuda"))
    for part in buf[pad + n:].split(1 << 28):
        assert part.min().item() == -1 and part.max().item() == -1
    c = kvq.KVCache("q8_0", 1, 1, 128, n + 2)
    for p in c.planes.values():
        p["payload"].random_(0, 255)
    before = c.planes["v"]["payload"].clone()
    old = scores.clone()
    assert kvq.evict_compact(c, keep, n, scores=scores) == n
    assert torch.equal(before, c.planes["v"]["payload"]) and torch.equal(scores, old)
