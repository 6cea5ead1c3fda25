"""A row whose attention failed shows in the running scores as well as in the output: NaN, not a share of weight
that is quietly missing. Failure is put in as one key of NaN scale, which leaves the row's sum NaN as the kernels'
own report of a wait that gave up does."""
import numpy as np
import pytest
import torch

import sub_byte_quantized_gb300 as kvq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["q4_0", "q6_0", "q8_0", "asym4_g32", "had_int4", "had_int2", "asym4_g32+q8_0"])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("Hq,nq,dtype", [(2, 1, torch.bfloat16), (8, 2, torch.bfloat16), (4, 20, torch.bfloat16),
                                         (8, 20, torch.bfloat16), (4, 20, torch.float32)])
def test_a_failed_rows_scores_are_nan(layout, D, Hq, nq, dtype):
    """One of two kv heads: 1 to 80 rows each, with and without scores that phase 1 leaves behind."""
    S, H, cut = 300, 2, 200
    w = 40 if layout.startswith("had") else 0
    g = torch.Generator("cuda").manual_seed(Hq)
    k, v = (torch.randn((1, H, S, D), device="cuda", generator=g) for _ in range(2))
    q = torch.randn((1, Hq, nq, D), device="cuda", generator=g).to(dtype)
    c = kvq.KVCache(layout, 1, H, D, S, n_recent=w)
    kvq.store(c, k, v, 0)
    want_out, want = kvq.decode_attend_weights(c, q, S, None, scores_out=torch.zeros((1, H, S), device="cuda"), causal=nq > 1,
                                               q_pos0=cut if nq > 1 else 0)
    want_out, want = want_out.clone(), want.clone()
    c.planes["k"]["scale"][0, 1, 7] = float("nan")
    out, got = kvq.decode_attend_weights(c, q, S, None, scores_out=torch.zeros((1, H, S), device="cuda"), causal=nq > 1,
                                         q_pos0=cut if nq > 1 else 0)
    assert torch.equal(out[:, :Hq // 2], want_out[:, :Hq // 2]) and torch.isnan(out[:, Hq // 2:]).all()
    end = cut + nq if nq > 1 else S                        # tokens that some row sees
    assert torch.equal(got[:, 0], want[:, 0])
    assert torch.isnan(got[0, 1, :end]).all() and not got[0, 1, end:].any()
    assert np.isfinite(want.cpu().numpy()).all()
