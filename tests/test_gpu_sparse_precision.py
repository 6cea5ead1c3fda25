"""Sparse attention is held to float32 in every layout and for every number of query heads of a kv head, with values of any
size: its error, as a share of the output's norm, against the oracle in 64 bits."""
import numpy as np
import pytest
import torch

import sub_byte_quantized_gb300 as kvq
from oracle import attention as OA, budget as OB
from tests.test_gpu_budget_precision import H, S, TOP_CODE, _inputs, _sums

pytestmark = pytest.mark.gpu
# (layout, head_dim, query heads of a kv head): the decode kernels, the row-side kernel, the tcgen05 kernel
CASES = [("q6_0", 128, 1), ("q6_0", 128, 8), ("q6_0", 256, 1), ("q6_0", 256, 8)]
CASES += [(layout, 128, heads) for layout in ("q4_0", "q8_0", "q4_0+q8_0", "had_int4", "had_int2", "asym4_g32") for heads in (4, 12, 32)]
CASES += [("q6_0", 128, 12), ("had_int4", 128, 80), ("had_int2", 128, 160)]
CASES += [(layout, 128, heads) for layout in ("asym4_g32+q8_0", "had_int2+had_int4") for heads in (1, 12, 40)]


@pytest.mark.parametrize("layout,D,heads", CASES)
@pytest.mark.parametrize("std,sink", [(1.0, False), (0.001, False), (1.0, True)])
def test_sparse_output_with_values_of_any_size(layout, D, heads, std, sink):
    """All blocks of 4096 tokens listed, in chunks of 256. The tolerance is that of scoring attention
    (test_gpu_budget_precision._check), whose kernels these are: random signs of the values, an error e of each
    token's weight and of the sum of all, P' in two f16 parts, the tensor cores' sums, and two roundings of 2^-25 in
    P' for p taken 2^12 times larger. (Fewer than nine rows of a mixed pair without a decode kernel add 16 tokens of
    four warps each, as 9 to 16 do.)"""
    k, v, qd, alpha = _inputs(std, sink, heads, 1, D)
    q = qd.float().numpy()
    dc, oc = kvq.KVCache(layout, 1, H, D, S), OA.OracleCache(layout, 1, H, D, S)
    kvq.store(dc, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), 0)
    oc.store(k, v, 0)
    sel = torch.arange(S // 64, dtype=torch.int32, device="cuda").repeat(1, H, 1, 1)
    out = kvq.sparse_attend(dc, qd.cuda(), sel, S, attn_scale=float(alpha), chunk=256)
    s, mass = OB.scores_dense(oc, q, alpha, S)
    err = 2 * (float(mass.max()) * ((D // 16 + D // 32 + 4) * 2.0 ** -23 + 2.0 ** -22)
               + 3 * 2.0 ** -24 * 1.5 * float(s.max() - s.min()) + 2.0 ** -22)
    l = np.exp(s - s.max(-1, keepdims=True)).sum(-1)
    low = 2 * 2.0 ** -37 * TOP_CODE[layout.split("+")[-1]] * np.sqrt(S * D * ((1 / l) ** 2).sum())
    ref = oc.attend(q, alpha, S)
    ref = ref[0] if isinstance(ref, tuple) else ref
    norm = np.linalg.norm(ref)
    tol = 1.5 * (err + 2.0 ** -21 + _sums(layout, D, heads, 256)) * norm + low
    got = np.linalg.norm(out.cpu().numpy().astype(np.float64) - ref)
    print(f"{layout} d{D} {heads} heads, std {std}, sink {sink}: {got / norm:.2e} of {tol / norm:.2e}")
    assert got <= tol
