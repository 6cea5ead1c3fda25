"""The output of scoring attention calls is held to float32 for values of any size and for rows whose weight lies
on one token: its error, as a share of the output's norm, against the oracle in 64 bits."""
import numpy as np
import pytest
import torch

import sub_byte_quantized_gb300 as kvq
from oracle import attention as OA, budget as OB

pytestmark = pytest.mark.gpu
S, H = 4096, 2
TOP_CODE = {"q8_0": 128, "q6_0": 32, "asym4_g32": 15, "q4_0": 8, "had_int4": 7, "had_int2": 1}


def _inputs(std, sink, rows, nq, D):
    """Keys and queries of scores near 0.01, values of zero mean (std: of all tokens, or of each); or (sink) scores
    near 0.1 and a first token without value that takes 2^14 times the others' weight."""
    rng = np.random.default_rng(11)
    alpha = np.float32((0.1 if sink else 0.01) / np.sqrt(D))
    Hq = H * rows // nq
    k = rng.standard_normal((1, H, S, D)).astype(np.float32)
    v = (np.broadcast_to(np.asarray(std), (S,))[:, None] * rng.standard_normal((1, H, S, D))).astype(np.float32)
    q = rng.standard_normal((1, Hq, nq, D)).astype(np.float32)
    if sink:
        q0 = rng.standard_normal((1, H, 1, D)).astype(np.float32)
        q = np.repeat(q0, Hq // H, 1) + 0.05 * q
        k[:, :, :1] = q0 * np.float32(14 * np.log(2)) / (alpha * (q0 * q0).sum(-1, keepdims=True))
        v[:, :, 0] = 0
    return k, v, torch.from_numpy(q).to(torch.bfloat16), alpha


def _sums(layout, D, rows, chunk):
    """What the tensor cores' additions may cost of a sum over a chunk. Each may truncate 2^-23 of the running sum;
    n roundings of 2^-24 to nearest are independent."""
    n = chunk // 64                                         # four warps take its 16-token tiles in turn
    if layout in ("had_int4", "had_int2") and rows > 64:    # all tokens in one accumulator, hi and lo
        return chunk // 16 * 2 * 2.0 ** -23
    if D == 128 and layout != "q6_0" and rows <= 8 and "+" not in layout or layout == "q4_0+q8_0" and rows <= 8:
        if layout == "asym4_g32":                           # two products of a tile by themselves, then one rounded addition
            return 2 * 2.0 ** -23 + np.sqrt(n) * 2.0 ** -24
        if layout.startswith("had"):                        # two products of every tile into the running sum
            return 2 * n * 2.0 ** -23
        return (2 + n) * 2.0 ** -23 + np.sqrt(n) * 2.0 ** -24   # every other tile by itself
    if D == 128 and (rows > 8 or "+" in layout):
        # 32 tokens by themselves (six products), or four warps and 16 tokens (three), then one rounded addition
        return 6 * 2.0 ** -23 + np.sqrt(chunk // 32) * 2.0 ** -24
    return n * 2.0 ** -23                                   # (Q6_0's own kernel) hi and lo apart


def _check(layout, rows, nq, std, sink=False, chunk=256, D=128, lift=12):
    """The values' signs are random and independent of every rounding of the weights, so an error of at most e in
    each token's weight moves the output by at most e of its norm in the mean square; 1.5 covers the spread over
    dims and rows. e: the score's and the exponent's own, for the token and once more for the sum of all (as in
    oracle.budget.weights); P' = p * scale as two f16 parts, 2^-21; the sums. Added to it what f16's subnormals
    cost: two roundings of 2^-25 in P', p being 2^lift times larger, times the code."""
    k, v, qd, alpha = _inputs(std, sink, rows, nq, D)
    q = qd.float().numpy()
    dc, oc = kvq.KVCache(layout, 1, H, D, S), OA.OracleCache(layout, 1, H, D, S)
    kvq.store(dc, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), 0)
    oc.store(k, v, 0)
    out, _ = kvq.decode_attend_weights(dc, qd.cuda(), S, None, scores_out=torch.zeros((1, H, S), device="cuda"),
                                       attn_scale=float(alpha), chunk=chunk)
    s, mass = OB.scores_dense(oc, q, alpha, S)
    err = 2 * (float(mass.max()) * ((D // 16 + D // 32 + 4) * 2.0 ** -23 + 2.0 ** -22)
               + 3 * 2.0 ** -24 * 1.5 * float(s.max() - s.min()) + 2.0 ** -22)
    l = np.exp(s - s.max(-1, keepdims=True)).sum(-1)
    low = 2 * 2.0 ** -(25 + lift) * TOP_CODE[layout.split("+")[-1]] * np.sqrt(S * D * ((1 / l) ** 2).sum())
    ref = oc.attend(q, alpha, S)
    ref = ref[0] if isinstance(ref, tuple) else ref
    norm = np.linalg.norm(ref)
    tol = 1.5 * (err + 2.0 ** -21 + _sums(layout, D, rows, chunk)) * norm + low
    got = np.linalg.norm(out.cpu().numpy().astype(np.float64) - ref)
    print(f"{layout} d{D} {rows} rows, std {std if np.isscalar(std) else 'mixed'}, sink {sink}, chunk {chunk}: "
          f"{got / norm:.2e} of {tol / norm:.2e}")
    assert got <= tol


CASES = [("q6_0", 128, 1, 1), ("q6_0", 128, 8, 1), ("q6_0", 256, 1, 1), ("q6_0", 256, 32, 8),
         ("asym4_g32", 128, 1, 1), ("asym4_g32", 128, 8, 1), ("asym4_g32", 128, 6, 2)]
CASES += [(layout, 128, rows, 1) for layout in ("q4_0", "q8_0", "q4_0+q8_0", "had_int4", "had_int2") for rows in (1, 8)]
CASES += [(layout, 128, 32, 8) for layout in ("q4_0", "q6_0", "q8_0", "asym4_g32", "had_int4", "had_int2", "q4_0+q8_0")]
CASES += [(layout, 128, rows, nq) for layout in ("asym4_g32+q8_0", "had_int2+had_int4") for rows, nq in ((1, 1), (12, 3), (40, 5))]
CASES += [(layout, 128, rows, 20) for layout in ("had_int4", "had_int2") for rows in (80, 160)]


@pytest.mark.parametrize("layout,D,rows,nq", CASES)
@pytest.mark.parametrize("std", [1.0, 0.1, 0.01, 0.001])
def test_output_with_values_of_any_size(layout, D, rows, nq, std):
    _check(layout, rows, nq, std, D=D)


@pytest.mark.parametrize("layout,D,rows,nq", CASES)
def test_output_of_rows_whose_weight_lies_on_one_token(layout, D, rows, nq):
    _check(layout, rows, nq, 1.0, sink=True, D=D)


@pytest.mark.parametrize("layout,D,rows,nq", CASES)
def test_output_with_values_that_grow_in_the_middle(layout, D, rows, nq):
    """Scales beyond 2 from some token of a chunk on: probabilities without the factor from there."""
    _check(layout, rows, nq, np.where(np.arange(S) < 150, 1e-3, 1e3), D=D, lift=0)


@pytest.mark.parametrize("layout,D,rows,nq", [c for c in CASES if c[:2] != ("q6_0", 256)])
def test_output_of_long_chunks(layout, D, rows, nq):
    """One chunk of all tokens."""
    _check(layout, rows, nq, 1.0, chunk=S, D=D)
