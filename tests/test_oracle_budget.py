"""Pins of the oracles of rotary positions and of the cache budget: hand-computed values and
identities, on the CPU."""
import math

import numpy as np
import pytest

from oracle import attention as OA, budget as OB, rope as OR
from synth import WORKLOADS, make_inputs


def test_rotation_by_hand():
    # a quarter turn: (a, b) -> (-b, a)
    rows = np.array([[0.0] * 8 + [1.0] * 8], np.float32)
    x = np.arange(1, 19, dtype=np.float32)[None]
    half = OR.rotate(x, rows)
    assert half[0, :8].tolist() == [-v for v in range(9, 17)] and half[0, 8:16].tolist() == list(range(1, 9))
    inter = OR.rotate(x, rows, interleaved=True)
    assert inter[0, :4].tolist() == [-2, 1, -4, 3]
    assert half[0, 16:].tolist() == inter[0, 16:].tolist() == [17, 18]


def test_rotation_keeps_the_relative_angle():
    f, _ = OR.frequencies(64)
    t = OR.table(f, 0, 200).astype(np.float32)
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 64)).astype(np.float32)
    for il in (False, True):
        dots = [float((OR.rotate(q, t[p:p + 1], il) * OR.rotate(k, t[p - 7:p - 6], il)).astype(np.float64).sum()) for p in (7, 60, 199)]
        assert np.ptp(dots) < 1e-4


def test_frequency_scalings():
    f, m = OR.frequencies(64)
    assert f[0] == 1.0 and m == 1.0 and abs(f[16] - 10000.0 ** -0.5) < 1e-12
    assert np.allclose(OR.frequencies(64, scaling="linear", factor=4.0)[0], f / 4, rtol=1e-15)
    ntk = OR.frequencies(64, scaling="ntk", factor=4.0)[0]
    assert ntk[0] == 1.0 and abs(ntk[-1] * 4.0 - f[-1]) < 1e-12             # the slowest dim is divided by factor
    for kind, lo, hi in (("banded", 1.0, 4.0), ("yarn", 1.0, 32.0)):
        g, m = OR.frequencies(64, scaling=kind, factor=8.0, original_len=4096, low=lo, high=hi)
        assert g[0] == f[0] and abs(g[-1] - f[-1] / 8) < 1e-15 and np.all(g <= f) and np.all(g >= f / 8 - 1e-18)
        assert abs(m - (0.1 * math.log(8) + 1 if kind == "yarn" else 1.0)) < 1e-12


def test_weights_sum_to_the_rows():
    w = WORKLOADS["c3_had_int4_decode"].scaled(batch=1)
    inp = make_inputs(w, kv_len=90, n_q=3)
    c = OA.OracleCache(w.layout, 1, 8, 128, 96, n_recent=16)
    c.store(inp["k"], inp["v"], 0)
    got, err = OB.weights(c, inp["q"], w.alpha, 90, True, 87)
    assert np.allclose(got.sum(-1), 2 * 3) and 0 < err < 1e-2 and got[..., 89].max() <= 2.0


def test_select_by_hand():
    s = np.array([[[5, 1, np.nan, 7, 7, 0.0, -0.0, np.inf, -np.inf, 2]]], np.float32)
    assert OB.select(s, [10], 3)[0, 0].tolist() == [3, 4, 7]
    assert OB.select(s, [10], 4, 1, 1)[0, 0].tolist() == [0, 3, 7, 9]
    assert OB.select(s, [10], 7)[0, 0].tolist() == [0, 1, 3, 4, 5, 7, 9]
    assert OB.select(s, [3], 5)[0, 0].tolist() == [0, 1, 2, -1, -1]
    assert OB.select(s, [0], 2)[0, 0].tolist() == [-1, -1]


@pytest.mark.parametrize("n_recent", [0, 5])
def test_compact_attends_the_kept_tokens(n_recent):
    w = WORKLOADS["c3_had_int4_decode"].scaled(batch=1)
    inp = make_inputs(w, kv_len=40)
    c = OA.OracleCache(w.layout, 1, 8, 128, 40, n_recent=n_recent)
    c.store(inp["k"], inp["v"], 0)
    kept = np.r_[0:3, 10:20, 33:40]
    want = OA.OracleCache(w.layout, 1, 8, 128, 40, n_recent=n_recent)
    want.store(inp["k"][:, :, kept], inp["v"][:, :, kept], 0)
    OB.compact(c.planes, np.broadcast_to(kept, (1, 8, 20)), [40], n_recent)
    a, _ = c.attend(inp["q"], w.alpha, 20)
    b, _ = want.attend(inp["q"], w.alpha, 20)
    assert np.array_equal(a, b)
