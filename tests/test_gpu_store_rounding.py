"""Where the stored codes turn: quotients at a half-integer and one or two steps of float32 beside it, scales at
the ends of their range, and values that are not finite; plain appends and rotary ones, bit for bit."""
import numpy as np
import pytest
import torch

import sub_byte_quantized_gb300 as kvq
from oracle import attention as OA, quant as OQ
from tests.gpu_helpers import planes_equal

pytestmark = pytest.mark.gpu
LAYOUTS = ["q4_0", "q6_0", "q8_0", "asym4_g32", "had_int4", "had_int2"]
TOP = {"q4_0": 8, "q6_0": 32, "q8_0": 128}


def _steps(x, n):
    """n steps of float32 away from zero (towards it for n < 0)."""
    return (x.astype(np.float32).view(np.int32) + np.int32(n)).view(np.float32)


def _turning_rows(layout, rng, n, D):
    if layout == "asym4_g32":
        # zero-points and spans that the f16 scales hold exactly, values z + (k + 1/2) s
        s = np.float16(rng.uniform(0.01, 4, (n, D // 32, 1))).astype(np.float32)
        z = np.float16(rng.uniform(-3, 3, (n, D // 32, 1))).astype(np.float32)
        x = (z + (rng.integers(0, 15, (n, D // 32, 32)) + np.float32(0.5)) * s).astype(np.float32)
        x = _steps(x, 0) + rng.integers(-2, 3, x.shape) * np.spacing(x)
        x[..., 3] = z[..., 0]
        x[..., 17] = (z + np.float32(15) * s)[..., 0]
        return x.reshape(n, D).astype(np.float32)
    if layout in TOP:
        t = TOP[layout]
        s = np.float16(2.0 ** rng.uniform(-14, 10, (n, D // 32, 1))).astype(np.float32)
        x = ((rng.integers(-t, t, (n, D // 32, 32)) + np.float32(0.5)) * s).astype(np.float32)
        x = x + rng.integers(-2, 3, x.shape).astype(np.float32) * np.spacing(x)
        x[..., 11] = (t * s)[..., 0] * rng.choice([-1, 1], x.shape[:-1])
        return x.reshape(n, D).astype(np.float32)
    # a rotated row of multiples of s / 2 (exact where 1 / sqrt(D) is a power of two), and neighbours of it
    q = 7 if layout == "had_int4" else 1
    y = rng.integers(-2 * q, 2 * q + 1, (n, D)) / 2.0
    y[:, 5] = q
    x = OQ.fwht(y, np.float64) / np.sqrt(D) * 2.0 ** rng.integers(-20, 20, (n, 1))
    x = x.astype(np.float32)
    x[n // 2:] += rng.integers(-1, 2, x[n // 2:].shape) * np.spacing(x[n // 2:])
    return x.astype(np.float32)


def _both(layout, k, v):
    """k and v through the plain and the rotary append (an angle of zero everywhere)."""
    B, H, n, D = k.shape
    R = 8 if "had" in layout else 0
    table = torch.zeros((1, D), device="cuda")
    table[:, :D // 2] = 1.0
    kd, vd = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda()
    a, b = (kvq.KVCache(layout, B, H, D, n, n_recent=R) for _ in range(2))
    kvq.store(a, kd, vd, 0)
    kvq.rope_store(b, table, kd, vd, 0, positions=torch.zeros((B, n), dtype=torch.int32, device="cuda"))
    return a, b, R


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("D", [128, 256])
def test_half_way_quotients(layout, D):
    rng = np.random.default_rng(D)
    k, v = (_turning_rows(layout, rng, 2 * 600, D).reshape(1, 2, 600, D) for _ in range(2))
    a, b, R = _both(layout, k, v)
    oc = OA.OracleCache(layout, 1, 2, D, 600, n_recent=R)
    oc.store(k, v, 0)
    planes_equal(a, oc)
    planes_equal(b, oc)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("D", [128, 256])
def test_ends_of_the_scale(layout, D):
    """Scales that are zero, subnormal, the least and the largest of their type, and beyond it."""
    rng = np.random.default_rng(D + 1)
    e = np.r_[np.arange(-149, -90, 3), np.arange(-40, 30), np.arange(90, 120, 3)]
    k, v = (np.ldexp(rng.standard_normal((1, 2, len(e), D)), e[:, None]).astype(np.float32) for _ in range(2))
    a, b, R = _both(layout, k, v)
    oc = OA.OracleCache(layout, 1, 2, D, len(e), n_recent=R)
    oc.store(k, v, 0)
    planes_equal(a, oc)
    planes_equal(b, oc)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_values_that_are_not_finite(layout):
    """An infinity takes the last code of its side (its block's scale saturates at the largest f16, or is
    infinite in a Hadamard row), a NaN the lowest code; NaN takes no part in a block's extremes."""
    D = 128
    rng = np.random.default_rng(4)
    x = rng.standard_normal((1, 1, 4, D)).astype(np.float32)
    x[0, 0, 0, 40] = np.inf
    x[0, 0, 1, 70] = -np.inf
    x[0, 0, 2, 3] = np.nan
    x[0, 0, 3] = 3e38                                            # the sums of a rotation overflow
    dc = kvq.KVCache(layout, 1, 1, D, 4)
    kvq.store(dc, torch.from_numpy(x).cuda(), torch.from_numpy(x).cuda(), 0)
    got = {n: t.cpu().numpy()[0, 0] for n, t in dc.planes["k"].items()}

    def codes(y, s, lo, hi):
        with np.errstate(all="ignore"):
            r = np.rint((y / s).astype(np.float32))
        return np.where(s > 0, np.where(np.isnan(r), lo, np.clip(r, lo, hi)), 0).astype(np.int64)

    with np.errstate(all="ignore"):
        if "had" in layout:
            q = 7 if layout == "had_int4" else 1
            y = OQ.rotate(x)[0, 0]
            s = np.fmax.reduce(np.abs(y), axis=-1, initial=np.float32(0)) / np.float32(q)
            assert np.array_equal(got["scale"], s)
            have = OQ.hadamard_layout_codes(layout, got["payload"], D)
            assert np.array_equal(have, codes(y, s[:, None], -q, q))
            return
        y = x[0, 0].reshape(4, D // 32, 32)
        if layout == "asym4_g32":
            mn, mx = np.fmin.reduce(y, axis=-1), np.fmax.reduce(y, axis=-1)
            s, z = OQ.fp16_round((mx - mn) / np.float32(15)), OQ.fp16_round(mn)
            assert np.array_equal(got["zero"], z)
            want = codes(y - z.astype(np.float32)[..., None], s.astype(np.float32)[..., None], 0, 15)
            have = OQ.unpack_nibbles(got["payload"], D)
        else:
            t = TOP[layout]
            s = OQ.fp16_round(np.fmax.reduce(np.abs(y), axis=-1) / np.float32(t))
            want = codes(y, s.astype(np.float32)[..., None], -t, t - 1)
            if layout == "q4_0":
                have = OQ.read_q4_0(OQ.unpack_nibbles(got["payload"], D))
            elif layout == "q6_0":
                have = OQ.read_q6_0(OQ.q6_0_fields(got["payload"], D // 32))
            else:
                have = OQ.read_q8_0(got["payload"])
    assert np.array_equal(got["scale"], s)
    assert np.array_equal(np.asarray(have).reshape(4, -1), want.reshape(4, -1))
