"""Oracle of the rotary positions: frequencies, table and rotation.

TEST INFRASTRUCTURE ONLY (see the package docstring). Position p turns pair i of a row by the angle
p f_i; with c and s the table's float32 cosine and sine,
    y_a = x_a c - x_b s,   y_b = x_b c + x_a s,
every product and every sum rounded to float32 by itself.
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(rot_dim, base=10000.0, scaling="none", factor=1.0, original_len=0.0, low=1.0, high=4.0):
    """(float64 frequencies in radians per position, magnitude): one scalar formula per pair."""
    out, mag = [], 1.0
    if scaling == "ntk":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    for i in range(rot_dim // 2):
        f = base ** (-2 * i / rot_dim)
        if scaling == "linear":
            f /= factor
        elif scaling == "banded":
            turns = original_len * f / (2 * math.pi)
            if turns <= low:
                f /= factor
            elif turns < high:
                w = (turns - low) / (high - low)
                f = (1 - w) * f / factor + w * f
        elif scaling == "yarn":
            def dim_of(turns):
                return rot_dim * math.log(original_len / (2 * math.pi * turns)) / (2 * math.log(base))
            lo = min(max(math.floor(dim_of(high)), 0), rot_dim - 1)
            hi = min(max(math.ceil(dim_of(low)), 0), rot_dim - 1)
            ramp = min(max((i - lo) / (hi - lo if hi > lo else 0.001), 0.0), 1.0)
            f = f / factor * ramp + f * (1 - ramp)
            mag = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
        out.append(f)
    return np.array(out), mag


def table(inv_freq, pos0, n_pos, magnitude=1.0):
    """float64 [n_pos][rot_dim]: cosines, then sines."""
    a = np.outer(np.arange(pos0, pos0 + n_pos, dtype=np.float64), np.asarray(inv_freq, np.float64))
    return np.concatenate([np.cos(a), np.sin(a)], 1) * magnitude


def rotate(x, rows, interleaved=False):
    """x float32 [..., n, D] by the table rows float32 [..., n, rot_dim] (broadcast over heads)."""
    x = np.asarray(x, np.float32)
    rot = rows.shape[-1]
    h = rot // 2
    c, s = rows[..., :h], rows[..., h:]
    y = x.copy()
    a_at = np.arange(0, rot, 2) if interleaved else np.arange(h)
    b_at = a_at + 1 if interleaved else a_at + h
    a, b = x[..., a_at], x[..., b_at]
    y[..., a_at] = a * c - b * s                       # numpy rounds every float32 operation
    y[..., b_at] = b * c + a * s
    return y
