"""Oracle of the serving-step calls: the page plan, the 8-bit block layouts, block bounds, block selection and
attention over selected blocks.

TEST INFRASTRUCTURE ONLY (see the package docstring). One request, block or row after the other, in plain loops.
"""
from __future__ import annotations

import numpy as np


def page_plan(seq_lens, new_lens, table, page, free, n_free, max_tokens):
    """The plan as include/kvq.h defines it; `table` and `free` (numpy int arrays) are updated. Returns a dict."""
    B, per = table.shape
    cap, n_free = per * page, int(min(max(int(n_free), 0), len(free)))
    old = [min(max(int(x), 0), cap) for x in seq_lens]
    for b in range(B):
        if new_lens[b] < 0:
            for j in range(-(-old[b] // page)):
                if n_free < len(free):
                    free[n_free] = table[b, j]
                    n_free += 1
    pages = tokens = 0
    lens, granted, cu, slots, positions = [], [], [0], [], []
    top = n_free
    for b in range(B):
        n, held = int(new_lens[b]), -(-old[b] // page)
        got = 0
        if 0 <= n <= cap - old[b]:
            need = -(-(old[b] + n) // page) - held
            pages += need
            if need == 0 or pages <= n_free:
                tokens += n
                if n == 0 or tokens <= max_tokens:
                    got = n
                    for j in range(need):
                        top -= 1
                        table[b, held + j] = free[top]
        lens.append(0 if n < 0 else old[b] + got)
        granted.append(got)
        cu.append(cu[-1] + got)
        for p in range(old[b], old[b] + got):
            slots.append(int(table[b, p // page]) * page + p % page)
            positions.append(p)
    none = [-1] * (max_tokens - len(slots))
    return {"lens": np.array(lens, np.int32), "granted": np.array(granted, np.int32), "n_free": np.array([top], np.int32),
            "cu_new": np.array(cu, np.int32), "slots": np.array(slots + none, np.int64), "positions": np.array(positions + none, np.int32)}


# ------------------------------------------------------------------ 8-bit layouts with a scale per block of 64 tokens
BLOCK_TOKENS = 64
TOP = {"int8_b64": 127, "e4m3_b64": 448}


def _e4m3_table():
    """Values of the e4m3 bytes 0 .. 0x7E: exponent 0 is subnormal (2^-9 steps), bias 7, three fraction bits."""
    v = []
    for b in range(0x7F):
        e, f = b >> 3, b & 7
        v.append(f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
    return np.array(v)


E4M3 = _e4m3_table()


def encode(layout, x):
    """Code bytes of values already divided by their scale: nearest, ties to even, saturating."""
    x = np.asarray(x, np.float64)
    if layout == "int8_b64":
        return np.clip(np.rint(x), -127, 127).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.searchsorted(E4M3, a)                          # E4M3[hi - 1] < a <= E4M3[hi]
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def decode(layout, b):
    if layout == "int8_b64":
        return b.view(np.int8).astype(np.float64)
    return E4M3[np.minimum(b & 0x7F, 0x7E)] * np.where(b & 0x80, -1.0, 1.0)


class BlockCache:
    """Logical view of one of the two layouts: payload u8 [B][H][cap][D], scale f32 [B][H][cap / 64] per plane."""

    def __init__(self, layout, batch, n_kv_heads, head_dim, capacity):
        self.layout, self.B, self.H, self.D, self.cap = layout, batch, n_kv_heads, head_dim, capacity
        self.planes = {t: {"payload": np.zeros((batch, n_kv_heads, capacity, head_dim), np.uint8),
                           "scale": np.zeros((batch, n_kv_heads, capacity // BLOCK_TOKENS), np.float32)} for t in ("k", "v")}

    def append(self, t, b, x, pos):
        """Rows x [H][n][D] (float32) of sequence b at positions pos .. pos + n; those outside [0, cap) are dropped."""
        pl, top = self.planes[t], np.float32(TOP[self.layout])
        lo, hi = max(pos, 0), min(pos + x.shape[1], self.cap)
        for first in range(lo, hi):
            if first > lo and first % BLOCK_TOKENS:
                continue                                   # not the first new row of its block
            blk = first // BLOCK_TOKENS
            end = min(hi, (blk + 1) * BLOCK_TOKENS)
            for h in range(self.H):
                new = x[h, first - pos:end - pos].astype(np.float32)
                need = np.float32(min(np.abs(new).max(), np.finfo(np.float32).max) / top)   # infinities: the largest value
                s = pl["scale"][b, h, blk] if first % BLOCK_TOKENS else np.float32(0)
                k = 0
                if s == 0:
                    s = need
                else:
                    while s < need:
                        s, k = np.float32(s * np.float32(2)), k + 1
                pl["scale"][b, h, blk] = s
                if k:
                    kept = pl["payload"][b, h, blk * BLOCK_TOKENS:first]
                    kept[...] = encode(self.layout, decode(self.layout, kept) * 2.0 ** -k)
                with np.errstate(divide="ignore", invalid="ignore"):
                    y = np.where(s > 0, new / s, np.float32(0))
                pl["payload"][b, h, first:end] = encode(self.layout, y)

    def store(self, k, v, positions):
        for t, x in (("k", k), ("v", v)):
            for b in range(self.B):
                self.append(t, b, np.asarray(x[b], np.float32), int(positions[b]))

    def values(self, t, b, h, n):
        pl = self.planes[t]
        return decode(self.layout, pl["payload"][b, h, :n]) * np.repeat(pl["scale"][b, h].astype(np.float64), BLOCK_TOKENS)[:n, None]

    def attend(self, q, alpha, lens, causal=False, blocks=None):
        return attend(lambda t, b, h, n: self.values(t, b, h, n), self.H, q, alpha, lens, causal, blocks)


def attend(values, H, q, alpha, lens, causal=False, blocks=None):
    """(float64 attention [B][H_q][n_q][D], bound of what a float32 computation may be off by). values(t, b, h, n): rows of
    a plane; causal rows are each sequence's newest; blocks [B][H][n_q][n_sel]: a row sees the tokens of these blocks alone
    (a list ends at the first entry that is not above the one before it).

    The bound, of a row with weights p_t: its score is off by the dot product's additions, which the tensor cores may
    truncate (D / 16 steps and a few of 2^-23 of the running sum, at most the mass sum |q_i k_i|), by a query in two f16
    parts (2^-22) and by a few roundings of the score itself; the weights follow it twice (numerator and sum). The product
    with V: p in two f16 parts (2^-21, and the second one's subnormals: 2^12 p is a multiple of 2^-24 there, so a p of at most 1
    is off by half of that, 2^-37, and the output by 2^-37 sum |v_t|, where p_t |v_t| may be far less), four truncated additions per 32 tokens, one rounded one for each of those, the
    chunks' sums and the exponentials' 2^-22."""
    q = np.asarray(q, np.float64)
    B, Hq, nq, D = q.shape
    g = Hq // H
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        n = int(lens[b])
        if n <= 0:
            continue
        for hq in range(Hq):
            k, v = values("k", b, hq // g, n), values("v", b, hq // g, n)
            for i in range(nq):
                last = n - nq + i if causal else n - 1
                seen = np.arange(n) <= last
                if blocks is not None:
                    some, before = np.zeros(n, bool), -1
                    for blk in blocks[b, hq // g, i]:
                        if blk <= before:
                            break
                        some[blk * BLOCK_TOKENS:(blk + 1) * BLOCK_TOKENS] = True
                        before = blk
                    seen &= some
                if not seen.any():
                    continue
                kk, vv = k[seen], v[seen]
                s = alpha * (kk @ q[b, hq, i])
                mass = abs(alpha) * (np.abs(kk) @ np.abs(q[b, hq, i]))
                p = np.exp(s - s.max())
                p /= p.sum()
                out[b, hq, i] = p @ vv
                ds = (mass * ((D / 16 + 4) * 2.0 ** -23 + 2.0 ** -21) + 6 * 2.0 ** -24 * np.abs(s)).max()
                tol[b, hq, i] = (p @ np.abs(vv)) * (2 * ds + 2.0 ** -20 + (len(s) / 32 + 24) * 2.0 ** -23) + 2.0 ** -37 * np.abs(vv).sum(0)
    return out, tol


# ------------------------------------------------------------------ bounds and selection of blocks
def key_rows(cache, b, h, n):
    """float32 key rows [n][D] that a contiguous cache's packed rows stand for (Hadamard layouts: rotated)."""
    if isinstance(cache, BlockCache):
        return cache.values("k", b, h, n).astype(np.float32)
    return cache.dequantized("k", n)[b, h].astype(np.float32)


def bounds(rows):
    """(codes int8 [blocks][2][D], scale f32 [blocks]) of the blocks of key rows [n][D]."""
    codes, scales = [], []
    for t in range(0, len(rows), BLOCK_TOKENS):
        lo, hi = rows[t:t + BLOCK_TOKENS].min(0), rows[t:t + BLOCK_TOKENS].max(0)
        s = np.float32(max(np.abs(lo).max(), np.abs(hi).max())) / np.float32(127)
        if s > 0:
            lo, hi = np.floor(lo / s), np.ceil(hi / s)
        else:
            lo, hi = lo * 0, hi * 0
        codes.append(np.clip(np.stack((lo, hi)), -127, 127).astype(np.int8))
        scales.append(s)
    return np.array(codes), np.array(scales, np.float32)


def select(codes, scale, q, limits, n_sel, n_sink, n_recent):
    """Lists [n_q][n_sel] of one kv head: codes [blocks][2][D], scale [blocks], q float32 [heads][n_q][D] (rotated where the
    layout is), limits [n_q]: the last token that each row sees."""
    out = np.full((q.shape[1], n_sel), -1, np.int32)
    for i, last in enumerate(limits):
        n = 0 if last < 0 else last // BLOCK_TOKENS + 1
        if n <= n_sel:
            out[i, :n] = np.arange(n)
            continue
        best = np.full(n, -np.inf, np.float32)
        for x in q[:, i].astype(np.float32):
            s = np.float32(np.abs(x).max()) / np.float32(127)
            q8 = np.clip(np.rint(x / s), -127, 127).astype(np.int64) if s > 0 else np.zeros(len(x), np.int64)
            dots = np.where(q8 > 0, q8 * codes[:n, 1].astype(np.int64), q8 * codes[:n, 0].astype(np.int64)).sum(1)
            best = np.maximum(best, dots.astype(np.float32) * s)
        best = best * scale[:n]
        keep = set(range(n_sink)) | set(range(n - n_recent, n))
        others = sorted((b for b in range(n) if b not in keep), key=lambda b: (-float(best[b]), b))
        out[i] = sorted(keep | set(others[:n_sel - len(keep)]))
    return out
