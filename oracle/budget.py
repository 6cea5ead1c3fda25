"""Oracle of a cache kept inside a budget: attention weight per token, selection, compaction.

TEST INFRASTRUCTURE ONLY (see the package docstring).

  * weights: the softmax weights of `oracle.attention`, summed over the query rows that share a kv head.
  * selection: the first n_sink tokens, the last n_recent, then the highest scores among the others, ties
    to the lowest index (NaN counts as -infinity, -0 as +0); ascending, -1 behind a short sequence.
  * compaction: row keep[i] of every plane becomes row i. The ring slot of token t is t mod n_recent, so
    with `cut` tokens gone the row of slot (j + cut) mod n_recent belongs at slot j.
"""
from __future__ import annotations

import numpy as np

from . import quant as Q
from .attention import prep_q_hadamard, visible_mask, _softmax_rows


def scores_dense(cache, q, alpha, kv_len):
    """float64 alpha * q . k_hat [B][H_q][n_q][kv_len], and sum |q_i| |k_i| alpha of the same shape."""
    q = np.asarray(q, np.float32)
    B, Hq, nq, D = q.shape
    g = Hq // cache.H
    s, mass = np.zeros((B, Hq, nq, kv_len)), np.zeros((B, Hq, nq, kv_len))
    had = Q.is_hadamard(cache.layout)
    if had:
        q_rot, s_q, q8 = prep_q_hadamard(q)
        x_all = q8.astype(np.float64) * s_q.astype(np.float64)[..., None]
    else:
        x_all = q.astype(np.float64)
    K = cache.dequantized("k", kv_len)
    nw = min(cache.n_recent, kv_len) if had else 0
    for b in range(B):
        for h in range(Hq):
            k = K[b, h // g]
            s[b, h] = x_all[b, h] @ k.T
            mass[b, h] = np.abs(x_all[b, h]) @ np.abs(k).T
            if nw:
                w = cache.planes["k"]["ring"][b, h // g, np.arange(kv_len - nw, kv_len) % cache.n_recent].astype(np.float64)
                s[b, h, :, kv_len - nw:] = q_rot[b, h].astype(np.float64) @ w.T
                mass[b, h, :, kv_len - nw:] = np.abs(q_rot[b, h]).astype(np.float64) @ np.abs(w).T
    return alpha * s, abs(alpha) * mass


def weights(cache, q, alpha, kv_len, causal=False, q_pos0=0):
    """(float64 [B][H_kv][kv_len] weights, relative error a float32 computation may have).

    The relative error of one weight exp(s - lse): the dot products are summed in float32 whose additions
    the tensor cores may truncate (2^-23 of the running sum, at most the mass sum |q_i k_i|; D / 16 steps,
    D / 32 block additions, and a few for the scales), a query in two f16 parts is off by 2^-22 of itself;
    s and lse are rounded in base 2 (three roundings of 2^-24, absolute, of up to 1.5 (|s| + |lse|)), and the
    exponentials by 2^-22; once for s and once, averaged, for lse."""
    s, mass = scores_dense(cache, q, alpha, kv_len)
    B, Hq, nq, _ = s.shape
    vis = visible_mask(nq, kv_len, causal, q_pos0)
    p, l = _softmax_rows(s, vis)
    with np.errstate(invalid="ignore", divide="ignore"):
        p = np.where(l > 0, p / l, 0.0)
    D = q.shape[-1]
    top = float(np.abs(s).max()) if s.size else 0.0
    err = 2 * (float(mass.max()) * ((D // 16 + D // 32 + 4) * 2.0 ** -23 + 2.0 ** -22)
               + 3 * 2.0 ** -24 * 1.5 * (2 * top + np.log(kv_len)) + 2.0 ** -22)
    return p.reshape(B, cache.H, -1, kv_len).sum(2), err


def select(scores, lens, n_keep, n_sink=0, n_recent=0):
    """int32 [B][H][n_keep] of scores [B][H][stride], one sequence and head at a time."""
    B, H, _ = scores.shape
    keep = np.full((B, H, n_keep), -1, np.int32)
    for b in range(B):
        L = int(lens[b])
        for h in range(H):
            if L <= n_keep:
                keep[b, h, :L] = np.arange(L)
                continue
            x = scores[b, h, :L].astype(np.float64)
            x = np.where(np.isnan(x), -np.inf, x)
            free = np.arange(n_sink, L - n_recent)
            order = free[np.lexsort((free, -x[free]))]            # score descending, then index ascending
            chosen = order[:n_keep - n_sink - n_recent]
            keep[b, h] = np.sort(np.concatenate([np.arange(n_sink), chosen, np.arange(L - n_recent, L)]))
    return keep


def compact(planes, keep, lens, n_recent, locate=None):
    """Moves the rows of `planes` (the "k" / "v" dict of an oracle cache) in place. locate(b, t) -> the
    leading index of token t of sequence b and its row (paged); contiguous rows otherwise."""
    at = locate or (lambda b, t: (b, t))
    B, H, n_keep = keep.shape
    for pl in planes.values():
        for name in ("payload", "scale", "zero"):
            if name not in pl:
                continue
            old = pl[name].copy()
            for b in range(B):
                for i in range(min(int(lens[b]), n_keep)):
                    d = at(b, i)
                    for h in range(H):
                        t = int(keep[b, h, i])
                        if 0 <= t < lens[b]:
                            s = at(b, t)
                            pl[name][d[0], h, d[1]] = old[s[0], h, s[1]]
        if "ring" in pl:
            for b in range(B):
                cut = max(0, int(lens[b]) - n_keep)
                pl["ring"][b] = np.roll(pl["ring"][b], -(cut % n_recent), axis=1)
