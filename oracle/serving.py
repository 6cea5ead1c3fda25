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
