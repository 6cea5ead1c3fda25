"""Rotary appends at the ends of what they are documented for, and the table by its kernel's own roundings."""
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import sub_byte_quantized_gb300 as kvq
from oracle import rope as OR

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("queries", [False, True])
@pytest.mark.parametrize("layout", ["q4_0", "had_int4", "q4_0+q8_0"])
def test_an_append_of_no_rows(layout, queries, paged):
    B, H, D, cap = 2, 2, 128, 128
    n_recent = 16 if layout.startswith("had") else 0
    x = torch.randn((B, H, 3, D), device="cuda").bfloat16()
    f, _ = kvq.rope_frequencies(D)
    table = kvq.rope_table(f, cap)
    if paged:
        c = kvq.PagedKVCache(layout, B, H, D, 64, 4, 2, n_recent=n_recent)
        c.set_block_table(torch.arange(4).view(2, 2))
        at, call = torch.tensor([5, 9], dtype=torch.int32, device="cuda"), kvq.paged_rope_store
    else:
        c, at, call = kvq.KVCache(layout, B, H, D, cap, n_recent=n_recent), cap, kvq.rope_store
    for p in c.planes.values():
        for t in p.values():
            t.copy_(torch.randint(0, 100, t.shape, device="cuda"))
    before = {(k, n): t.clone() for k, p in c.planes.items() for n, t in p.items()}
    none = x[:, :, :0]
    got = call(c, table, none, none, at, q=none if queries else None,
               positions=torch.empty((B, 0), dtype=torch.int32, device="cuda"))
    assert got.shape == (B, H, 0, D) if queries else got is None
    torch.cuda.synchronize()
    for (k, n), t in before.items():
        assert torch.equal(c.planes[k][n], t)


def test_rotated_queries_beside_the_projection_in_one_buffer():
    """q_out right before and right behind the inputs' memory is no overlap; anywhere inside it is refused."""
    B, n, Hq, H, D = 2, 3, 4, 2, 128
    size, out = B * n * (Hq + 2 * H) * D, B * Hq * n * D
    buf = torch.randn(size + 2 * out, device="cuda").bfloat16()
    x = buf[out:out + size].view(B, n, Hq + 2 * H, D).transpose(1, 2)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    f, _ = kvq.rope_frequencies(D)
    table = kvq.rope_table(f, 16)
    c = kvq.KVCache("q4_0", B, H, D, 16)
    want = kvq.rope_store(c, table, k, v, 2, q=q)
    first = {(t, m): y.clone() for t, p in c.planes.items() for m, y in p.items()}
    for at in (0, out + size):
        got = buf[at:at + out].view(B, Hq, n, D)
        assert kvq.rope_store(c, table, k, v, 2, q=q, q_out=got) is got and torch.equal(got, want)
        for (t, m), y in first.items():
            assert torch.equal(c.planes[t][m], y)
    for at in (8, out, out + 8 * D, size + out - 8):
        with pytest.raises(kvq.KvqError, match="overlaps"):
            kvq.rope_store(c, table, k, v, 2, q=q, q_out=buf[at:at + out].view(B, Hq, n, D))
    same = q[:1, :, :1]
    with pytest.raises(kvq.KvqError, match="overlaps"):
        kvq.rope_store(kvq.KVCache("q4_0", 1, H, D, 16), table, k[:1, :, :1], v[:1, :, :1], 2, q=same, q_out=same)


# An entry's error, step by step: the angle is held to 2^-33 of a turn; what is left of it after the nearest quarter
# turn, at most pi / 4, is rounded to float32; the polynomials in z = u^2 (z, and their last sum but one, rounded: at
# most 4 roundings of 2^-26 in the entry) end in one addition to a value below 1; the magnitude's product is rounded.
ENTRY_TOL = 2 * math.pi * 2.0 ** -33 + math.pi / 4 * 2.0 ** -24 + 4 * 2.0 ** -26 + 2.0 ** -25


@pytest.mark.parametrize("rot,n_pos,pos0", [(64, 2000, 0), (128, 40000, 7), (256, 333, 2 ** 20)])
@pytest.mark.parametrize("scaling", ["none", "yarn"])
def test_table_entries_by_the_kernels_own_steps(rot, n_pos, pos0, scaling):
    """In 64 bits an angle below 2^21 radians is off by 2^-32 at most."""
    f, mag = kvq.rope_frequencies(rot, 10000.0, scaling, 4.0, 4096)
    got = kvq.rope_table(f, n_pos, pos0=pos0, magnitude=mag).cpu().numpy()
    want = OR.table(f.numpy(), pos0, n_pos, np.float32(mag))
    worst = np.abs(got - want).max()
    print(worst, ENTRY_TOL * mag)
    assert worst <= ENTRY_TOL * mag + (2.0 ** -24 if mag != 1 else 0) + 2.0 ** -32


def test_table_entries_of_far_positions_by_the_kernels_own_steps():
    """Against angles in rational arithmetic."""
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494")
    f = torch.linspace(0.0, 3.0, 64, dtype=torch.float64)
    for pos0 in (10 ** 6 + 1, 2 ** 31 - 9):
        got = kvq.rope_table(f, 8, pos0=pos0).cpu().numpy()
        for p in range(8):
            a = np.array([float((Decimal(pos0 + p) * Decimal(x)) % two_pi) for x in f.tolist()])
            assert np.abs(got[p, :64] - np.cos(a)).max() <= ENTRY_TOL + 1e-15
            assert np.abs(got[p, 64:] - np.sin(a)).max() <= ENTRY_TOL + 1e-15
