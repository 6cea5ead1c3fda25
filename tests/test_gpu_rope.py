"""Rotary table and rotary appends against the oracle: the table within a few roundings of the 64-bit
value at near and far positions, q and the packed planes bit for bit."""
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import sub_byte_quantized_gb300 as kvq
from oracle import attention as OA, paged as OP, rope as OR
from tests.gpu_helpers import planes_equal
from sub_byte_quantized_gb300._lib import KvqError

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# sinpif and cospif are off by at most one ulp (2^-23), their argument by one rounding (0.8 * 2^-24 in the
# value), the magnitude's product by one more; values are at most the magnitude
TABLE_TOL = 2.0 ** -23 + 2 * 2.0 ** -24


@pytest.mark.parametrize("rot,n_pos,pos0", [(16, 1, 0), (48, 37, 5), (128, 1000, 0), (256, 3, 100), (112, 4099, 77)])
@pytest.mark.parametrize("scaling", ["none", "yarn"])
def test_table(rot, n_pos, pos0, scaling):
    f, mag = kvq.rope_frequencies(rot, 10000.0, scaling, 4.0, 4096)
    got = kvq.rope_table(f, n_pos, pos0=pos0, magnitude=mag).cpu().numpy()
    want = OR.table(f.numpy(), pos0, n_pos, np.float32(mag))
    assert np.abs(got - want).max() <= TABLE_TOL * mag


def test_table_of_far_positions():
    """Every quarter turn and the last positions an int32 holds, against exact rational angles."""
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494")
    f = torch.tensor([1.0, math.pi / 2, 0.1234567, 1e-9, 0.0, 65536.0, 3.0, 2.0 ** -40], dtype=torch.float64)
    for pos0 in (0, 10 ** 6, 2 ** 31 - 9):
        got = kvq.rope_table(f, 8, pos0=pos0).cpu().numpy()
        for p in range(8):
            for i, x in enumerate(f.tolist()):
                a = float((Decimal(pos0 + p) * Decimal(x)) % two_pi)
                # a's own rounding: at most 2 pi * 2^-53
                assert abs(got[p, i] - math.cos(a)) <= TABLE_TOL + 1e-15
                assert abs(got[p, 8 + i] - math.sin(a)) <= TABLE_TOL + 1e-15


def test_table_into_a_given_buffer_on_another_stream():
    f, _ = kvq.rope_frequencies(64)
    out = torch.full((10, 64), float("nan"), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert kvq.rope_table(f, 10, out=out, stream=s) is out
    s.synchronize()
    assert torch.equal(out, kvq.rope_table(f, 10))
    assert kvq.rope_table(f, 0).shape == (0, 64)
    with pytest.raises(ValueError):
        kvq.rope_table(f, 11, out=out)
    with pytest.raises(ValueError):
        kvq.rope_table(f.float(), 11)


def _round(x, dtype):
    return torch.from_numpy(x).to(DT[dtype])


def _inputs(seed, B, Hq, H, n, D, dtype, fused=True):
    """q, k, v views of one projection's output (or of separate tensors), and their float32 values."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, n, (Hq + 2 * H) * D), generator=g)
    x[..., torch.randperm(x.shape[-1], generator=g)[:5]] *= 8.0
    x = x.to(DT[dtype]).cuda()
    v = x.view(B, n, Hq + 2 * H, D).transpose(1, 2)
    parts = [v[:, :Hq], v[:, Hq:Hq + H], v[:, Hq + H:]]
    if not fused:
        parts = [t.contiguous() for t in parts]
    return parts, [t.float().cpu().numpy() for t in parts]


def _table(rot, n_pos, seed=0):
    f, _ = kvq.rope_frequencies(rot, 10000.0 + seed)
    t = kvq.rope_table(f, n_pos)
    return t, t.cpu().numpy()


def _check(layout, D, B, Hq, H, n, rot, interleaved, dtype, pos0, cap, n_recent=0, positions=None, fused=True, seed=3):
    (q, k, v), (q32, k32, v32) = _inputs(seed, B, Hq, H, n, D, dtype, fused)
    table, t32 = _table(rot, 3 * cap)
    dc = kvq.KVCache(layout, B, H, D, cap, n_recent=n_recent)
    oc = OA.OracleCache(layout, B, H, D, cap, n_recent=n_recent)
    at = np.broadcast_to(np.arange(pos0, pos0 + n), (B, n)) if positions is None else positions
    rows = t32[np.clip(at, 0, 3 * cap - 1)][:, None]
    oc.store(OR.rotate(k32, rows, interleaved), v32, pos0)
    pos = None if positions is None else torch.from_numpy(np.ascontiguousarray(positions, dtype=np.int32)).cuda()
    got = kvq.rope_store(dc, table, k, v, pos0, q=q, positions=pos, interleaved=interleaved)
    planes_equal(dc, oc)
    assert torch.equal(got.cpu(), _round(OR.rotate(q32, rows, interleaved), dtype))
    return dc


@pytest.mark.parametrize("layout", ["q4_0", "q6_0", "q8_0", "asym4_g32", "had_int4", "had_int2", "q4_0+q8_0", "had_int2+had_int4"])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_store_layouts(layout, D, interleaved):
    for dtype, rot, n in (("bf16", D, 1), ("f32", 48, 5), ("f16", 16, 37)):
        _check(layout, D, 2, 6, 3, n, rot, interleaved, dtype, 3, 64, n_recent=8 if "had" in layout else 0)


@pytest.mark.parametrize("rot", [16, 32, 80, 96, 112, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_rope_store_partial_dims(rot, dtype):
    for interleaved in (False, True):
        _check("q8_0", 128, 1, 4, 2, 9, rot, interleaved, dtype, 0, 16)
        _check("had_int4", 128, 1, 4, 2, 9, rot, interleaved, dtype, 0, 16, n_recent=4)


def test_rope_store_positions_apart_from_slots():
    pos = np.array([[7, 100, 2], [150, 0, 191]])
    _check("q4_0", 128, 2, 4, 2, 3, 128, False, "bf16", 11, 64, positions=pos)
    # positions outside the table are clamped into it
    _check("q4_0", 128, 2, 4, 2, 3, 128, True, "bf16", 11, 64, positions=np.array([[-5, 192, 2 ** 31 - 1], [-2 ** 31, 3, 4]]))


def test_rope_store_dense_inputs_many_rows():
    _check("asym4_g32", 256, 1, 8, 4, 700, 64, True, "f16", 0, 701, fused=False)
    _check("had_int4", 128, 2, 4, 2, 300, 128, False, "bf16", 5, 320, n_recent=64, fused=False)


def test_rope_store_without_queries_equals_store_of_rotated_keys():
    (_, k, v), (_, k32, v32) = _inputs(5, 1, 2, 2, 6, 128, "f32")
    table, t32 = _table(64, 100)
    a, b = (kvq.KVCache("q6_0", 1, 2, 128, 32) for _ in range(2))
    assert kvq.rope_store(a, table, k, v, 4) is None
    kvq.store(b, torch.from_numpy(OR.rotate(k32, t32[4:10][None, None])).cuda(), v.contiguous(), 4)
    for t in ("k", "v"):
        for name in a.planes[t]:
            assert torch.equal(a.planes[t][name], b.planes[t][name])
    kvq.rope_store(a, table, k[:, :, :0], v[:, :, :0], 32)                    # nothing to append


@pytest.mark.parametrize("layout,D,n_recent", [("q4_0", 128, 0), ("had_int2", 128, 4), ("asym4_g32", 256, 0), ("q4_0+q8_0", 128, 0)])
def test_paged_rope_store(layout, D, n_recent):
    B, Hq, H, n, page, per = 3, 4, 2, 5, 64, 3
    (q, k, v), (q32, k32, v32) = _inputs(9, B, Hq, H, n, D, "bf16")
    table, t32 = _table(96, 500)
    dc = kvq.PagedKVCache(layout, B, H, D, page, B * per, per, n_recent=n_recent)
    tab = np.random.default_rng(2).permutation(B * per).reshape(B, per)
    dc.set_block_table(tab)
    oc = OP.OraclePagedCache(layout, B, H, D, page, B * per, per, n_recent, tab)
    # a page border, the last row that fits and beyond it, and slots before the sequence: rows outside are
    # not written, their queries are
    slots = np.array([62, per * page - 2, -3], np.int32)
    at = slots[:, None] + np.arange(n)
    rows = t32[np.clip(at, 0, 499)][:, None]
    oc.store(OR.rotate(k32, rows), v32, slots)
    got = kvq.paged_rope_store(dc, table, k, v, torch.from_numpy(slots).cuda(), q=q)
    for t in ("k", "v"):
        for name, op in oc.planes[t].items():
            assert np.array_equal(dc.planes[t]["recent" if name == "ring" else name].cpu().numpy(), op), (t, name)
    assert torch.equal(got.cpu(), _round(OR.rotate(q32, rows), "bf16"))


def test_paged_slot_whose_end_passes_int32():
    """slots[b] + j beyond int32 is outside the sequence, not a small slot."""
    (q, k, v), _ = _inputs(1, 1, 2, 2, 3, 128, "bf16")
    table, _ = _table(128, 10)
    dc = kvq.PagedKVCache("q4_0", 1, 2, 128, 64, 1, 1)
    before = dc.planes["k"]["payload"].clone()
    kvq.paged_rope_store(dc, table, k, v, torch.tensor([2 ** 31 - 2], dtype=torch.int32, device="cuda"), q=q)
    assert torch.equal(dc.planes["k"]["payload"], before)


def test_broadcast_and_refused_views():
    table, t32 = _table(128, 20)
    dc = kvq.KVCache("q8_0", 2, 2, 128, 16)
    k = torch.randn((1, 1, 4, 128), device="cuda")
    kb = k.expand(2, 2, 4, 128)                                                # strides of 0
    kvq.rope_store(dc, table, kb, kb, 0)
    oc = OA.OracleCache("q8_0", 2, 2, 128, 16)
    k32 = np.broadcast_to(k.cpu().numpy(), (2, 2, 4, 128))
    oc.store(OR.rotate(k32, t32[:4][None, None]), k32, 0)
    planes_equal(dc, oc)
    odd = torch.randn((2, 2, 4, 130), device="cuda")[..., :128]                # rows not 16-byte aligned
    with pytest.raises(KvqError):
        kvq.rope_store(dc, table, odd, odd, 0)
    with pytest.raises(ValueError):
        kvq.rope_store(dc, table, kb.transpose(2, 3).contiguous().transpose(2, 3), kb, 0)
    with pytest.raises(ValueError):
        kvq.rope_store(dc, table, kb, kb.half(), 0)
    with pytest.raises(ValueError):
        kvq.rope_store(dc, table, kb, kb, 0, q=torch.randn((2, 4, 3, 128), device="cuda"))
    with pytest.raises(ValueError):
        kvq.rope_store(dc, table, kb, kb, 0, positions=torch.zeros((2, 4), dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        kvq.rope_store(dc, table.cpu(), kb, kb, 0)


@pytest.mark.parametrize("layout", ["q4_0", "q6_0", "q8_0", "asym4_g32", "q8_0+q4_0"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_store_prompts(layout, dtype, interleaved):
    """Rows enough for blocks of several passes: whole ones, and a last one that ends inside a pass."""
    _check(layout, 128, 2, 4, 2, 301, 128, interleaved, dtype, 7, 320)
    _check(layout, 128, 1, 2, 1, 128, 80, interleaved, dtype, 0, 128, fused=False)
    _check(layout, 256, 1, 4, 2, 145, 256, interleaved, dtype, 3, 160)
    _check(layout, 256, 1, 1, 1, 65, 112, interleaved, dtype, 0, 70, positions=np.arange(64, -1, -1)[None] * 3 % 200)
