"""Block bounds, block selection and attention over selected blocks, in every layout, and the three as a decode loop uses them
behind a page plan."""
import numpy as np
import pytest
import torch

import sub_byte_quantized_gb300 as kvq
from oracle import attention as OA, quant as Q, serving as OV
from tests.gpu_helpers import check_close

pytestmark = pytest.mark.gpu
LAYOUTS = ["q4_0", "q6_0", "q8_0", "asym4_g32", "had_int4", "had_int2", "int8_b64", "e4m3_b64", "q4_0+q8_0", "had_int2+had_int4"]
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _oracle(layout, B, H, D, cap):
    return OV.BlockCache(layout, B, H, D, cap) if layout in OV.TOP else OA.OracleCache(layout, B, H, D, cap)


def _make(layout, B, H, D, S, page=0, seed=0):
    """A filled device cache (contiguous, or a pool with a shuffled table) and its oracle."""
    rng = np.random.default_rng(seed)
    cap = (S + 63) // 64 * 64 + 64
    k, v = (rng.standard_normal((B, H, S, D)).astype(np.float32) for _ in range(2))
    k[..., rng.permutation(D)[:4]] *= 6.0
    k += np.repeat(rng.standard_normal((B, H, cap // 64, D)), 64, 2)[:, :, :S].astype(np.float32)     # blocks that differ
    o = _oracle(layout, B, H, D, cap)
    o.store(k, v, [0] * B if layout in OV.TOP else 0)
    kd, vd = (torch.from_numpy(x).cuda() for x in (k, v))
    if not page:
        c = kvq.KVCache(layout, B, H, D, cap)
        kvq.store(c, kd, vd, 0)
        return c, o, None
    per = -(-cap // page)
    c = kvq.PagedKVCache(layout, B, H, D, page, B * per + 2, per)
    table = torch.from_numpy(rng.permutation(B * per + 2)[:B * per].reshape(B, per))
    c.set_block_table(table)
    kvq.paged_store(c, kd, vd, torch.zeros(B, dtype=torch.int32, device="cuda"))
    return c, o, table.cuda()


def _logical(x, table):
    """A plane of bounds as [B][H][blocks][...]."""
    return x if table is None else x[table].transpose(1, 2).flatten(2, 3)


def _queries(B, Hq, n_q, D, dtype="bf16", seed=1):
    q = torch.from_numpy(np.random.default_rng(seed).standard_normal((B, Hq, n_q, D)).astype(np.float32)).to(DT[dtype])
    return q.cuda(), q.float().numpy()


def _limits(lens, n_q, causal):
    return [[n - n_q + i if causal else n - 1 for i in range(n_q)] for n in lens]


def _bounds(c, o, table, lens):
    b = kvq.BlockBounds(c)
    if table is None:
        kvq.block_bounds(c, b, 0, lens[0])
    else:
        kvq.paged_block_bounds(c, b, torch.tensor(lens, dtype=torch.int32, device="cuda"), max(max(lens), 1))
    codes, scale = _logical(b.codes, table).cpu().numpy(), _logical(b.scale, table).cpu().numpy()
    for i, n in enumerate(lens):
        for h in range(c.n_kv_heads):
            if n:
                wc, ws = OV.bounds(OV.key_rows(o, i, h, n))
                assert np.array_equal(scale[i, h, :len(ws)].view(np.uint32), ws.view(np.uint32)), (i, h)
                assert np.array_equal(codes[i, h, :len(ws)], wc), (i, h)
            assert not scale[i, h, -(-n // 64):].any()
    return b, codes, scale


def _rotated(layout, q):
    return Q.rotate(q) if layout.startswith("had") else q


def _select(c, b, codes, scale, layout, q, qn, lens, causal, n_sel, sink, recent):
    B, H, n_q = c.batch, c.n_kv_heads, q.shape[2]
    g = q.shape[1] // H
    if isinstance(c, kvq.KVCache):
        got = kvq.block_select(c, b, q, lens[0], n_sel, sink, recent, causal=causal, q_pos0=lens[0] - n_q if causal else 0)
    else:
        got = kvq.paged_block_select(c, b, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), max(max(lens), 1), n_sel, sink, recent, causal=causal)
    qr = _rotated(layout, qn)
    for i in range(B):
        for h in range(H):
            want = OV.select(codes[i, h], scale[i, h], qr[i, h * g:(h + 1) * g], _limits(lens, n_q, causal)[i], n_sel, sink, recent)
            assert np.array_equal(got[i, h].cpu().numpy(), want), (i, h)
    return got


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("page", [0, 64, 128])
def test_bounds_and_selection(layout, D, page):
    B, H, S = 2, 2, 1000
    c, o, table = _make(layout, B, H, D, S, page)
    lens = [S, S] if not page else [S, 333]
    b, codes, scale = _bounds(c, o, table, lens)
    for gqa, n_q, dtype, causal, n_sel, sink, recent in ((1, 1, "bf16", False, 5, 1, 1), (4, 1, "f32", False, 3, 0, 0), (9, 3, "f16", True, 7, 2, 3), (2, 70, "bf16", True, 15, 1, 1),
                                                         (1, 1, "bf16", False, 40, 1, 1), (1, 2, "f16", False, 1, 0, 1)):
        q, qn = _queries(B, H * gqa, n_q, D, dtype)
        _select(c, b, codes, scale, layout, q, qn, lens, causal, n_sel, sink, recent)


def test_bounds_are_renewed_where_tokens_are_new():
    """Only the blocks of the newest tokens change; a length inside a block leaves its later rows out; empty sequences."""
    c, o, table = _make("q4_0", 4, 2, 128, 500, 64)
    lens = [0, 1, 129, 500]
    b, codes, scale = _bounds(c, o, table, lens)
    b.codes.fill_(5)
    b.scale.fill_(7.0)
    d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kvq.paged_block_bounds(c, b, d, 2)
    got, s = _logical(b.codes, table).cpu().numpy(), _logical(b.scale, table).cpu().numpy()
    for i, blocks in enumerate(([], [0], [1, 2], [7])):
        for blk in range(s.shape[2]):
            if blk in blocks:
                assert np.array_equal(got[i, :, blk], codes[i, :, blk]) and np.array_equal(s[i, :, blk], scale[i, :, blk])
            else:
                assert (got[i, :, blk] == 5).all() and (s[i, :, blk] == 7.0).all()
    c, o, _ = _make("int8_b64", 1, 2, 128, 300)
    b, codes, scale = _bounds(c, o, None, [300])
    b.codes.fill_(5)
    kvq.block_bounds(c, b, 130, 300)
    assert (b.codes[:, :, :2] == 5).all() and np.array_equal(b.codes[:, :, 2:5].cpu().numpy(), codes[:, :, 2:5]) and (b.codes[:, :, 5:] == 5).all()


def test_selection_of_equal_scores_and_zero_queries():
    """Ties go to the lowest index; a zero query scores every block 0; blocks of zeros."""
    B, H, D, S = 1, 2, 128, 64 * 20
    c = kvq.KVCache("q8_0", B, H, D, S)
    k = torch.ones((B, H, S, D), device="cuda")
    k[:, 1, 640:] = 0.0
    kvq.store(c, k, k, 0)
    b = kvq.BlockBounds(c)
    kvq.block_bounds(c, b, 0, S)
    q = torch.ones((B, 4, 3, D), device="cuda")
    q[:, :, 1] = 0.0
    q[:, :, 2] = -1.0
    got = kvq.block_select(c, b, q, S, 4, n_sink=0, n_recent=0).cpu().numpy()
    assert got[0, 0].tolist() == [[0, 1, 2, 3]] * 3
    assert got[0, 1].tolist() == [[0, 1, 2, 3], [0, 1, 2, 3], [10, 11, 12, 13]]


def test_selection_over_many_blocks():
    """More blocks than one CTA of the selection takes: bounds given, 300000 blocks of which few are looked at."""
    n, D, n_sel = 20000, 128, 333
    c = kvq.KVCache("had_int2", 1, 1, D, 64 * n)
    b = kvq.BlockBounds(c)
    g = torch.Generator("cuda").manual_seed(1)
    b.codes.copy_(torch.randint(-127, 128, b.codes.shape, device="cuda", generator=g))
    b.scale.copy_(torch.rand(b.scale.shape, device="cuda", generator=g))
    q, qn = _queries(1, 3, 2, D)
    got = kvq.block_select(c, b, q, 64 * n - 5, n_sel, 4, 7, causal=True, q_pos0=64 * n - 100).cpu().numpy()
    want = OV.select(b.codes[0, 0].cpu().numpy(), b.scale[0, 0].cpu().numpy(), Q.rotate(qn)[0], [64 * n - 100, 64 * n - 99], n_sel, 4, 7)
    assert np.array_equal(got[0, 0], want)


def _lists(rng, B, H, limits, n_sel):
    """Ascending lists with ends of every kind: full ones, short ones, empty ones, the row's last block and not."""
    n_q = len(limits[0])
    sel = np.full((B, H, n_q, n_sel), -1, np.int32)
    for b in range(B):
        for h in range(H):
            for i in range(n_q):
                n = limits[b][i] // 64 + 1 if limits[b][i] >= 0 else 0
                m = min(n, rng.integers(0, n_sel + 1)) if rng.random() < 0.5 else min(n, n_sel)
                sel[b, h, i, :m] = np.sort(rng.permutation(n)[:m])
    return sel


def _gathered(c, table, b, h, blocks, layout, D):
    """A one-sequence cache of the listed blocks' rows."""
    d = kvq.KVCache(layout, 1, 1, D, 64 * len(blocks))
    at = torch.as_tensor(np.concatenate([np.arange(64 * e, 64 * e + 64) for e in blocks]), device="cuda")
    for t in ("k", "v"):
        for name, x in d.planes[t].items():
            x.copy_(_logical(c.planes[t][name], table)[b, h][at[::64] // 64 if x.shape[2] != len(at) else at][None, None])
    return d


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("page", [0, 64, 256])
@pytest.mark.parametrize("gqa,n_q,dtype,causal", [(4, 1, "bf16", False), (1, 1, "f32", False), (3, 4, "f16", True), (12, 2, "bf16", True)])
def test_sparse_attention(layout, D, page, gqa, n_q, dtype, causal):
    B, H, S = 2, 2, 700
    c, o, table = _make(layout, B, H, D, S, page)
    lens = [S, S] if not page else [130, S]
    q, qn = _queries(B, H * gqa, n_q, D, dtype)
    limits = _limits(lens, n_q, causal)
    for seed, n_sel in ((0, 4), (1, 11), (2, 1)):
        sel = _lists(np.random.default_rng(seed), B, H, limits, n_sel)
        sd = torch.from_numpy(sel).cuda()
        for chunk in (0, 64):
            if page:
                got = kvq.paged_sparse_attend(c, q, sd, torch.tensor(lens, dtype=torch.int32, device="cuda"), S, causal=causal, chunk=chunk)
            else:
                got = kvq.sparse_attend(c, q, sd, S, causal=causal, q_pos0=S - n_q if causal else 0, chunk=chunk)
            if layout in ("int8_b64", "e4m3_b64"):
                want, tol = o.attend(qn, 1 / np.sqrt(D), lens, causal, sel)
                assert (np.abs(got.cpu().numpy() - want) <= tol).all()
                continue
            # the dense call over the same rows, moved together
            for b in range(B):
                for h in range(H):
                    for i in range(n_q):
                        blocks = sel[b, h, i][sel[b, h, i] >= 0]
                        x = got[b, h * gqa:(h + 1) * gqa, i:i + 1]
                        if not len(blocks):
                            assert not x.any()
                            continue
                        n = 64 * (len(blocks) - 1) + min(64, limits[b][i] + 1 - 64 * blocks[-1])
                        ref = kvq.decode_attend(_gathered(c, table, b, h, blocks, layout, D), q[b:b + 1, h * gqa:(h + 1) * gqa, i:i + 1].contiguous(), int(n))
                        assert (x - ref[0]).norm() <= 2e-5 * ref.norm(), (b, h, i, float((x - ref[0]).norm() / ref.norm()))


@pytest.mark.parametrize("layout", ["q4_0", "had_int4", "int8_b64"])
def test_every_block_is_the_dense_attention(layout):
    c, o, table = _make(layout, 2, 2, 128, 700, 64)
    q, qn = _queries(2, 8, 1, 128)
    lens = torch.tensor([700, 65], dtype=torch.int32, device="cuda")
    sel = torch.full((2, 2, 1, 12), -1, dtype=torch.int32, device="cuda")
    sel[0, :, :, :11] = torch.arange(11)
    sel[1, :, :, :2] = torch.arange(2)
    got, want = kvq.paged_sparse_attend(c, q, sel, lens, 700), kvq.paged_decode_attend(c, q, lens, 700)
    assert (got - want).norm() <= 1e-5 * want.norm()
    check_close(got.cpu().numpy(), want.double().cpu().numpy())


def test_lists_that_are_not_lists():
    """A list ends at the first entry that does not ascend, is negative or lies behind what the row sees; no access leaves the cache."""
    c, o, table = _make("int8_b64", 1, 2, 128, 700, 64)
    q, qn = _queries(1, 4, 1, 128)
    sel = np.array([[[[3, 3, 5, 6]], [[2, 9, 10, 2 ** 31 - 1]]], [[[-5, 1, 2, 3]], [[11, 0, 1, 2]]], [[[4, -1, 6, 7]], [[0, 2, 1, 9]]]], np.int32)
    for s in sel:
        got = kvq.paged_sparse_attend(c, q, torch.from_numpy(s[None]).cuda(), torch.tensor([700], dtype=torch.int32, device="cuda"), 700)
        clean = s[None].copy()
        clean[clean > 10] = -1
        want, tol = o.attend(qn, 1 / np.sqrt(128), [700], False, clean)
        assert (np.abs(got.cpu().numpy() - want) <= tol).all()


def test_serving_loop():
    """plan -> ragged append -> bounds -> selection -> sparse attention, step after step, requests coming, growing and ending."""
    rng = np.random.default_rng(11)
    B, H, Hq, D, page, per, n_pages, n_sel = 4, 2, 8, 128, 64, 8, 24, 4
    for layout in ("e4m3_b64", "q8_0"):
        c = kvq.PagedKVCache(layout, B, H, D, page, n_pages, per)
        bounds = kvq.BlockBounds(c)
        free = torch.from_numpy(rng.permutation(n_pages)).to(torch.int32).cuda()
        state = dict(lens=torch.zeros(B, dtype=torch.int32, device="cuda"), n_free=torch.tensor([n_pages], dtype=torch.int32, device="cuda"))
        oracle = [_oracle(layout, 1, H, D, page * per) for _ in range(B)]
        lens = [0] * B
        for step, new in enumerate(([200, 65, 0, 400], [1, 1, 130, 1], [1, -1, 1, 1], [1, 300, 1, -1], [3, 1, 1, 500], [1, 1, 1, 1])):
            nd = torch.tensor(new, dtype=torch.int32, device="cuda")
            p = kvq.page_plan(state["lens"], nd, c.block_table, page, free, state["n_free"], 640, lens_out=state["lens"], n_free_out=state["n_free"])
            granted = p.granted.tolist()
            k, v = (rng.standard_normal((640, H, D)).astype(np.float32) for _ in range(2))
            kvq.paged_store_slots(c, *(torch.from_numpy(x).cuda() for x in (k, v)), p.slots)
            at = 0
            for b in range(B):
                if new[b] < 0:
                    lens[b] = 0
                if granted[b]:
                    kk, vv = (x[at:at + granted[b]].transpose(1, 0, 2)[None] for x in (k, v))
                    oracle[b].store(kk, vv, [lens[b]] if layout in OV.TOP else lens[b])
                lens[b] += granted[b]
                at += granted[b]
            assert p.lens.tolist() == lens and p.cu_new.tolist()[-1] == at
            kvq.paged_block_bounds(c, bounds, p.lens, max(max(granted), 1))
            q, qn = _queries(B, Hq, 1, D, seed=step)
            sel = kvq.paged_block_select(c, bounds, q, p.lens, page * per, n_sel)
            out = kvq.paged_sparse_attend(c, q, sel, p.lens, page * per).cpu().numpy()
            for b in range(B):
                for h in range(H):
                    if lens[b]:
                        codes, scale = OV.bounds(OV.key_rows(oracle[b], 0, h, lens[b]))
                        want = OV.select(codes, scale, qn[b, h * 4:h * 4 + 4], [lens[b] - 1], n_sel, 1, 1)
                        assert np.array_equal(sel[b, h].cpu().numpy(), want)

                def values(t, _, h, n, o=oracle[b]):
                    return o.values(t, 0, h, n) if layout in OV.TOP else o.dequantized(t, n)[0, h]
                want, tol = OV.attend(values, H, qn[b:b + 1], 1 / np.sqrt(D), [lens[b]], False, sel[b:b + 1].cpu().numpy())
                assert (np.abs(out[b:b + 1] - want) <= tol + (2e-5 * np.abs(want).max() if layout == "q8_0" else 0)).all(), (layout, step, b)


def test_wrappers_refuse():
    c, _, _ = _make("q4_0", 1, 2, 128, 100)
    b, other = kvq.BlockBounds(c), kvq.BlockBounds(kvq.KVCache("q4_0", 1, 2, 128, 64))
    q, _ = _queries(1, 4, 1, 128)
    sel = torch.zeros((1, 2, 1, 3), dtype=torch.int32, device="cuda")
    for f in (lambda: kvq.block_bounds(c, other, 0, 10), lambda: kvq.block_select(c, other, q, 100, 2), lambda: kvq.block_select(c, b, q.cpu(), 100, 2),
              lambda: kvq.block_select(c, b, q[..., ::2], 100, 2), lambda: kvq.block_select(c, b, q, 100, 2, sel=sel),
              lambda: kvq.sparse_attend(c, q, sel.long(), 100), lambda: kvq.sparse_attend(c, q, sel[:, :1], 100), lambda: kvq.sparse_attend(c, q, sel.cpu(), 100),
              lambda: kvq.sparse_attend(c, q, sel, 100, out=torch.empty((1, 4, 1, 128), dtype=torch.float16, device="cuda"))):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(kvq.KvqError):
        kvq.sparse_attend(c, q, sel, 1000)
