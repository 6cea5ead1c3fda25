"""The 8-bit layouts with a scale per block of 64 tokens: appends bit for bit, attention against the float64 oracle within
what float32 arithmetic may be off by, through every entry point that takes a layout."""
import numpy as np
import pytest
import torch

import sub_byte_quantized_gb300 as kvq
from oracle import serving as OV
from sub_byte_quantized_gb300 import api

pytestmark = pytest.mark.gpu
LAYOUTS = ["int8_b64", "e4m3_b64"]
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _rows(rng, shape, dtype="bf16", scale=1.0):
    x = (rng.standard_normal(shape) * scale).astype(np.float32)
    x[..., rng.permutation(shape[-1])[:4]] *= 6.0
    t = torch.from_numpy(x).to(DT[dtype])
    return t.cuda(), t.float().numpy()


def _logical(cache, b_table=None):
    """Device planes as [B][H][cap] rows and [B][H][cap / 64] scales."""
    out = {}
    for t, pl in cache.planes.items():
        p, s = pl["payload"], pl["scale"]
        if b_table is not None:
            p, s = (x[b_table].transpose(1, 2).flatten(2, 3) for x in (p, s))
        out[t] = (p.cpu().numpy(), s.cpu().numpy())
    return out


def _same(cache, oracle, table=None, lens=None):
    for t, (p, s) in _logical(cache, table).items():
        want = oracle.planes[t]
        assert np.array_equal(s.view(np.uint32), want["scale"].view(np.uint32)), t
        if lens is None:
            assert np.array_equal(p, want["payload"]), t
        else:
            for b, n in enumerate(lens):
                assert np.array_equal(p[b, :, :n], want["payload"][b, :, :n]), (t, b)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_contiguous_appends(layout, D, dtype):
    """Appends of one row, a few, whole blocks, across blocks, growing and shrinking values, and a block begun again."""
    rng = np.random.default_rng(1)
    B, H, cap = 2, 3, 320
    c, o = kvq.KVCache(layout, B, H, D, cap), OV.BlockCache(layout, B, H, D, cap)
    pos = 0
    for n, scale in ((1, 1e-3), (1, 1.0), (2, 3e-4), (5, 40.0), (1, 41.0), (8, 900.0), (9, 1.0), (100, 5e3), (1, 1e-6), (64, 1.0), (63, 2e4)):
        (k, kn), (v, vn) = (_rows(rng, (B, H, n, D), dtype, scale) for _ in range(2))
        kvq.store(c, k, v, pos)
        o.store(kn, vn, [pos] * B)
        _same(c, o)
        pos += n
    for n, at in ((64, 64), (10, 128), (1, 200), (0, 0)):
        (k, kn), (v, vn) = (_rows(rng, (B, H, n, D), dtype, 0.1) for _ in range(2))
        kvq.store(c, k, v, at)
        o.store(kn, vn, [at] * B)
        _same(c, o)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_append_extremes(layout):
    """Zero rows, the smallest subnormals, the largest values, half-way quotients, a scale that grows by 2^200."""
    D, cap = 128, 256
    c, o = kvq.KVCache(layout, 1, 1, D, cap), OV.BlockCache(layout, 1, 1, D, cap)
    rng = np.random.default_rng(2)
    rows = [np.zeros(D), np.full(D, 2.0 ** -149), np.full(D, 1e-40), rng.standard_normal(D) * 1e-38, rng.standard_normal(D), np.zeros(D),
            np.linspace(-3.0e38, 3.0e38, D), np.full(D, np.finfo(np.float32).max)]
    half = np.arange(D) - 63.5
    half[0] = 127.0
    blocks = [rows, [half, half * 0.5, half * 4.0], [np.full(D, -0.0), -np.linspace(0, 1, D)], [np.linspace(0, 1, D) * 2.0 ** -100, np.linspace(0, 1, D) * 2.0 ** 100]]
    with np.errstate(over="ignore"):
        for i, block in enumerate(blocks):
            for j, r in enumerate(block):
                x = r.astype(np.float32).reshape(1, 1, 1, D)
                d = torch.from_numpy(x).cuda()
                kvq.store(c, d, d.flip(-1).contiguous(), 64 * i + j)
                o.store(x, x[..., ::-1], [64 * i + j])
                _same(c, o)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("page", [64, 128])
def test_paged_and_ragged_appends(layout, page):
    """paged_store with positions that begin in front of the sequence or pass its end, and the same bytes by slots."""
    rng = np.random.default_rng(3)
    B, H, D, per = 4, 2, 128, 512 // page
    a, b = (kvq.PagedKVCache(layout, B, H, D, page, 2 * B * per, per) for _ in range(2))
    table = torch.from_numpy(rng.permutation(2 * B * per)[:B * per].reshape(B, per))
    a.set_block_table(table)
    o = OV.BlockCache(layout, B, H, D, 512)
    pos = np.array([0, 61, 128, -2])
    for n, scale in ((3, 1.0), (1, 30.0), (70, 2.0), (1, 100.0), (130, 3.0), (200, 1.0)):
        (k, kn), (v, vn) = (_rows(rng, (B, H, n, D), "bf16", scale) for _ in range(2))
        kvq.paged_store(a, k, v, torch.from_numpy(pos.astype(np.int32)).cuda())
        o.store(kn, vn, pos)
        _same(a, o, table.cuda())
        p = torch.from_numpy(pos)[:, None] + torch.arange(n)
        ok = (p >= 0) & (p < 512)
        at = p.clamp(0, 511)
        slots = torch.where(ok, torch.gather(table, 1, at // page) * page + at % page, -1).flatten().cuda()
        tok = torch.cat((k, v), 1).transpose(1, 2).reshape(B * n, 2, H, D)
        kvq.paged_store_slots(b, tok[:, 0], tok[:, 1], slots)
        for t in ("k", "v"):
            for name in ("payload", "scale"):
                assert torch.equal(a.planes[t][name], b.planes[t][name])
        pos = pos + n


def test_ragged_append_of_mixed_runs():
    """Prompts, single rows and pages that lie next to each other in the pool, in one call."""
    rng = np.random.default_rng(5)
    H, D, page, n_pages = 2, 128, 64, 24
    c = kvq.PagedKVCache("int8_b64", 1, H, D, page, n_pages, 1)
    o = OV.BlockCache("int8_b64", 1, H, D, page * n_pages)
    runs = [(0, 200), (640, 1), (705, 1), (770, 3), (832, 64), (896, 64), (1000, 9), (1023, 1), (1100, 8), (64 * 20 + 60, 4)]
    slots = np.concatenate([np.arange(a, a + n) for a, n in runs])
    order = [np.arange(a, a + n) for a, n in runs]
    for _ in range(2):
        (k, kn), (v, vn) = (_rows(rng, (len(slots), H, D), "f16") for _ in range(2))
        kvq.paged_store_slots(c, k, v, torch.from_numpy(slots).cuda())
        i = 0
        for at in order:
            for x, t in ((kn, "k"), (vn, "v")):
                o.append(t, 0, x[i:i + len(at)].transpose(1, 0, 2), int(at[0]))
            i += len(at)
        for t in ("k", "v"):
            assert np.array_equal(c.planes[t]["payload"].transpose(0, 1).flatten(1, 2).cpu().numpy(), o.planes[t]["payload"][0])
            assert np.array_equal(c.planes[t]["scale"][..., 0].t().cpu().numpy(), o.planes[t]["scale"][0])


def _filled(layout, B, H, D, S, rng, paged=0, dtype="bf16", scale=1.0):
    cap = (S + 64) // 64 * 64
    o = OV.BlockCache(layout, B, H, D, cap)
    (k, kn), (v, vn) = (_rows(rng, (B, H, S, D), dtype, scale) for _ in range(2))
    o.store(kn, vn, [0] * B)
    if not paged:
        c = kvq.KVCache(layout, B, H, D, cap)
        kvq.store(c, k, v, 0)
        return c, o
    per = -(-cap // paged)
    c = kvq.PagedKVCache(layout, B, H, D, paged, B * per + 3, per)
    c.set_block_table(torch.from_numpy(rng.permutation(B * per + 3)[:B * per].reshape(B, per)))
    kvq.paged_store(c, k, v, torch.zeros(B, dtype=torch.int32, device="cuda"))
    return c, o


def _near(got, want_tol, what=""):
    want, tol = want_tol
    err = np.abs(got.cpu().numpy().astype(np.float64) - want)
    assert (err <= tol).all(), (what, float((err / np.maximum(tol, 1e-300)).max()), float(err.max()))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("gqa,n_q,S,causal", [(1, 1, 1, False), (8, 1, 65, False), (4, 1, 1000, False), (2, 5, 333, True), (3, 1, 64, False), (8, 3, 129, True), (1, 70, 200, True)])
def test_attend(layout, D, dtype, gqa, n_q, S, causal):
    rng = np.random.default_rng(7)
    B, H = 2, 2
    c, o = _filled(layout, B, H, D, S, rng)
    q, qn = _rows(rng, (B, H * gqa, n_q, D), dtype)
    for chunk in (0, 64):
        got = kvq.decode_attend(c, q, S, causal=causal, q_pos0=S - n_q if causal else 0, chunk=chunk)
        _near(got, o.attend(qn, 1 / np.sqrt(D), [S] * B, causal), chunk)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("page,n_q,dtype", [(64, 1, "bf16"), (128, 4, "f32"), (64, 40, "f16")])
def test_paged_attend(layout, D, page, n_q, dtype):
    """Ragged lengths: empty, one token, pages that end inside a stage, shorter than the causal rows."""
    rng = np.random.default_rng(8)
    B, H, S = 5, 2, 400
    c, o = _filled(layout, B, H, D, S, rng, page)
    q, qn = _rows(rng, (B, 3 * H, n_q, D), dtype)
    lens = [0, 1, 65, 191, 400]
    d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for causal in (False, True):
        for chunk in (0, 128):
            got = kvq.paged_decode_attend(c, q, d, S, causal=causal, chunk=chunk)
            want = [o.attend(qn, 1 / np.sqrt(D), [n if i == b else 0 for i in range(B)], causal) for b, n in enumerate(lens)]
            _near(got, (sum(w[0] for w in want), sum(w[1] for w in want)), (causal, chunk))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("scale", [1e-30, 1e-3, 1e20])
def test_attend_over_values_of_any_size(layout, scale):
    """The scales join in float32: values far from 1 lose nothing (attention scale set for keys of their size)."""
    rng = np.random.default_rng(9)
    c, o = _filled(layout, 1, 2, 128, 700, rng, dtype="f32", scale=scale)
    q, qn = _rows(rng, (1, 8, 1, 128), "f32")
    alpha = float(np.float32(1 / np.sqrt(128) / scale))
    _near(kvq.decode_attend(c, q, 700, attn_scale=alpha), o.attend(qn, alpha, [700]))


@pytest.mark.parametrize("layout", LAYOUTS)
def test_rows_behind_the_length_are_not_seen(layout):
    rng = np.random.default_rng(10)
    c, o = _filled(layout, 1, 2, 128, 300, rng)
    q, qn = _rows(rng, (1, 4, 1, 128))
    for t in ("k", "v"):
        c.planes[t]["payload"][:, :, 300:] = 0x7F             # e4m3: NaN
    for n in (1, 63, 64, 65, 299, 300):
        ref = o.attend(qn, 1 / np.sqrt(128), [n])
        got = kvq.decode_attend(c, q, n)
        assert torch.isfinite(got).all()
        _near(got, ref, n)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_one_call_steps_equal_their_parts(layout):
    """append_decode_attend, its paged and host-buffer forms and the static call give the bits of store and attend."""
    rng = np.random.default_rng(11)
    B, H, D, n0, new = 2, 2, 128, 250, 3
    lens = torch.full((B,), n0 + new, dtype=torch.int32, device="cuda")
    for paged in (0, 64):
        c, _ = _filled(layout, B, H, D, n0, np.random.default_rng(11), paged)
        d, _ = _filled(layout, B, H, D, n0, np.random.default_rng(11), paged)
        (k, _), (v, _) = (_rows(rng, (B, H, new, D), scale=30.0) for _ in range(2))
        q, _ = _rows(rng, (B, 4 * H, new, D))
        if paged:
            kvq.paged_store(c, k, v, lens - new)
            want = kvq.paged_decode_attend(c, q, lens, n0 + new, causal=True)
            got = kvq.paged_append_decode_attend(d, k, v, q, lens, n0 + new, causal=True)
            host = kvq.paged_append_decode_attend_host(d, k.cpu(), v.cpu(), q.cpu(), lens.cpu(), n0 + new, causal=True)
        else:
            kvq.store(c, k, v, n0)
            want = kvq.decode_attend(c, q, n0 + new, causal=True, q_pos0=n0)
            got = kvq.append_decode_attend(d, k, v, n0, q, n0 + new, causal=True, q_pos0=n0)
            assert torch.equal(want, api.decode_attend_static(c, q, n0 + new, causal=True, q_pos0=n0))
            host = kvq.append_decode_attend_host(d, k.cpu().pin_memory(), v.cpu().pin_memory(), n0, q.cpu().pin_memory(), n0 + new, causal=True, q_pos0=n0)
        assert torch.equal(got, want) and torch.equal(host.cuda(), want)
        for t in ("k", "v"):
            for name in ("payload", "scale"):
                assert torch.equal(c.planes[t][name], d.planes[t][name])


@pytest.mark.parametrize("layout", LAYOUTS)
def test_decode_loop_in_a_graph(layout):
    """A captured paged step (append, attend), replayed while the lengths on the device grow across blocks."""
    rng = np.random.default_rng(12)
    B, H, D, S = 3, 2, 128, 120
    c, o = _filled(layout, B, H, D, S, rng, 64)
    lens = torch.tensor([60, 63, 120], dtype=torch.int32, device="cuda")
    k, v, q = (torch.zeros((B, h, 1, D), dtype=torch.bfloat16, device="cuda") for h in (H, H, 4 * H))
    out = torch.zeros((B, 4 * H, 1, D), device="cuda")
    ws = torch.empty(max(256, kvq.paged_attend_workspace_bytes(c, 4 * H, 1, 128)), dtype=torch.uint8, device="cuda")
    call = lambda: kvq.paged_append_decode_attend(c, k, v, q, lens, 128, out=out, workspace=ws)     # noqa: E731
    keep = {t: {n: x.clone() for n, x in pl.items()} for t, pl in c.planes.items()}
    call()
    for t, pl in keep.items():
        for n, x in pl.items():
            c.planes[t][n].copy_(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for step in range(6):
        lens += 1
        new = [_rows(rng, x.shape, scale=3.0 ** step) for x in (k, v, q)]
        for x, (d, _) in zip((k, v, q), new):
            x.copy_(d)
        g.replay()
        n = lens.cpu().numpy()
        o.store(new[0][1], new[1][1], n - 1)
        _near(out, o.attend(new[2][1], 1 / np.sqrt(D), n), step)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_ragged_runs_of_one_block(layout):
    """Runs of one block in a call: tokens without a slot between them, a slot twice, a longer run behind a short one."""
    rng = np.random.default_rng(6)
    H, D, page, n_pages = 2, 256, 128, 8
    slots = np.array([5, 6, -1, 8, 9, 9, 8] + [-1] * 64 + list(range(20, 64)) + [64, -1, 70, 66] + [-1] * 30 + [300, 500] + [2 ** 40, 512, 512])
    want = [[5, 6], [8, 9], [9], [8], list(range(20, 64)), [64], [70], [66], [300], [500], [512], [512]]
    c, o = kvq.PagedKVCache(layout, 1, H, D, page, n_pages, 1), OV.BlockCache(layout, 1, H, D, page * n_pages)
    for scale in (1.0, 50.0, 0.1):
        (k, kn), (v, vn) = (_rows(rng, (len(slots), H, D), "f32", scale) for _ in range(2))
        k[4:] *= 3.0                                       # scales grow from run to run
        kn[4:] *= 3.0
        kvq.paged_store_slots(c, k, v, torch.from_numpy(slots).cuda())
        at = [i for i, s in enumerate(slots) if 0 <= s < page * n_pages]
        for run in want:
            i, at = at[:len(run)], at[len(run):]
            for x, t in ((kn, "k"), (vn, "v")):
                o.append(t, 0, x[i].transpose(1, 0, 2), run[0])
        for t in ("k", "v"):
            assert np.array_equal(c.planes[t]["scale"].transpose(0, 1).flatten(1, 2).cpu().numpy(), o.planes[t]["scale"][0])
            assert np.array_equal(c.planes[t]["payload"].transpose(0, 1).flatten(1, 2).cpu().numpy(), o.planes[t]["payload"][0])


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (128, "f32"), (128, "f16"), (256, "bf16")])
@pytest.mark.parametrize("gqa,n_q,S,causal", [(2, 130, 300, True), (8, 40, 130, True), (1, 33, 64, False), (16, 3, 500, False), (3, 129, 129, True), (1, 128, 1, False)])
def test_attend_many_rows(layout, D, dtype, gqa, n_q, S, causal):
    """Groups of rows of every kind: full, ended by the last row, rows that see one token, blocks that no row of a group sees."""
    rng = np.random.default_rng(13)
    B, H = 1, 2
    c, o = _filled(layout, B, H, D, S, rng)
    q, qn = _rows(rng, (B, H * gqa, n_q, D), dtype)
    want = o.attend(qn, 1 / np.sqrt(D), [S] * B, causal)
    for chunk in (0, 64, 192):
        _near(kvq.decode_attend(c, q, S, causal=causal, q_pos0=S - n_q if causal else 0, chunk=chunk), want, chunk)
    if causal and S > n_q:                                 # rows that are not the newest
        kv = S - 1
        got = kvq.decode_attend(c, q, S, causal=True, q_pos0=kv - n_q)
        _near(got, o.attend(qn, 1 / np.sqrt(D), [kv] * B, True))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_paged_attend_many_rows(layout, dtype):
    rng = np.random.default_rng(14)
    B, H, S, D, n_q = 4, 2, 330, 128, 70
    c, o = _filled(layout, B, H, D, S, rng, 64)
    q, qn = _rows(rng, (B, 2 * H, n_q, D), dtype)
    lens = [0, 20, 191, 330]
    d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for causal in (False, True):
        want = [o.attend(qn, 1 / np.sqrt(D), [n if i == b else 0 for i in range(B)], causal) for b, n in enumerate(lens)]
        for chunk in (0, 128):
            got = kvq.paged_decode_attend(c, q, d, S, causal=causal, chunk=chunk)
            _near(got, (sum(w[0] for w in want), sum(w[1] for w in want)), (causal, chunk))


@pytest.mark.parametrize("n_q", [1, 64])
@pytest.mark.parametrize("paged", [False, True])
def test_units_dealt_over_many_heads(n_q, paged):
    """More heads than CTAs, so that CTAs pass from one head to the next, and sequences of every length in between."""
    rng = np.random.default_rng(15)
    B, H, D, S = 70, 8, 128, 200
    c, o = _filled("int8_b64", B, H, D, S, rng, 64 if paged else 0)
    q, qn = _rows(rng, (B, 2 * H, n_q, D))
    lens = rng.integers(0, S + 1, B) if paged else np.full(B, S)
    lens[:3] = [S, 0, 1] if paged else S
    if paged:
        got = kvq.paged_decode_attend(c, q, torch.from_numpy(lens.astype(np.int32)).cuda(), S, causal=n_q > 1)
    else:
        got = kvq.decode_attend(c, q, S, causal=n_q > 1, q_pos0=S - n_q if n_q > 1 else 0)
    some = [0, 1, 2, 3, 34, 69]
    keep = np.zeros(B, int)
    keep[some] = lens[some]
    want, tol = o.attend(qn, 1 / np.sqrt(D), keep, n_q > 1)
    err = np.abs(got.cpu().numpy() - want)
    assert (err[some] <= tol[some]).all() and torch.isfinite(got).all()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("D,n_q", [(128, 1), (128, 70), (256, 1)])
def test_nothing_to_attend_to(layout, D, n_q):
    """All sequences empty: zeros, whatever the output held, for dealt out and for planned chunks."""
    rng = np.random.default_rng(21)
    c, _ = _filled(layout, 3, 2, D, 100, rng, 64)
    q, _ = _rows(rng, (3, 4, n_q, D))
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    for chunk in (0, kvq.paged_attend_plan_chunk(c, 4, n_q, [0, 0, 0])):
        out = torch.full((3, 4, n_q, D), float("nan"), device="cuda")
        kvq.paged_decode_attend(c, q, lens, 100, chunk=chunk, out=out)
        assert (out == 0).all()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n_q", [1, 70])
def test_planned_chunk(layout, n_q):
    rng = np.random.default_rng(22)
    c, o = _filled(layout, 3, 2, 128, 700, rng, 64)
    q, qn = _rows(rng, (3, 4, n_q, 128))
    lens = [700, 3, 129]
    chunk = kvq.paged_attend_plan_chunk(c, 4, n_q, lens)
    got = kvq.paged_decode_attend(c, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), 700, chunk=chunk)
    want = [o.attend(qn, 1 / np.sqrt(128), [n if i == b else 0 for i in range(3)]) for b, n in enumerate(lens)]
    _near(got, (sum(w[0] for w in want), sum(w[1] for w in want)), chunk)
