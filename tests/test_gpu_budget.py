"""Attention with running weights, selection and compaction against the oracle, and the three together as a
decode loop uses them."""
import numpy as np
import pytest
import torch

import sub_byte_quantized_gb300 as kvq
from oracle import attention as OA, budget as OB, paged as OP, rope as OR
from synth import WORKLOADS, make_inputs
from tests.gpu_helpers import check_close, planes_equal

pytestmark = pytest.mark.gpu
LAYOUTS = ["q4_0", "q6_0", "q8_0", "asym4_g32", "had_int4", "had_int2", "q4_0+q8_0", "had_int2+had_int4"]


def _inputs(seed, B, Hq, H, S, nq, D, dtype="bf16"):
    rng = np.random.default_rng(seed)
    k, v = (rng.standard_normal((B, H, S, D)).astype(np.float32) for _ in range(2))
    k[..., rng.permutation(D)[:4]] *= 6.0
    q = rng.standard_normal((B, Hq, nq, D)).astype(np.float32)
    dt = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[dtype]
    qd = torch.from_numpy(q).to(dt)
    return k, v, qd.float().numpy(), qd.cuda()


def _caches(layout, k, v, cap, n_recent=0):
    B, H, S, D = k.shape
    dc, oc = kvq.KVCache(layout, B, H, D, cap, n_recent=n_recent), OA.OracleCache(layout, B, H, D, cap, n_recent=n_recent)
    kvq.store(dc, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), 0)
    oc.store(k, v, 0)
    return dc, oc


def _close(got, want, err, old=None, decay=0.0):
    """|got - want| within the weights' relative error, plus the two roundings of the update and what the
    flush of subnormal exponentials may drop."""
    total = want if old is None else want + decay * old.astype(np.float64)
    tol = err * want + 2.0 ** -23 * (want + (0 if old is None else np.abs(decay * old))) + 1e-35
    bad = np.abs(got - total) > tol
    assert not bad.any(), (bad.sum(), np.abs(got - total).max(), (np.abs(got - total) / tol).max())


def _check(layout, D, B, Hq, H, S, nq, causal=False, dtype="bf16", n_recent=0, decay=0.5, chunk=0, seed=0, q_pos0=None):
    k, v, q, qd = _inputs(seed, B, Hq, H, S, nq, D, dtype)
    dc, oc = _caches(layout, k, v, S + 3, n_recent)
    alpha = 1 / np.sqrt(D)
    q0 = (S - nq if q_pos0 is None else q_pos0) if causal else 0
    want, err = OB.weights(oc, q, np.float32(alpha), S, causal, q0)
    old = np.abs(np.random.default_rng(seed + 1).standard_normal((B, H, S + 2))).astype(np.float32)
    sc = torch.from_numpy(old).cuda()
    so = torch.full_like(sc, float("nan"))
    out, got = kvq.decode_attend_weights(dc, qd, S, sc, scores_out=so, decay=decay, causal=causal, q_pos0=q0, attn_scale=float(np.float32(alpha)),
                                         chunk=chunk)
    assert got is so
    g = got.cpu().numpy()
    assert np.isnan(g[..., S:]).all() and torch.equal(sc.cpu(), torch.from_numpy(old))
    _close(g[..., :S], want, err, old[..., :S], np.float32(decay))
    ref = oc.attend(q, np.float32(alpha), S, causal, q0)
    check_close(out.cpu().numpy(), ref[0] if isinstance(ref, tuple) else ref)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f32", "f16"])
def test_weights_layouts(layout, D, dtype):
    w = 24 if "had" in layout else 0
    _check(layout, D, 2, 4, 2, 333, 1, dtype=dtype, n_recent=w)
    _check(layout, D, 1, 6, 2, 205, 5, causal=True, dtype=dtype, n_recent=w)


@pytest.mark.parametrize("S", [1, 2, 15, 16, 17, 31, 33, 64, 127, 513, 700])
def test_weights_lengths(S):
    _check("q4_0", 128, 1, 4, 2, S, 1)
    _check("had_int4", 128, 1, 4, 2, S, 1, n_recent=32)                        # window longer than, equal to, shorter than the cache
    _check("asym4_g32", 128, 1, 2, 1, S, min(S, 3), causal=True)


@pytest.mark.parametrize("Hq,nq", [(1, 1), (7, 1), (8, 1), (9, 1), (16, 4), (13, 5), (4, 17), (1, 129)])
@pytest.mark.parametrize("layout", ["q8_0", "had_int4", "q6_0"])
def test_weights_row_counts(layout, Hq, nq):
    """One pass over the rows, a full one, one row more, several."""
    _check(layout, 128, 1, Hq, 1, 300, nq, causal=nq > 1, n_recent=40 if "had" in layout else 0)


def test_weights_many_rows_without_mask_and_from_the_start():
    _check("q4_0", 128, 1, 8, 2, 600, 40, causal=False)
    _check("had_int2", 128, 1, 8, 2, 600, 40, causal=True, q_pos0=0, n_recent=70)   # most tokens are seen by no row
    _check("q4_0", 256, 1, 4, 2, 500, 40, causal=True, q_pos0=3)


def test_weights_chunks():
    for chunk in (64, 192, 4096):
        _check("q8_0", 128, 2, 4, 2, 901, 1, chunk=chunk)


def test_weights_in_place_none_and_nan_behind_decay_zero():
    k, v, q, qd = _inputs(3, 1, 4, 2, 150, 1, 128)
    dc, _ = _caches("q4_0", k, v, 160)
    _, a = kvq.decode_attend_weights(dc, qd, 150, None, scores_out=torch.zeros((1, 2, 160), device="cuda"))
    _, b = kvq.decode_attend_weights(dc, qd, 150, torch.full((1, 2, 160), float("nan"), device="cuda"), decay=0.0)
    assert torch.equal(a[..., :150], b[..., :150])                              # earlier scores are not read
    c = a.clone()
    _, d = kvq.decode_attend_weights(dc, qd, 150, c, decay=1.0)
    assert d.data_ptr() == c.data_ptr() and torch.equal(c[..., :150], a[..., :150] + a[..., :150])
    _, e = kvq.decode_attend_weights(dc, qd, 150, a, scores_out=torch.zeros_like(a))
    assert torch.equal(e, c)                                                    # equal calls, equal bits
    with pytest.raises(ValueError):
        kvq.decode_attend_weights(dc, qd, 150, None)
    with pytest.raises(ValueError):
        kvq.decode_attend_weights(dc, qd, 150, a, scores_out=torch.zeros((1, 2, 150), device="cuda"))


@pytest.mark.parametrize("layout,D,n_recent", [("q4_0", 128, 0), ("q6_0", 256, 0), ("had_int4", 128, 40), ("q4_0+q8_0", 128, 0)])
@pytest.mark.parametrize("nq", [1, 20])
def test_paged_weights(layout, D, n_recent, nq):
    lens = [300, 0, 1, 65, 640, 12]                                             # an empty one, rows before the start (causal, nq 20)
    B, Hq, H, page, per = len(lens), 6, 2, 64, 10
    k, v, q, qd = _inputs(7, B, Hq, H, max(lens), nq, D)
    dc = kvq.PagedKVCache(layout, B, H, D, page, B * per, per, n_recent=n_recent)
    tab = np.random.default_rng(1).permutation(B * per).reshape(B, per)
    dc.set_block_table(tab)
    oc = OP.OraclePagedCache(layout, B, H, D, page, B * per, per, n_recent, tab)
    # every sequence stored up to its own length (the window holds its newest tokens)
    for b, n in enumerate(lens):
        at = np.full(B, -10 ** 6, np.int32)
        at[b] = 0
        if n:
            kvq.paged_store(dc, torch.from_numpy(k[:, :, :n].copy()).cuda(), torch.from_numpy(v[:, :, :n].copy()).cuda(),
                            torch.from_numpy(at).cuda())
            oc.store(k[:, :, :n], v[:, :, :n], at)
    alpha = np.float32(1 / np.sqrt(D))
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    old = np.abs(np.random.default_rng(8).standard_normal((B, H, 700))).astype(np.float32)
    so = torch.full((B, H, 700), -7.0, device="cuda")
    out, got = kvq.paged_decode_attend_weights(dc, qd, sl, 640, torch.from_numpy(old).cuda(), scores_out=so, decay=0.9, causal=nq > 1,
                                               attn_scale=float(alpha))
    g = got.cpu().numpy()
    check_close(out.cpu().numpy(), oc.attend(q, alpha, lens, nq > 1))
    for b, n in enumerate(lens):
        assert (g[b, :, n:] == -7.0).all()
        if n:
            want, err = OB.weights(oc.sequence(b, n), q[b:b + 1], alpha, n, nq > 1, n - nq)
            _close(g[b:b + 1, :, :n], want, err, old[b:b + 1, :, :n], np.float32(0.9))


# ------------------------------------------------------------------ selection
def _select(scores, n, n_keep, sink=0, recent=0, lens=None):
    B, H, _ = scores.shape
    keep = torch.full((B, H, n_keep), -9, dtype=torch.int32, device="cuda")
    new = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    sl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    kvq.evict_select(torch.from_numpy(scores).cuda(), n, n_keep, sink, recent, seq_lens=sl, keep=keep, new_lens=new)
    real = [n] * B if lens is None else [min(max(x, 0), n) for x in lens]
    assert np.array_equal(keep.cpu().numpy(), OB.select(scores, real, n_keep, sink, recent))
    assert new.tolist() == [min(x, n_keep) for x in real]


@pytest.mark.parametrize("n,n_keep,sink,recent", [(1, 1, 0, 0), (2, 1, 0, 0), (33, 5, 1, 2), (64, 63, 0, 63), (64, 64, 1, 1), (65, 100, 4, 4),
                                                  (1000, 1, 0, 0), (1000, 999, 3, 7), (1000, 10, 5, 5), (8192, 4000, 4, 64),
                                                  (8193, 31, 0, 0), (20011, 9000, 4, 256), (70001, 69000, 0, 1)])
def test_select_sizes(n, n_keep, sink, recent):
    rng = np.random.default_rng(n + n_keep)
    _select(np.exp(3 * rng.standard_normal((2, 3, n))).astype(np.float32), n, n_keep, sink, recent)
    _select(rng.standard_normal((1, 1, n + 7)).astype(np.float32), n, n_keep, sink, recent)      # rows longer than the cache, signs


@pytest.mark.parametrize("values", [[0.0], [0.0, -0.0], [1.0, 2.0], [np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, 3e38],
                                    [1.0, 1.0 + 2 ** -23, 1.0 + 2 ** -22], [np.nan], [-np.inf, np.nan]])
def test_select_ties_and_specials(values):
    rng = np.random.default_rng(5)
    x = rng.choice(np.array(values, np.float32), (1, 2, 9000))
    for n, keep in ((9000, 4500), (9000, 1), (100, 37), (9000, 8999)):
        _select(x, n, keep, min(2, keep - 1), 0)


def test_select_ragged_lengths():
    rng = np.random.default_rng(6)
    lens = [500, 499, 0, 1, 4000, -3, 9999, 501]                                # clamped into [0, 4000]
    _select(rng.standard_normal((8, 2, 4100)).astype(np.float32), 4000, 500, 4, 60, lens)


def test_select_longer_than_shared_memory():
    rng = np.random.default_rng(7)
    _select(rng.standard_normal((1, 1, 450001)).astype(np.float32), 450001, 100003, 4, 1000)


# ------------------------------------------------------------------ compaction
def _keep(rng, B, H, n, n_keep, recent):
    s = rng.standard_normal((B, H, n)).astype(np.float32)
    return s, OB.select(s, [n] * B, n_keep, min(4, n_keep - recent), recent)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("in_place", [True, False])
def test_compact_layouts(layout, D, in_place):
    R = 48 if "had" in layout else 0
    for n, n_keep in ((700, 333), (130, 129), (100, 60), (100, 120)):
        rng = np.random.default_rng(n)
        k, v = (rng.standard_normal((2, 3, n, D)).astype(np.float32) for _ in range(2))
        dc, oc = _caches(layout, k, v, n + 5, R)
        scores, keep = _keep(rng, 2, 3, n, n_keep, max(R, 8))
        old = rng.random((2, 3, n + 2)).astype(np.float32)
        sc = torch.from_numpy(old).cuda()
        m = min(n, n_keep)
        OB.compact(oc.planes, keep, [n, n], R)
        kd = torch.from_numpy(keep).cuda()
        if in_place:
            assert kvq.evict_compact(dc, kd, n, scores=sc) == m
            planes_equal(dc, oc)
            got = sc.cpu().numpy()
            assert np.array_equal(got[..., n:], old[..., n:])
        else:
            dst = kvq.KVCache(layout, 2, 3, D, m, n_recent=R)
            before = {t: {x: y.clone() for x, y in p.items()} for t, p in dc.planes.items()}
            so = torch.full((2, 3, m + 9), -5.0, device="cuda")
            assert kvq.evict_compact(dc, kd, n, dst=dst, scores=sc, scores_out=so) == m
            planes_equal(dst, oc, m)
            for t in ("k", "v"):
                assert all(torch.equal(before[t][x], y) for x, y in dc.planes[t].items())
            got = so.cpu().numpy()
            assert np.array_equal(sc.cpu().numpy(), old) and (got[..., n:] == -5.0).all()
        want = np.take_along_axis(old[..., :n], np.maximum(keep[..., :m], 0).astype(np.int64), 2)
        assert np.array_equal(got[..., :m], want) and (got[..., m:min(n, got.shape[2])] == 0).all()


def test_compact_long_in_place_with_few_heads():
    """Several rounds of a whole cluster: shifts that grow along the cache, and a kept prefix."""
    n, n_keep = 40000, 23000
    rng = np.random.default_rng(11)
    dc = kvq.KVCache("q4_0", 1, 2, 128, n)
    for t in ("k", "v"):
        dc.planes[t]["payload"].copy_(torch.randint(0, 256, dc.planes[t]["payload"].shape, dtype=torch.uint8))
        dc.planes[t]["scale"].copy_(torch.rand(dc.planes[t]["scale"].shape))
    lists = [np.sort(rng.choice(n, n_keep, replace=False)), np.r_[0:20000, n - 3000:n]]
    keep = torch.from_numpy(np.stack(lists)[None].astype(np.int32)).cuda()
    want = {t: {x: torch.stack([y[0, h, torch.from_numpy(lists[h]).cuda()] for h in range(2)])[None] for x, y in p.items()}
            for t, p in dc.planes.items()}
    kvq.evict_compact(dc, keep, n)
    for t in ("k", "v"):
        assert all(torch.equal(dc.planes[t][x][:, :, :n_keep], y) for x, y in want[t].items())


def test_compact_entries_out_of_range_move_nothing():
    rng = np.random.default_rng(12)
    k, v = (rng.standard_normal((1, 1, 50, 128)).astype(np.float32) for _ in range(2))
    dc, oc = _caches("q8_0", k, v, 50)
    keep = np.array([[[0, 3, -1, 50, 2 ** 31 - 1, 20, -2 ** 31]]], np.int32)
    OB.compact(oc.planes, keep, [50], 0)
    kvq.evict_compact(dc, torch.from_numpy(keep).cuda(), 50)
    planes_equal(dc, oc)


@pytest.mark.parametrize("layout,D,n_recent", [("q4_0", 128, 0), ("q6_0", 128, 0), ("asym4_g32", 256, 0), ("had_int2", 128, 100), ("had_int4", 256, 7)])
def test_paged_compact(layout, D, n_recent):
    lens, n_keep = [640, 0, 200, 199, 577, 1], 200
    B, H, page, per = len(lens), 2, 64, 10
    rng = np.random.default_rng(13)
    dc = kvq.PagedKVCache(layout, B, H, D, page, B * per + 3, per, n_recent=n_recent)
    tab = rng.permutation(B * per + 3)[:B * per].reshape(B, per)
    dc.set_block_table(tab)
    oc = OP.OraclePagedCache(layout, B, H, D, page, B * per + 3, per, n_recent, tab)
    for t in ("k", "v"):
        for name, x in oc.planes[t].items():
            y = rng.integers(0, 256, x.shape).astype(np.uint8) if x.dtype == np.uint8 else rng.random(x.shape).astype(x.dtype)
            oc.planes[t][name] = y
            dc.planes[t]["recent" if name == "ring" else name].copy_(torch.from_numpy(y))
    s = rng.standard_normal((B, H, 650)).astype(np.float32)
    keep = OB.select(s, lens, n_keep, 4, max(n_recent, 16))
    OB.compact(oc.planes, keep, lens, n_recent, oc.locate)
    sc = torch.from_numpy(s).cuda()
    kvq.paged_evict_compact(dc, torch.from_numpy(keep).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), 640, scores=sc)
    for t in ("k", "v"):
        for name, x in oc.planes[t].items():
            assert np.array_equal(dc.planes[t]["recent" if name == "ring" else name].cpu().numpy(), x), (t, name)
    got = sc.cpu().numpy()
    for b, n in enumerate(lens):
        m = min(n, n_keep)
        want = np.take_along_axis(s[b], np.maximum(keep[b, :, :m], 0).astype(np.int64), 1)
        assert np.array_equal(got[b, :, :m], want) and (got[b, :, m:640] == 0).all() and np.array_equal(got[b, :, 640:], s[b, :, 640:])


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("layout,n_recent", [("q4_0", 0), ("had_int4", 16)])
def test_decode_loop_inside_a_budget(layout, n_recent):
    """Rotary append, attention with weights, and a cut back to the budget every eighth step, against the same
    loop of the oracle: every plane bit for bit, and at each cut the same lists from the library's scores."""
    B, Hq, H, D, budget = 2, 4, 2, 128, 40
    dc, oc = kvq.KVCache(layout, B, H, D, 64, n_recent=n_recent), OA.OracleCache(layout, B, H, D, 64, n_recent=n_recent)
    f, _ = kvq.rope_frequencies(D)
    table = kvq.rope_table(f, 256)
    t32 = table.cpu().numpy()
    scores = torch.zeros((B, H, 64), device="cuda")
    rng = np.random.default_rng(21)
    alpha = np.float32(1 / np.sqrt(D))
    n, at = 0, 0
    for step, n_new in enumerate([30] + [1] * 40):
        q, k, v = (rng.standard_normal((B, h, n_new, D)).astype(np.float32) for h in (Hq, H, H))
        pos = np.broadcast_to(np.arange(at, at + n_new), (B, n_new))
        qd = kvq.rope_store(dc, table, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), n, q=torch.from_numpy(q).cuda(),
                            positions=torch.from_numpy(np.array(pos, dtype=np.int32, order="C")).cuda())
        rows = t32[pos][:, None]
        oc.store(OR.rotate(k, rows), v, n)
        q = OR.rotate(q, rows)
        n, at = n + n_new, at + n_new
        old = scores.cpu().numpy()
        out, _ = kvq.decode_attend_weights(dc, qd, n, scores, decay=0.95, causal=n_new > 1, q_pos0=n - n_new if n_new > 1 else 0,
                                           attn_scale=float(alpha))
        ref = oc.attend(q, alpha, n, n_new > 1, n - n_new)
        check_close(out.cpu().numpy(), ref[0] if isinstance(ref, tuple) else ref)
        want, err = OB.weights(oc, q, alpha, n, n_new > 1, n - n_new)
        _close(scores.cpu().numpy()[..., :n], want, err, old[..., :n], np.float32(0.95))
        if n > budget and step % 8 == 0:
            now = scores.cpu().numpy()
            keep = kvq.evict_select(scores, n, budget, n_sink=2, n_recent=max(8, n_recent))
            lists = OB.select(now, [n] * B, budget, 2, max(8, n_recent))
            assert np.array_equal(keep.cpu().numpy(), lists)
            OB.compact(oc.planes, lists, [n] * B, n_recent)
            n = kvq.evict_compact(dc, keep, n, scores=scores)
            planes_equal(dc, oc, n)
            assert (scores.cpu().numpy()[..., n:] == 0).all()
    assert at == 70 and n <= budget + 8


def test_captured_step_replays():
    """The paged step (append, weights, selection, compaction) in a graph: replays equal eager calls, and two
    graphs with workspaces of their own do not disturb each other."""
    B, Hq, H, D, page, per = 2, 4, 2, 128, 64, 4
    rng = np.random.default_rng(22)
    f, _ = kvq.rope_frequencies(64)
    table = kvq.rope_table(f, 300)

    def make():
        dc = kvq.PagedKVCache("q8_0", B, H, D, page, B * per, per)
        dc.set_block_table(np.arange(B * per).reshape(B, per))
        return dc
    x = torch.from_numpy(rng.standard_normal((B, 200, (Hq + 2 * H) * D)).astype(np.float32)).cuda()
    lens = torch.tensor([200, 131], dtype=torch.int32, device="cuda")

    def heads(t):
        t = t.view(B, -1, Hq + 2 * H, D).transpose(1, 2)
        return t[:, :Hq], t[:, Hq:Hq + H], t[:, Hq + H:]

    def fill(dc):
        _, k, v = heads(x)
        kvq.paged_rope_store(dc, table, k, v, torch.zeros(B, dtype=torch.int32, device="cuda"))
        return torch.rand((B, H, 256), generator=torch.Generator("cuda").manual_seed(1), device="cuda")

    def step(dc, tok, scores, ws):
        q, k, v = heads(tok)
        q = kvq.paged_rope_store(dc, table, k, v, lens - 1, q=q)
        out, _ = kvq.paged_decode_attend_weights(dc, q, lens, 200, scores, workspace=ws)
        keep = kvq.evict_select(scores, 200, 100, 4, 10, seq_lens=lens)
        kvq.paged_evict_compact(dc, keep, lens, 200, scores=scores)
        return out, keep

    need = kvq.paged_attend_weights_workspace_bytes(make(), Hq, 1, 200)
    tok = torch.from_numpy(rng.standard_normal((B, 1, (Hq + 2 * H) * D)).astype(np.float32)).cuda()
    eager = make()
    es = fill(eager)
    eout, ekeep = step(eager, tok, es, torch.empty(need, dtype=torch.uint8, device="cuda"))
    graphs = []
    for _ in range(2):
        dc = make()
        sc, ws = fill(dc), torch.empty(need, dtype=torch.uint8, device="cuda")
        warm = make()
        step(warm, tok, fill(warm), ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out, keep = step(dc, tok, sc, ws)
        graphs.append((g, dc, sc, out, keep))
    for g, *_ in graphs:
        g.replay()
    torch.cuda.synchronize()
    for _, dc, sc, out, keep in graphs:
        assert torch.equal(out, eout) and torch.equal(keep, ekeep) and torch.equal(sc, es)
        for t in ("k", "v"):
            assert all(torch.equal(dc.planes[t][n], eager.planes[t][n]) for n in dc.planes[t])


def test_two_streams_at_once():
    """The same call from two streams, each with its own buffers."""
    k, v, q, qd = _inputs(31, 1, 8, 2, 3000, 1, 128)
    dc, _ = _caches("q4_0", k, v, 3000)
    _, want = kvq.decode_attend_weights(dc, qd, 3000, None, scores_out=torch.zeros((1, 2, 3000), device="cuda"))
    lists = kvq.evict_select(want, 3000, 1000)
    torch.cuda.synchronize()
    got = []
    for _ in range(2):
        s = torch.cuda.Stream()
        so = torch.zeros((1, 2, 3000), device="cuda")
        ws = torch.empty(kvq.attend_weights_workspace_bytes(dc, 8, 1, 3000), dtype=torch.uint8, device="cuda")
        out, keep = torch.empty((1, 8, 1, 128), device="cuda"), torch.empty((1, 2, 1000), dtype=torch.int32, device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        got.append((s, so, ws, out, keep))
    for s, so, ws, out, keep in got:
        for _ in range(3):
            kvq.decode_attend_weights(dc, qd, 3000, None, scores_out=so, out=out, workspace=ws, stream=s)
            kvq.evict_select(so, 3000, 1000, keep=keep, stream=s)
    torch.cuda.synchronize()
    for _, so, _, _, keep in got:
        assert torch.equal(so, want) and torch.equal(keep, lists)
