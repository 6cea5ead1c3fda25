"""The cache-budget operators at sizes where their kernels change form: groups of query rows, tiles beyond one
CTA's share, more heads than SMs, planes beyond 4 GB."""
import numpy as np
import pytest
import torch

import sub_byte_quantized_gb300 as kvq
from oracle import attention as OA, budget as OB, rope as OR
from tests.test_gpu_budget import LAYOUTS, _check, test_paged_weights as paged_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype,Hq,nq", [("bf16", 2, 150), ("f32", 2, 70), ("f16", 4, 33)])
def test_weights_row_groups(layout, dtype, Hq, nq):
    """300 rows of 16-bit queries, 140 of f32: a second group over the same tokens; 132 rows: two accumulators."""
    w = 50 if "had" in layout else 0
    _check(layout, 128, 1, Hq, 1, 290, nq, causal=True, dtype=dtype, n_recent=w)
    _check(layout, 128, 1, Hq, 1, 131, nq, dtype=dtype, n_recent=w)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights_row_passes_of_wide_heads(layout, dtype):
    w = 33 if "had" in layout else 0
    _check(layout, 256, 1, 8, 2, 300, 20, causal=True, dtype=dtype, n_recent=w)   # 80 rows
    _check(layout, 256, 1, 2, 1, 100, 32, dtype=dtype, n_recent=w)                # 64: one pass


def test_weights_more_heads_than_sms():
    """Tiles (or units) of a head in as few CTAs as hold them."""
    _check("q4_0", 128, 20, 24, 8, 2200, 3, causal=True)                          # 18 tiles: 16 and 2
    _check("had_int4", 128, 20, 24, 8, 300, 3, causal=True, n_recent=40)
    _check("q6_0", 256, 20, 40, 20, 500, 35, causal=True)                         # 70 rows, 16 units
    _check("asym4_g32", 256, 20, 40, 20, 300, 2)


@pytest.mark.parametrize("layout", ["q4_0", "q8_0", "had_int4"])
@pytest.mark.parametrize("D", [128, 256])
def test_weights_shortest(layout, D):
    """One token under many rows, a window that holds every token, one that leaves one."""
    for S, nq, w in ((1, 20, 0), (1, 1, 0), (5, 12, 8), (9, 3, 8)):
        _check(layout, D, 1, 2, 1, S, nq, n_recent=w if "had" in layout else 0)
        if nq <= S:
            _check(layout, D, 1, 2, 1, S, nq, causal=True, q_pos0=0, n_recent=w if "had" in layout else 0)


def test_planes_beyond_four_gigabytes():
    """Rows of 128 bytes behind byte 2^32 of a plane: appended, weighed, selected and moved."""
    H, D, far = 4, 128, 1 << 23
    n = far + 5
    dc = kvq.KVCache("q8_0", 1, H, D, n)
    for p in dc.planes.values():
        for t in p.values():
            t.zero_()
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn((1, H, 5, D), generator=g) for _ in range(2))
    f, _ = kvq.rope_frequencies(D)
    table = kvq.rope_table(f, 5, pos0=far)
    pos = torch.arange(5, dtype=torch.int32, device="cuda")[None]
    kvq.rope_store(dc, table, k.cuda(), v.cuda(), far, positions=pos)
    small = kvq.KVCache("q8_0", 1, H, D, 5)
    kvq.store(small, torch.from_numpy(OR.rotate(k.numpy(), table.cpu().numpy()[None, None])).cuda(), v.cuda(), 0)
    for t in ("k", "v"):
        for name, x in small.planes[t].items():
            assert torch.equal(dc.planes[t][name][:, :, far:], x)
    # weights: the zero rows all score 0, the last five their own dot products; the sums of 2^23 exponentials
    # are float32 with at most 2^13 additions in a row
    q = torch.randn((1, H, 9, D), generator=g)
    kd = small.planes["k"]["payload"].cpu().numpy().view(np.int8).reshape(H, 5, D // 32, 32).astype(np.float64)
    kd = (kd * small.planes["k"]["scale"].cpu().numpy().astype(np.float64)[0][..., None]).reshape(H, 5, D)
    for nq in (1, 9):
        qq = q[:, :, :nq].contiguous()
        alpha = 1.0                                              # (far above 1 / sqrt(D): the five stand out)
        s = np.einsum("hrd,htd->hrt", qq[0].numpy().astype(np.float64), kd) * alpha
        total = far + np.exp(s).sum(-1)
        scores = torch.zeros((1, H, n), device="cuda")
        kvq.decode_attend_weights(dc, qq.cuda(), n, None, scores_out=scores, attn_scale=alpha)
        want = (np.exp(s) / total[..., None]).sum(1)
        got = scores[0, :, far:].cpu().numpy()
        assert (np.abs(got - want) <= 2.0 ** -10 * want).all()
        rest = (1 / total).sum(1)
        lo, hi = scores[0, :, :far].min(1).values.cpu().numpy(), scores[0, :, :far].max(1).values.cpu().numpy()
        assert (np.abs(lo - rest) <= 2.0 ** -10 * rest).all() and (np.abs(hi - rest) <= 2.0 ** -10 * rest).all()
    scores[0, :, ::1 << 20] = 2.0                                # eight far apart
    keep = kvq.evict_select(scores, n, 13, n_recent=5)
    want = torch.cat([torch.arange(0, far, 1 << 20), torch.arange(far, n)]).int().cuda()
    assert torch.equal(keep, want.expand(1, H, 13))
    dst = kvq.KVCache("q8_0", 1, H, D, 13)
    so = torch.empty((1, H, 13), device="cuda")
    last = scores[:, :, far:].clone()
    kvq.evict_compact(dc, keep, n, dst=dst, scores=scores, scores_out=so)
    kvq.evict_compact(dc, keep, n, scores=scores)
    for c in (dc, dst):
        for t in ("k", "v"):
            for name, x in small.planes[t].items():
                assert torch.equal(c.planes[t][name][:, :, 8:13], x) and not c.planes[t][name][:, :, :8].any()
    assert torch.equal(so[:, :, 8:], last) and torch.equal(scores[:, :, :13], so) and not scores[:, :, 13:].any()


@pytest.mark.parametrize("layout", ["q4_0", "q8_0", "q4_0+q8_0", "had_int4", "had_int2", "asym4_g32", "q6_0"])
@pytest.mark.parametrize("first", [0, 100, 470, 511])
def test_weights_with_values_of_any_size(layout, first):
    """Values of up to 4e4 from one token on (their scales reach far beyond 2), small ones before it: the output
    stays within float32's reach of the sum of |weight * value|."""
    S, D = 512, 128
    rng = np.random.default_rng(first)
    k, v = (rng.standard_normal((1, 2, S, D)).astype(np.float32) for _ in range(2))
    v[:, :, :first] *= 1e-3
    v[:, :, first:] *= 1e4
    q = rng.standard_normal((1, 4, 1, D)).astype(np.float32)
    dc, oc = kvq.KVCache(layout, 1, 2, D, S), OA.OracleCache(layout, 1, 2, D, S)
    kvq.store(dc, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), 0)
    oc.store(k, v, 0)
    alpha = np.float32(0.3)
    out, _ = kvq.decode_attend_weights(dc, torch.from_numpy(q).cuda(), S, None, scores_out=torch.zeros((1, 2, S), device="cuda"),
                                       attn_scale=float(alpha))
    ref = oc.attend(q, alpha, S)
    ref = ref[0] if isinstance(ref, tuple) else ref
    s, _ = OB.scores_dense(oc, q, alpha, S)
    p = np.exp(s - s.max(-1, keepdims=True))
    l = p.sum(-1, keepdims=True)
    av = np.abs(oc.dequantized("v", S))[:, [0, 0, 1, 1]]
    mass = np.einsum("bhqt,bhtd->bhqd", p / l, av)
    # Beside a scale of 2 or more the probabilities p <= 1 and P' = p * scale are held as two f16 parts without the
    # factor 2^12: the lo parts are multiples of 2^-24, off by at most 2^-25 each. Per token that is 2^-25 |v| from
    # p's and 2^-25 |code| from P', over l.
    code = 128 if "q8" in layout else 32 if layout == "q6_0" else 15
    low = 2.0 ** -25 * (av.sum(2, keepdims=True) + S * code) / l
    if "had" in layout:                                         # the rotation back adds up every dim
        mass, low = (np.broadcast_to(x.sum(-1, keepdims=True) / np.sqrt(D), x.shape) for x in (mass, low))
    # probabilities: the scores' float32 (|s| < 64: 2^-18); products and sums: 2^-20 of the mass
    assert (np.abs(out.cpu().numpy() - ref) <= 2.0 ** -17 * mass + low).all()


@pytest.mark.parametrize("layout", ["had_int4", "had_int2"])
@pytest.mark.parametrize("Hq,nq", [(5, 13), (4, 24), (4, 32), (3, 43)])
def test_weights_of_an_observation_window(layout, Hq, nq):
    """65 to 129 rows per kv head over a Hadamard body of one stage of 64 tokens, of two, three and many, with rows
    that see a part of the last ones only."""
    for S, w, causal in ((50, 0, True), (64 + 40, 40, True), (129, 0, False), (161, 30, True), (1000, 64, True), (2600, 0, True)):
        if nq <= S:
            _check(layout, 128, 2, 2 * Hq, 2, S, nq, causal=causal, n_recent=w)
    _check(layout, 128, 1, Hq, 1, 700, nq, causal=True, q_pos0=0, n_recent=20, chunk=192)
    _check(layout, 128, 1, Hq, 1, 700, nq, causal=True, q_pos0=100, chunk=64)


@pytest.mark.parametrize("layout,n_recent", [("had_int4", 40), ("had_int4", 0), ("had_int2", 130), ("q8_0", 0)])
@pytest.mark.parametrize("nq", [30, 42, 100])
def test_paged_weights_of_an_observation_window(layout, n_recent, nq):
    """90, 126 and 300 rows over sequences of their own lengths: an empty one, some shorter than the rows' reach."""
    paged_weights(layout, 128, n_recent, nq)


@pytest.mark.parametrize("layout,D", [("q6_0", 128), ("q8_0", 256), ("asym4_g32", 128), ("had_int2", 256)])
@pytest.mark.parametrize("H,n,n_keep", [(1, 7000, 5000), (2, 2500, 2400), (8, 900, 431)])
def test_compact_in_place_again_and_again(layout, D, H, n, n_keep):
    """Rows are read before another CTA of the cluster writes over them, every time: shifts of a few rows to
    thousands, 40 random lists."""
    g = torch.Generator("cuda").manual_seed(n)
    dc = kvq.KVCache(layout, 2, H, D, n)
    for p in dc.planes.values():
        p["payload"].copy_(torch.randint(0, 256, p["payload"].shape, dtype=torch.uint8, device="cuda", generator=g))
        for name in ("scale", "zero"):
            if name in p:
                p[name].copy_(torch.rand(p[name].shape, device="cuda", generator=g))
    first = {t: {name: x.clone() for name, x in p.items()} for t, p in dc.planes.items()}
    scores = torch.rand((2, H, n), device="cuda", generator=g)
    for i in range(40):
        keep = torch.rand((2, H, n), device="cuda", generator=g)
        keep[..., : n // 2] *= (i % 4) / 3                       # few early cuts, or many
        keep = keep.topk(n_keep, -1).indices.sort(-1).values
        for t, p in dc.planes.items():
            for name, x in p.items():
                x.copy_(first[t][name])
        sc = scores.clone()
        kvq.evict_compact(dc, keep.int(), n, scores=sc)
        for t, p in dc.planes.items():
            for name, x in p.items():
                if x.dim() < 3 or x.shape[2] != n:
                    continue
                at = keep if x.dim() == 3 else keep[..., None].expand(-1, -1, -1, x.shape[-1])
                assert torch.equal(x[:, :, :n_keep], first[t][name].gather(2, at)), (i, t, name)
        assert torch.equal(sc[..., :n_keep], scores.gather(2, keep)) and not sc[..., n_keep:].any()
