"""The serving-step calls on a stream that is not the current one, with the buffers left to the call, and in graphs."""
import numpy as np
import pytest
import torch

import sub_byte_quantized_gb300 as kvq
from sub_byte_quantized_gb300 import api

pytestmark = pytest.mark.gpu
B, HQ, H, D, N = 2, 8, 2, 128, 700


def _cache(layout="int8_b64"):
    g = torch.Generator("cuda").manual_seed(3)
    k, v = (torch.randn((B, H, N, D), device="cuda", generator=g) for _ in range(2))
    c = kvq.PagedKVCache(layout, B, H, D, 64, 2 * B * 12, 12)
    c.set_block_table(torch.randperm(2 * B * 12, generator=torch.Generator().manual_seed(1))[:B * 12].view(B, 12))
    kvq.paged_store(c, k, v, torch.zeros(B, dtype=torch.int32, device="cuda"))
    return c


def _calls():
    """Every new call that makes buffers of its own: name -> f(stream) -> its outputs."""
    g = torch.Generator("cuda").manual_seed(4)
    q, many = (torch.randn((B, HQ, n, D), device="cuda", generator=g).bfloat16() for n in (1, 50))
    lens = torch.tensor([N, 130], dtype=torch.int32, device="cuda")
    c = _cache()
    b = kvq.BlockBounds(c)
    kvq.paged_block_bounds(c, b, lens, N)
    sel = kvq.paged_block_select(c, b, q, lens, N, 4)
    new, table, free, n_free = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([40, 3], [[1, 2, 3, 0]] * 2, list(range(30)), [20]))
    short = lens.clamp(max=170)
    return {
        "page_plan": lambda s: list(kvq.page_plan(short, new, table, 64, free, n_free, 64, stream=s)),
        "paged_block_select": lambda s: kvq.paged_block_select(c, b, q, lens, N, 4, stream=s),
        "paged_sparse_attend": lambda s: kvq.paged_sparse_attend(c, q, sel, lens, N, stream=s),
        "paged_decode_attend": lambda s: kvq.paged_decode_attend(c, q, lens, N, stream=s),
        "many rows": lambda s: kvq.paged_decode_attend(c, many, lens, N, causal=True, stream=s),
    }


def test_buffers_belong_to_the_calls_stream(monkeypatch):
    calls = _calls()
    want = {}
    for name, f in calls.items():
        got = f(None)
        want[name] = [t.clone() for t in (got if isinstance(got, list) else [got])]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    made = []
    empty = torch.empty

    def spy(*a, **k):
        t = empty(*a, **k)
        if t.is_cuda:
            made.append(torch.cuda.current_stream().cuda_stream)
        return t
    for name, f in calls.items():
        made.clear()
        monkeypatch.setattr(api.torch, "empty", spy)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
        got = f(s)
        monkeypatch.undo()
        assert made and all(x == s.cuda_stream for x in made), name
        s.synchronize()
        for x, y in zip(got if isinstance(got, list) else [got], want[name]):
            assert torch.equal(x, y), name


def test_two_calls_at_once_on_two_streams():
    """Attention, selection and sparse attention overlap on two streams, each with its own workspace: the same bits as alone."""
    c = _cache("e4m3_b64")
    b = kvq.BlockBounds(c)
    lens = torch.tensor([N, 333], dtype=torch.int32, device="cuda")
    kvq.paged_block_bounds(c, b, lens, N)
    qs = [torch.randn((B, HQ, 1, D), device="cuda").bfloat16() for _ in range(2)]

    def step(q, s=None):
        sel = kvq.paged_block_select(c, b, q, lens, N, 5, stream=s)
        return kvq.paged_decode_attend(c, q, lens, N, stream=s), sel, kvq.paged_sparse_attend(c, q, sel, lens, N, stream=s)
    want = [[t.clone() for t in step(q)] for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        got = [step(q, s) for q, s in zip(qs, streams)]
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            for u, v in zip(x, y):
                assert torch.equal(u, v)


def test_a_serving_step_in_a_graph():
    """plan, ragged append, bounds, selection and sparse attention captured once; replayed while requests grow, end and come back."""
    rng = np.random.default_rng(2)
    n_pages, per, page, tokens, n_sel = 16, 4, 64, 32, 3
    c = kvq.PagedKVCache("int8_b64", B, H, D, page, n_pages, per)
    d = kvq.PagedKVCache("int8_b64", B, H, D, page, n_pages, per)
    bounds, other = kvq.BlockBounds(c), kvq.BlockBounds(d)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")              # noqa: E731
    lens, new, free, n_free = i32([0, 0]), i32([20, 12]), i32(list(range(n_pages))), i32([n_pages])
    state2 = [t.clone() for t in (lens, free, n_free)]
    k, v = (torch.zeros((tokens, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros((B, HQ, 1, D), dtype=torch.bfloat16, device="cuda")

    def step(cache, bnd, lens, free, n_free):
        p = kvq.page_plan(lens, new, cache.block_table, page, free, n_free, tokens, lens_out=lens, n_free_out=n_free)
        kvq.paged_store_slots(cache, k, v, p.slots)
        kvq.paged_block_bounds(cache, bnd, p.lens, tokens)
        sel = kvq.paged_block_select(cache, bnd, q, p.lens, page * per, n_sel)
        return kvq.paged_sparse_attend(cache, q, sel, p.lens, page * per), sel, p.granted
    warm = [t.clone() for t in (lens, free, n_free)]
    step(d, other, *warm)                                  # (the extension's first calls, outside the capture)
    for t in d.planes.values():
        for x in t.values():
            x.zero_()
    d.block_table.zero_()
    other.codes.zero_(), other.scale.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(c, bounds, lens, free, n_free)
    for want_new in ([20, 12], [1, 1], [5, -1], [1, 31], [1, 1], [-1, 1], [32, 0]):
        new.copy_(i32(want_new))
        for x in (k, v, q):
            x.copy_(torch.from_numpy(rng.standard_normal(x.shape).astype(np.float32)))
        g.replay()
        eager = step(d, other, *state2)
        for a, b in zip(out, eager):
            assert torch.equal(a, b), want_new
        assert torch.equal(lens, state2[0]) and torch.equal(n_free, state2[2]) and torch.equal(c.block_table, d.block_table)
        for t in ("k", "v"):
            for name in ("payload", "scale"):
                assert torch.equal(c.planes[t][name], d.planes[t][name])
