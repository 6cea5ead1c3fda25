"""Calls put on a stream that is not the current one, with the buffers left to the call: they are made on the
stream of the launch, so nothing on the current stream is given their memory while the call runs."""
import numpy as np
import pytest
import torch

import sub_byte_quantized_gb300 as kvq
from sub_byte_quantized_gb300 import api

pytestmark = pytest.mark.gpu
B, HQ, H, D, N = 2, 8, 2, 128, 700


def _cache(layout="q4_0", paged=False):
    n_recent = 32 if layout.startswith("had") else 0
    g = torch.Generator("cuda").manual_seed(3)
    k, v = (torch.randn((B, H, N, D), device="cuda", generator=g) for _ in range(2))
    if not paged:
        c = kvq.KVCache(layout, B, H, D, N + 8, n_recent=n_recent)
        kvq.store(c, k, v, 0)
        return c
    c = kvq.PagedKVCache(layout, B, H, D, 64, 2 * B * 12, 12, n_recent=n_recent)
    c.set_block_table(torch.randperm(2 * B * 12, generator=torch.Generator().manual_seed(1))[:B * 12].view(B, 12))
    kvq.paged_store(c, k, v, torch.zeros(B, dtype=torch.int32, device="cuda"))
    return c


def _calls():
    """Every call that makes buffers of its own: name -> f(stream) -> its outputs."""
    g = torch.Generator("cuda").manual_seed(4)
    q = torch.randn((B, HQ, 1, D), device="cuda", generator=g).bfloat16()
    new = [torch.randn((B, h, 1, D), device="cuda", generator=g).bfloat16() for h in (H, H, HQ)]
    lens = torch.tensor([N, 130], dtype=torch.int32, device="cuda")
    after = lens + 1
    slots = torch.tensor([N, 130], dtype=torch.int32, device="cuda")
    c, p, hc = _cache(), _cache(paged=True), _cache("had_int4")
    scores = torch.rand((B, H, N + 4), device="cuda", generator=g)
    freq, _ = kvq.rope_frequencies(D)
    table = kvq.rope_table(freq, N + 8)
    hq = q.cpu()
    host = [x.cpu().pin_memory() for x in new]
    so, po = torch.zeros_like(scores), torch.zeros_like(scores)
    return {
        "decode_attend": lambda s: kvq.decode_attend(c, q, N, stream=s),
        "append_decode_attend": lambda s: kvq.append_decode_attend(c, new[0], new[1], N, q, N + 1, stream=s),
        "decode_attend_static": lambda s: api.decode_attend_static(c, q, N, stream=s),
        "paged_decode_attend": lambda s: kvq.paged_decode_attend(p, q, lens, N, stream=s),
        "paged_append_decode_attend": lambda s: kvq.paged_append_decode_attend(p, new[0], new[1], q, after, N + 1, stream=s),
        "append_decode_attend_host": lambda s: kvq.append_decode_attend_host(c, host[0], host[1], N, hq, N + 1, stream=s),
        "debug_scores_i32": lambda s: api.debug_scores_i32(hc, q, N, stream=s),
        "debug_attend_scores_i32": lambda s: api.debug_attend_scores_i32(hc, q, N, stream=s),
        "rope_table": lambda s: kvq.rope_table(freq, 500, stream=s),
        "rope_store": lambda s: kvq.rope_store(c, table, new[0], new[1], N, q=new[2], stream=s),
        "paged_rope_store": lambda s: kvq.paged_rope_store(p, table, new[0], new[1], slots, q=new[2], stream=s),
        "decode_attend_weights": lambda s: kvq.decode_attend_weights(c, q, N, scores, scores_out=so, stream=s),
        "paged_decode_attend_weights": lambda s: kvq.paged_decode_attend_weights(p, q, lens, N, scores, scores_out=po, stream=s),
        "evict_select": lambda s: kvq.evict_select(scores, N, 100, n_recent=10, stream=s),
    }


def _tensors(x):
    return [x] if isinstance(x, torch.Tensor) else [t for y in x for t in _tensors(y)]


@pytest.mark.parametrize("as_handle", [False, True])
def test_a_calls_own_buffers_belong_to_its_stream(monkeypatch, as_handle):
    calls = _calls()
    want = {name: [t.clone() for t in _tensors(f(None))] for name, f in calls.items()}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    made = []
    empty, full, zeros = torch.empty, torch.full, torch.zeros

    def spy(f):
        def g(*a, **k):
            t = f(*a, **k)
            if t.is_cuda:
                made.append((torch.cuda.current_stream().cuda_stream, t.data_ptr(), t.numel() * t.element_size()))
            return t
        return g
    for name, f in calls.items():
        made.clear()
        for n, x in (("empty", empty), ("full", full), ("zeros", zeros)):
            monkeypatch.setattr(api.torch, n, spy(x))
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)                      # the call's kernels are still to come when it returns
        got = f(s.cuda_stream if as_handle else s)
        monkeypatch.undo()
        assert made and all(x[0] == s.cuda_stream for x in made), name
        # what the current stream is given next is none of it
        others = [torch.empty(size, dtype=torch.uint8, device="cuda") for _, _, size in made]
        for o in others:
            for _, at, size in made:
                assert o.data_ptr() + o.numel() <= at or at + size <= o.data_ptr(), name
        s.synchronize()
        for a, b in zip(_tensors(got), want[name]):
            assert torch.equal(a, b), name


def test_the_legacy_stream_by_its_handle():
    f = _calls()["evict_select"]
    a, b = f(0), f(None)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_a_workspace_made_inside_a_capture_is_the_graphs():
    """Captured on a stream that is passed by name while it is also the current one, and replayed on other inputs."""
    c = _cache()
    q = torch.randn((B, HQ, 1, D), device="cuda").bfloat16()
    scores = torch.zeros((B, H, N), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        kvq.decode_attend_weights(c, q, N, None, scores_out=scores, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out, _ = kvq.decode_attend_weights(c, q, N, None, scores_out=scores, stream=s)
    q.copy_(torch.randn((B, HQ, 1, D), device="cuda").bfloat16())
    g.replay()
    torch.cuda.synchronize()
    want, ws = kvq.decode_attend_weights(c, q, N, None, scores_out=torch.zeros_like(scores))
    assert torch.equal(out, want) and torch.equal(scores, ws)
    assert np.isfinite(out.cpu().numpy()).all()


def test_an_output_dropped_while_it_is_read_on_the_current_stream():
    """Its memory goes to nobody, on the call's stream either, before that read is over."""
    calls = _calls()
    s, here = torch.cuda.Stream(), torch.cuda.current_stream()
    for name, f in calls.items():
        if name.endswith("_host"):                          # (its output is the host's)
            continue
        want = [t.clone() for t in _tensors(f(None))]
        s.wait_stream(here)
        got = [t for t in _tensors(f(s))]
        here.wait_stream(s)
        torch.cuda._sleep(40_000_000)
        kept = [(t.data_ptr(), t.numel() * t.element_size()) for t in got]
        copies = [t.clone() for t in got]
        own = [i for i, t in enumerate(got) if not (name.endswith("weights") and i == 1)]   # (scores_out is the caller's)
        del got
        with torch.cuda.stream(s):
            for i in own:
                t = torch.empty(kept[i][1], dtype=torch.uint8, device="cuda")
                assert t.data_ptr() + t.numel() <= kept[i][0] or kept[i][0] + kept[i][1] <= t.data_ptr(), name
                t.zero_()
        torch.cuda.synchronize()
        for a, b in zip(copies, want):
            assert torch.equal(a, b), name
