"""Page plans and the ragged append by their slot maps, against the oracle."""
import numpy as np
import pytest
import torch

import sub_byte_quantized_gb300 as kvq
from oracle import serving as OV

pytestmark = pytest.mark.gpu


def _dev(x, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).cuda()


def _check(seq, new, table, page, free, n_free, tokens, in_place=False):
    t, f = np.array(table, np.int32), np.array(free, np.int32)
    args = [_dev(seq), _dev(new), _dev(t), _dev(f), _dev([n_free])]
    want = OV.page_plan(seq, new, t, page, f, n_free, tokens)
    kw = dict(lens_out=args[0], granted=args[1], n_free_out=args[4]) if in_place else {}
    got = kvq.page_plan(args[0], args[1], args[2], page, args[3], args[4], tokens, **kw)
    for name, w in want.items():
        assert np.array_equal(getattr(got, name).cpu().numpy(), w), name
    assert np.array_equal(args[2].cpu().numpy(), t) and np.array_equal(args[3].cpu().numpy(), f)
    if not in_place:
        assert np.array_equal(args[0].cpu().numpy(), seq) and np.array_equal(args[1].cpu().numpy(), new) and args[4].item() == n_free
    return got


@pytest.mark.parametrize("batch,hi,new,page,spare,share", [
    (1, 0, 1, 64, 1, 1.0), (1, 0, 0, 64, 1, 1.0), (3, 64, 64, 64, 2, 1.0), (33, 700, 40, 64, 20, 0.7), (256, 5000, 1, 128, 300, 1.0),
    (1024, 200, 3, 64, 30, 1.2), (1025, 300, 5, 64, 500, 0.9), (3001, 130, 70, 64, 2500, 0.5), (64, 0, 4000, 128, 1200, 1.0), (5, 9000, 2000, 512, 9, 2.0)])
@pytest.mark.parametrize("seed", [0, 1])
def test_plan(batch, hi, new, page, spare, share, seed):
    rng = np.random.default_rng(seed)
    per = (hi + new + page - 1) // page + (seed == 0)      # seed 1: some requests meet the table's end
    per = max(per, 1)
    seq, want = rng.integers(0, hi + 1, batch), rng.integers(0, new + 1, batch)
    want[rng.random(batch) < 0.1] = -1
    pool = rng.permutation(batch * per + spare)
    table = pool[:batch * per].reshape(batch, per)
    free = np.concatenate((pool[batch * per:], np.full(batch * per, -7)))
    if seed:
        free = free[:spare + 3]                            # not every page that is given back has room
    _check(seq, want, table, page, free, spare, int(batch * new * share), in_place=bool(seed))


def test_plan_edges():
    table, free = np.arange(8).reshape(4, 2), np.arange(100, 110)
    _check([5, 128, 0, 64], [-1, -1, -1, -1], table, 64, free, 3, 0)               # all end; one holds nothing
    _check([128, 127, 1, 64], [1, 1, 127, 64], table, 64, free, 0, 300)            # full, the last slot, no free page
    _check([-5, 4000, 0, 0], [3, 0, 2 ** 31 - 1, 1], table, 64, free, 10, 300)     # lengths out of range are clamped
    _check([0, 0, 0, 0], [1, 1, 1, 1], table, 64, free, 99, 2)                     # more free than the list holds; tokens for two
    _check([0, 0, 0, 0], [0, 0, 0, 0], table, 64, free, -3, 5)
    _check([0] * 4, [2 ** 30] * 4, np.zeros((4, 1 << 11), int), 1 << 19, np.arange(1 << 14), 1 << 14, 100)   # sums past 2^31


def test_plan_of_many_tokens_and_its_graph():
    """The two-launch form, captured and replayed on changing lengths in place: a decode loop's state stays on the device."""
    rng = np.random.default_rng(5)
    B, per, page = 40, 200, 64
    seq, table, free = np.zeros(B, np.int64), np.zeros((B, per), np.int32), rng.permutation(B * per)
    new = rng.integers(1, 3000, B)
    d = [_dev(seq), _dev(new), _dev(table), _dev(free), _dev([B * per])]
    call = lambda: kvq.page_plan(d[0], d[1], d[2], page, d[3], d[4], 20000, lens_out=d[0], granted=d[1], n_free_out=d[4], **bufs)  # noqa: E731
    bufs = {}
    warm = [x.clone() for x in d]
    p = kvq.page_plan(warm[0], warm[1], warm[2], page, warm[3], warm[4], 20000)
    bufs = dict(cu_new=p.cu_new, slots=p.slots, positions=p.positions)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    n_free = B * per
    for step in range(4):
        new = rng.integers(-1, 900, B)
        d[1].copy_(_dev(new))
        g.replay()
        want = OV.page_plan(seq, new, table, page, free, n_free, 20000)
        for name, t in (("lens", d[0]), ("granted", d[1]), ("n_free", d[4]), ("cu_new", p.cu_new), ("slots", p.slots), ("positions", p.positions)):
            assert np.array_equal(t.cpu().numpy(), want[name]), (step, name)
        assert np.array_equal(d[2].cpu().numpy(), table) and np.array_equal(d[3].cpu().numpy(), free)
        seq, n_free = want["lens"], int(want["n_free"][0])


ROWS = ["q4_0", "q6_0", "q8_0", "asym4_g32", "had_int4", "had_int2", "q4_0+q8_0"]


@pytest.mark.parametrize("layout", ROWS)
@pytest.mark.parametrize("D,dtype", [(128, torch.bfloat16), (256, torch.float32), (128, torch.float16)])
def test_ragged_append_writes_the_rows_of_the_paged_append(layout, D, dtype):
    """Every token's bytes and scales are those of paged_store; tokens without a slot write nothing."""
    B, H, page, per = 3, 2, 64, 4
    g = torch.Generator("cuda").manual_seed(2)
    n = 70
    kv = torch.randn((B * n, 3 * H * D), device="cuda", generator=g).to(dtype)     # k, something else, v of a token side by side
    k, _, v = kv.view(B * n, 3, H, D).unbind(1)
    a, b = (kvq.PagedKVCache(layout, B, H, D, page, 2 * B * per, per) for _ in range(2))
    table = torch.randperm(2 * B * per, generator=torch.Generator().manual_seed(1))[:B * per].view(B, per)
    first = torch.tensor([0, 37, 100], dtype=torch.int32)
    a.set_block_table(table)
    kvq.paged_store(a, *(x.view(B, n, H, D).transpose(1, 2).contiguous() for x in (k, v)), first.cuda())
    pos = first.long()[:, None] + torch.arange(n)
    slots = (torch.gather(table, 1, pos // page) * page + pos % page).flatten().cuda()
    drop = torch.arange(B * n, device="cuda") % 11 == 3
    kvq.paged_store_slots(b, k, v, torch.where(drop, torch.tensor([-1, 2 ** 40], device="cuda")[torch.arange(B * n, device="cuda") % 2], slots))
    for t in ("k", "v"):
        for name, x in a.planes[t].items():
            x, y = (p.transpose(1, 2).flatten(0, 1).flatten(1) for p in (x, b.planes[t][name]))     # pool rows
            assert torch.equal(x[slots[~drop]], y[slots[~drop]]), (t, name)
            assert not y[slots[drop]].any()
            kept = torch.ones(len(x), dtype=torch.bool, device="cuda")
            kept[slots] = False
            assert not y[kept].any()


def test_wrappers_refuse():
    c = kvq.PagedKVCache("q4_0", 1, 2, 128, 64, 4, 4)
    k, s = torch.zeros((3, 2, 128), device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in ((k[..., :64], k, s), (k, k.half(), s), (k.int(), k.int(), s), (k, k, s.int()), (k, k, s[:2]), (k, k, s.cpu()), (k[0], k[0], s)):
        with pytest.raises(ValueError):
            kvq.paged_store_slots(c, *bad)
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    table, free = torch.zeros((2, 4), dtype=torch.int32, device="cuda"), torch.zeros(9, dtype=torch.int32, device="cuda")
    for bad in ((i[:1], i, table, 64, free, i[:1], 4), (i, i.long(), table, 64, free, i[:1], 4), (i, i, table.t(), 64, free, i[:1], 4),
                (i, i, table, 64, free, i, 4), (i, i, table[0], 64, free, i[:1], 4), (i, i.cpu(), table, 64, free, i[:1], 4)):
        with pytest.raises(ValueError):
            kvq.page_plan(*bad)
    with pytest.raises(kvq.KvqError):
        kvq.page_plan(i, i.clone(), table, 60, free, torch.zeros(1, dtype=torch.int32, device="cuda"), 4)
