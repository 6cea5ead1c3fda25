"""The operators of a serving step over a packed K/V cache in blocks of 64 tokens that are measured here,
each in its plain form (elementary torch operations) and as a user's calls of the library:

  plan     a step's pages, block-table entries and slot map, from the requests' lengths
  append   rows quantised into an 8-bit cache with one scale per block of 64 tokens and head
  attend   attention over that cache
  select   bounds of the keys of each block of 64 tokens, and the blocks that they select for each query
  sparse   attention over the selected blocks alone

`listed()` and `draw()` give the cases, `prepare()` what a program holds before the call, `run()` one
call and its outputs, `work()` the bytes and operations it cannot do without, `exact()` the outputs
from the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TOKENS = 64                                         # tokens of a block
TOP = {"int8_b64": 127.0, "e4m3_b64": 448.0}        # largest code value of the block layouts


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the decode step of a serving batch: one token for each of 256 requests, some of which have ended
        {"name": "plan 256 decode rows", "kind": "plan", "batch": 256, "page": 64, "hi": 8192, "new_lo": 1, "new_hi": 1, "tokens": 256, "spare": 300},
        # a step of whole prompts, more than the pool's free pages hold: the last ones have to wait
        {"name": "plan 64 prompts", "kind": "plan", "batch": 64, "page": 128, "hi": 0, "new_lo": 501, "new_hi": 8191, "tokens": 262144, "spare": 2000},
        # the decode step's append: blocks that are partly full, so that a larger value changes their scale
        {"name": "append 1 token x 64, paged e4m3", "kind": "append", "layout": "e4m3_b64", "batch": 64, "hkv": 8, "d": 128, "lo": 1, "hi": 1,
         "cap": 2048, "page": 64, "dtype": "bf16", "by_slots": False},
        # a step of prompts and decode rows in one ragged run of tokens, by the slot map
        {"name": "append ragged x 16 by slots, int8", "kind": "append", "layout": "int8_b64", "batch": 16, "hkv": 8, "d": 128, "lo": 1, "hi": 1531,
         "cap": 4096, "page": 128, "dtype": "bf16", "by_slots": True},
        # one decode step at 128K tokens with 64 query heads on 8 kv heads
        {"name": "attend 1 row, 128K, int8", "kind": "attend", "layout": "int8_b64", "batch": 1, "hq": 64, "hkv": 8, "d": 128, "n_q": 1,
         "lo": 131072, "hi": 131072, "page": 0, "dtype": "bf16", "causal": False},
        # one decode step of a ragged serving batch
        {"name": "attend 1 row, ragged x 16, e4m3", "kind": "attend", "layout": "e4m3_b64", "batch": 16, "hq": 32, "hkv": 8, "d": 128, "n_q": 1,
         "lo": 1021, "hi": 16379, "page": 64, "dtype": "bf16", "causal": False},
        # a prefill chunk of 256 rows behind 3840 cached tokens
        {"name": "attend 256 rows x 8, 4096, int8", "kind": "attend", "layout": "int8_b64", "batch": 8, "hq": 16, "hkv": 8, "d": 128, "n_q": 256,
         "lo": 4096, "hi": 4096, "page": 0, "dtype": "bf16", "causal": True},
        # the first decode step behind a 128K prompt: every block's bounds are made, then 64 of them are selected
        {"name": "select 64 of 2048, after a prompt", "kind": "select", "layout": "q4_0", "batch": 1, "hq": 64, "hkv": 8, "d": 128, "n_q": 1,
         "lo": 131072, "hi": 131072, "page": 0, "dtype": "bf16", "causal": False, "fresh": 131072, "n_sel": 64},
        # a decode step of a ragged batch: the newest block's bounds are renewed, then the selection
        {"name": "select 32 of up to 255 x 32", "kind": "select", "layout": "int8_b64", "batch": 32, "hq": 32, "hkv": 8, "d": 128, "n_q": 1,
         "lo": 1021, "hi": 16317, "page": 64, "dtype": "bf16", "causal": False, "fresh": 1, "n_sel": 32},
        # a decode step over 64 blocks (4096 tokens) of a 128K cache
        {"name": "sparse 64 blocks of 128K, q4_0", "kind": "sparse", "layout": "q4_0", "batch": 1, "hq": 64, "hkv": 8, "d": 128, "n_q": 1,
         "lo": 131072, "hi": 131072, "page": 0, "dtype": "bf16", "causal": False, "n_sel": 64},
        # a decode step of a ragged batch, some sequences shorter than the selection
        {"name": "sparse 32 blocks x 32, int8", "kind": "sparse", "layout": "int8_b64", "batch": 32, "hq": 32, "hkv": 8, "d": 128, "n_q": 1,
         "lo": 1021, "hi": 16317, "page": 64, "dtype": "bf16", "causal": False, "n_sel": 32},
        # 64 rows of a prompt, each with blocks of its own
        {"name": "sparse 64 rows x 32 blocks, q8_0", "kind": "sparse", "layout": "q8_0", "batch": 1, "hq": 32, "hkv": 8, "d": 128, "n_q": 64,
         "lo": 32749, "hi": 32749, "page": 64, "dtype": "bf16", "causal": True, "n_sel": 32},
    ]


def _log(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("plan", "append", "append", "attend", "attend", "attend", "select", "select", "sparse", "sparse"))
    page = rng.choice((0, 64, 128))
    if kind == "plan":
        batch, hi, new = _log(rng, 1, 1024), _log(rng, 1, 9000), _log(rng, 1, 2000)
        return {"kind": kind, "batch": batch, "page": 64 * 2 ** rng.randint(0, 3), "hi": rng.choice((0, hi)), "new_lo": rng.randint(0, new),
                "new_hi": new, "tokens": min(200000, max(1, int(batch * new * rng.uniform(0.3, 1.3)))), "spare": _log(rng, 1, 3000)}
    hkv, d = rng.choice((1, 2, 4, 8)), rng.choice((128, 128, 256))
    c = {"kind": kind, "layout": rng.choice(tuple(TOP)), "batch": _log(rng, 1, 8), "hkv": hkv, "d": d, "page": page, "dtype": rng.choice(tuple(DTYPES))}
    if kind == "append":
        hi = rng.choice((1, 2, _log(rng, 3, 900)))
        by_slots = page > 0 and rng.random() < 0.6
        return dict(c, batch=_log(rng, 1, 32 if hi < 10 else 4), hi=hi, lo=rng.randint(1, hi) if by_slots else hi,
                    cap=128 * ((hi + rng.randint(0, 500)) // 128 + 2), by_slots=by_slots)
    hi = _log(rng, 1 if kind == "attend" else 130, 8000)
    n_q = rng.choice((1, 1, 1, 2, _log(rng, 3, 70 if kind == "attend" else 20)))
    n_q = min(n_q, hi)
    c = dict(c, hq=hkv * rng.choice((1, 2, 4, 8)), n_q=n_q, lo=rng.randint(1, hi) if page else hi, hi=hi, causal=n_q > 1)
    if kind == "attend":
        return c
    c["layout"] = rng.choice(("int8_b64", "e4m3_b64", "q4_0", "q8_0"))
    c["n_sel"] = _log(rng, 3, 40)
    if kind == "select":
        c["fresh"] = rng.choice((1, min(c["lo"], 100), c["lo"]))
    return c


# ------------------------------------------------------------------------------- the packed layouts
def _row_bytes(layout, d):
    return d // 2 if layout == "q4_0" else d


def _e4m3(x):
    """Nearest e4m3 bytes, saturating."""
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _byte_codes(layout, x, s):
    """Code bytes of the block layouts: x by the scale, nearest, 0 where the scale is 0 (divisions by tensors: correctly rounded)."""
    y = torch.where(s > 0, x / torch.where(s > 0, s, 1.0), 0.0)
    return _e4m3(y) if layout == "e4m3_b64" else y.round().clamp(-127.0, 127.0).to(torch.int32).bitwise_and(255).to(torch.uint8)


def _code_values(layout, payload):
    return payload.view(torch.float8_e4m3fn).float() if layout == "e4m3_b64" else payload.view(torch.int8).float()


def _pack32(layout, x):
    """float32 rows [..., D] -> (payload, f16 scales) of q4_0 or q8_0: blocks of 32 values, scale = amax / 8 or / 128."""
    b = x.reshape(x.shape[:-1] + (x.shape[-1] // 32, 32))
    top = 8 if layout == "q4_0" else 128
    s = (b.abs().amax(-1, keepdim=True) / float(top)).clamp(max=65504.0).half()    # a power of two: the reciprocal is exact
    f = s.float()
    c = torch.where(f > 0, torch.round(b / torch.where(f > 0, f, 1.0)).clamp(-top, top - 1), 0.0).to(torch.int32)
    p = (c[..., 0::2] & 15) | ((c[..., 1::2] & 15) << 4) if layout == "q4_0" else c & 255
    return p.to(torch.uint8).flatten(-2), s[..., 0]


def _unpack(layout, payload, scale, to=torch.float32):
    """The values that rows [..., row bytes] stand for; scale [..., D/32], or for the block layouts one per row [...]."""
    if layout in TOP:
        return _code_values(layout, payload).to(to) * scale.to(to).unsqueeze(-1)
    if layout == "q4_0":
        u = torch.stack((payload & 15, payload >> 4), -1).flatten(-2).to(torch.int32)
        c = (u ^ 8) - 8
    else:
        c = payload.view(torch.int8)
    c = c.to(to)
    return (c.reshape(c.shape[:-1] + (scale.shape[-1], 32)) * scale.to(to).unsqueeze(-1)).flatten(-2)


# ------------------------------------------------------------------------------------------ prepare
def _lens(case):
    """The batch's lengths: spread evenly over the case's range, so that the work is the case's own."""
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    return [hi - (hi - lo) * i // max(1, b - 1) for i in range(b)]


def _make_cache(case, cap, gen, full=True):
    """The cache's planes as tensors [pages][H][page][...] with a shuffled table; a contiguous cache is one page a sequence.
    Its values have a few channels far larger than the rest."""
    b, h, d, layout = case["batch"], case["hkv"], case["d"], case["layout"]
    cap = (cap + 63) // 64 * 64
    page = case["page"] or cap
    per = (cap + page - 1) // page
    c = {"layout": layout, "b": b, "h": h, "d": d, "page": page, "per": per}
    c["table"] = (torch.randperm(b * per, device="cuda", generator=gen).reshape(b, per) if case["page"]
                  else torch.arange(b, device="cuda")[:, None]).to(torch.int32)
    big = torch.randperm(d, device="cuda", generator=gen)[:4]
    c["k"], c["v"] = _plane(c, gen, big, full), _plane(c, gen, big.flip(0)[:2], full)
    if own:
        import sub_byte_quantized_gb300 as kvq
        if case["page"]:
            c["handle"] = kvq.PagedKVCache(layout, b, h, d, page, b * per, per)
            c["handle"].set_block_table(c["table"])
        else:
            c["handle"] = kvq.KVCache(layout, b, h, d, cap)
        for t in ("k", "v"):
            for name, x in c[t].items():
                c["handle"].planes[t][name].view(x.shape).copy_(x)
            c[t] = {name: c["handle"].planes[t][name].view(x.shape) for name, x in c[t].items()}
    return c


def _plane(c, gen, big, full):
    lead, d, layout = (c["b"] * c["per"], c["h"], c["page"]), c["d"], c["layout"]
    if not full and layout in TOP:
        return {"payload": torch.zeros(lead + (d,), device="cuda", dtype=torch.uint8), "scale": torch.zeros(lead[:2] + (lead[2] // TOKENS,), device="cuda")}
    x = torch.randn(lead + (d,), device="cuda", generator=gen)
    x[..., big] *= 6.0
    if layout not in TOP:
        payload, scale = _pack32(layout, x)
        return {"payload": payload, "scale": scale}
    s = x.reshape(lead[:2] + (lead[2] // TOKENS, TOKENS * d)).abs().amax(-1)
    s = s / torch.full_like(s, TOP[layout])
    return {"payload": _byte_codes(layout, x, s.repeat_interleave(TOKENS, -1)[..., None]), "scale": s}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case, "kind": case["kind"]}
    if case["kind"] == "plan":
        return _prepare_plan(s, case, gen)
    b, h, d = case["batch"], case["hkv"], case["d"]
    dtype = DTYPES[case["dtype"]]
    if case["kind"] == "append":
        new = _lens(case)
        c = s["cache"] = _make_cache(case, case["cap"], gen, full=False)
        first = torch.randint(0, case["cap"] - case["hi"] + 1, (b,), device="cuda", generator=gen)
        s["pos0"] = seed % (case["cap"] - case["hi"] + 1)
        if not case["page"]:
            first = torch.full_like(first, s["pos0"])
        # every sequence's earlier tokens are in the cache: the block that the first new one falls into is partly full
        t = torch.arange(c["page"] * c["per"], device="cuda")
        old = torch.randn((b, t.numel(), h, d), device="cuda", generator=gen) * 0.7
        at = torch.where(t < first[:, None], _slots(c, torch.arange(b, device="cuda")[:, None], t), -1)
        _put(c["k"], c, at.flatten(), old.flatten(0, 1))
        _put(c["v"], c, at.flatten(), old.flatten(0, 1).flip(0))
        del old
        if case["by_slots"]:                        # the projection's output of all new tokens, k and v heads side by side
            seq = torch.repeat_interleave(torch.arange(b, device="cuda"), torch.tensor(new, device="cuda"))
            begin = torch.tensor([sum(new[:i]) for i in range(b)], device="cuda")
            s["slots"] = _slots(c, seq, first[seq] + torch.arange(seq.numel(), device="cuda") - begin[seq])
            s["kv"] = torch.randn((seq.numel(), 2 * h * d), device="cuda", generator=gen).to(dtype)
            return s
        s["positions"] = first.to(torch.int32)
        s["k_new"], s["v_new"] = (torch.randn((b, h, case["hi"], d), device="cuda", generator=gen).to(dtype) for _ in range(2))
        return s
    s["lens"] = _lens(case)
    s["seq_lens"] = torch.tensor(s["lens"], device="cuda", dtype=torch.int32)
    n = max(s["lens"])
    c = s["cache"] = _make_cache(case, n, gen)
    s["q"] = torch.randn((b, case["hq"], case["n_q"], d), device="cuda", generator=gen).to(dtype)
    if case["kind"] == "select":
        lead = (b * c["per"], h, c["page"] // TOKENS)
        codes = torch.randint(-127, 1, lead + (2, d), device="cuda", generator=gen, dtype=torch.int8)
        codes[..., 1, :] = -codes[..., 1, :]
        scale = torch.rand(lead, device="cuda", generator=gen) * 0.02 + 0.02
        s["codes"], s["scale"] = codes, scale
        if own:
            import sub_byte_quantized_gb300 as kvq
            s["bounds"] = kvq.BlockBounds(c["handle"])
            s["codes"], s["scale"] = s["bounds"].codes.view(codes.shape), s["bounds"].scale.view(scale.shape)
            s["codes"].copy_(codes)
            s["scale"].copy_(scale)
    if case["kind"] == "sparse":
        x = torch.rand((b, h, case["n_q"], (n + TOKENS - 1) // TOKENS), device="cuda", generator=gen)
        s["sel"] = _top(x, _limits(s), case["n_sel"])
    return s


def _prepare_plan(s, case, gen):
    b, page = case["batch"], case["page"]
    rand = lambda lo, hi, shape: torch.randint(lo, hi + 1, shape, device="cuda", generator=gen, dtype=torch.int32)  # noqa: E731
    per = (case["hi"] + case["new_hi"] + page - 1) // page + 1
    s["seq_lens"] = rand(0, case["hi"], (b,))
    s["new_lens"] = rand(case["new_lo"], case["new_hi"], (b,))
    s["new_lens"][rand(0, 15, (b,)) == 0] = -1      # requests that have ended
    held = (s["seq_lens"] + page - 1) // page
    pool = torch.randperm(b * per + case["spare"], device="cuda", generator=gen).to(torch.int32)
    s["table"] = torch.where(torch.arange(per, device="cuda") < held[:, None], pool[:b * per].view(b, per), 0).contiguous()
    s["free"] = torch.cat((pool[b * per:], torch.zeros(b * per, device="cuda", dtype=torch.int32)))
    s["n_free"] = torch.tensor([case["spare"]], device="cuda", dtype=torch.int32)
    return s


# ---------------------------------------------------------------------------------- the plain forms
def _plain_plan(s):
    case = s["case"]
    page, tokens, table, free = case["page"], case["tokens"], s["table"], s["free"]
    b, per = table.shape
    old, new = s["seq_lens"].long().clamp(0, per * page), s["new_lens"].long()
    held = (old + page - 1) // page
    j = torch.arange(per, device="cuda")
    # pages of ended requests go behind the free ones
    back = torch.where(new < 0, held, 0)
    n_free = s["n_free"].long().clamp(0, free.numel())
    at = n_free + torch.cumsum(back, 0)[:, None] - back[:, None] + j
    live = (j < back[:, None]) & (at < free.numel())
    grown = torch.cat((free, free.new_zeros(1)))
    grown[torch.where(live, at, free.numel())] = table
    free.copy_(grown[:-1])
    n_free = (n_free + back.sum()).clamp(max=free.numel())
    # in the requests' order: what the table, the free pages and the step's tokens have room for
    ok = (new >= 0) & (old + new <= per * page)
    need = torch.where(ok, (old + new + page - 1) // page - held, 0)
    ok = ok & ((need == 0) | (torch.cumsum(need, 0) <= n_free))
    want = torch.where(ok, new, 0)
    ok = ok & ((want == 0) | (torch.cumsum(want, 0) <= tokens))
    granted, need = torch.where(ok, new, 0), torch.where(ok, need, 0)
    taken = torch.cumsum(need, 0)
    k = j - held[:, None]
    pick = (n_free - 1 - (taken - need)[:, None] - k).clamp(0, free.numel() - 1)
    table.copy_(torch.where((k >= 0) & (k < need[:, None]), free[pick], table))
    ends = torch.cumsum(granted, 0)
    i = torch.arange(tokens, device="cuda")
    seq = torch.searchsorted(ends, i, right=True).clamp(max=b - 1)
    pos = old[seq] + i - (ends - granted)[seq]
    some = i < ends[-1]
    row = torch.gather(table[seq], 1, (pos // page).clamp(0, per - 1)[:, None])[:, 0].long() * page + pos % page
    return {"lens": torch.where(new < 0, 0, old + granted).to(torch.int32), "granted": granted.to(torch.int32), "n_free": (n_free - taken[-1]).to(torch.int32),
            "cu_new": torch.cat((ends.new_zeros(1), ends)).to(torch.int32), "slots": torch.where(some, row, -1),
            "positions": torch.where(some, pos, -1).to(torch.int32), "table": table, "free": free}


def _slots(c, seq, t):
    """Pool rows of the tokens t of the sequences seq."""
    return c["table"].long()[seq, (t // c["page"]).clamp(max=c["per"] - 1)] * c["page"] + t % c["page"]


def _put(plane, c, slots, x):
    """Rows x [T][H][D] (float32) into the pool rows slots [T] (-1: none). A block whose first new row is its first
    row gets the scale that its new rows need; any other keeps its scale, or doubles it until they fit, and then the
    codes of the rows in front of them are rounded once more."""
    layout, h = c["layout"], c["h"]
    slots, x = slots[slots >= 0], x[slots >= 0]
    n = plane["scale"].numel() // h
    block = slots // TOKENS
    first = torch.full((n,), TOKENS, device="cuda").scatter_reduce_(0, block, slots % TOKENS, "amin")
    top = torch.zeros((n, h), device="cuda").scatter_reduce_(0, block[:, None].expand(-1, h), x.abs().amax(-1), "amax")
    hit = (first < TOKENS).nonzero()[:, 0]
    per = c["page"] // TOKENS
    p, i = hit // per, hit % per
    old = torch.where(first[hit, None] > 0, plane["scale"][p, :, i], 0.0)
    need = top[hit] / torch.full_like(top[hit], TOP[layout])
    grow = (need > old) & (old > 0)
    (mo, eo), (mn, en) = torch.frexp(torch.where(grow, old, 1.0)), torch.frexp(torch.where(grow, need, 1.0))
    k = torch.where(grow, (en - eo + (mn > mo)).clamp(max=64), 0)
    plane["scale"][p, :, i] = torch.where(need > old, torch.where(grow, torch.ldexp(old, k), need), old)
    rows = plane["payload"].view(-1, h, per, TOKENS, c["d"])
    was = rows[p, :, i]
    value = torch.ldexp(_code_values(layout, was), -k[:, :, None, None])
    less = _e4m3(value) if layout == "e4m3_b64" else value.round().to(torch.int32).bitwise_and(255).to(torch.uint8)
    kept = torch.arange(TOKENS, device="cuda")[:, None] < first[hit, None, None, None]
    rows[p, :, i] = torch.where(kept & (k > 0)[:, :, None, None], less, was)
    page, row = slots // c["page"], slots % c["page"]
    plane["payload"][page, :, row] = _byte_codes(layout, x, plane["scale"][page, :, row // TOKENS][..., None])


def _plain_append(s):
    case, c = s["case"], s["cache"]
    if case["by_slots"]:
        k, v = (x.float() for x in s["kv"].view(-1, 2, c["h"], c["d"]).unbind(1))
        slots = s["slots"]
    else:
        first = s["positions"].long()[:, None] if case["page"] else s["pos0"]
        t = first + torch.arange(case["hi"], device="cuda").expand(c["b"], -1)
        slots = _slots(c, torch.arange(c["b"], device="cuda")[:, None], t).flatten()
        k, v = (x.float().transpose(1, 2).flatten(0, 1) for x in (s["k_new"], s["v_new"]))
    _put(c["k"], c, slots, k)
    _put(c["v"], c, slots, v)
    return {"k": c["k"], "v": c["v"]}


def _values(c, plane, at, to=torch.float32):
    """The values of the pool rows `at` = (page, head, row) of a plane."""
    page, head, row = at
    scale = plane["scale"][page, head, row // TOKENS] if c["layout"] in TOP else plane["scale"][page, head, row]
    return _unpack(c["layout"], plane["payload"][page, head, row], scale, to)


def _where(c, t):
    """(page, head, row) of the logical tokens t [B][1 or H][...]: each shaped [B][H][...]."""
    ones = (1,) * (t.dim() - 2)
    b = torch.arange(c["b"], device="cuda").view(-1, 1, *ones)
    h = torch.arange(c["h"], device="cuda").view(1, -1, *ones)
    page = c["table"].long()[b, (t // c["page"]).clamp(max=c["per"] - 1)]
    return page, h, t % c["page"]


def _limits(s):
    """The last token that each query row sees, [B][1][n_q]; negative where there is none."""
    case, lens = s["case"], s["seq_lens"].long()[:, None, None]
    i = torch.arange(case["n_q"], device="cuda")
    return lens - case["n_q"] + i if case["causal"] else (lens - 1).expand(-1, 1, case["n_q"])


def _softmax(x):
    """Over the last axis; a row that sees nothing gets zeros."""
    m = x.amax(-1, keepdim=True)
    p = (x - torch.where(m == -math.inf, 0.0, m)).exp()
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, 1.0)


def _plain_attend(s):
    case, c = s["case"], s["cache"]
    n, g, n_q = max(s["lens"]), case["hq"] // case["hkv"], case["n_q"]
    at = _where(c, torch.arange(n, device="cuda").expand(c["b"], 1, n))
    q = s["q"].float().reshape(c["b"], c["h"], g * n_q, c["d"])
    sees = torch.arange(n, device="cuda") <= _limits(s).repeat(1, 1, g)[..., None]
    x = torch.where(sees, q @ _values(c, c["k"], at).transpose(-1, -2) / math.sqrt(c["d"]), -math.inf)
    return (_softmax(x) @ _values(c, c["v"], at)).reshape(c["b"], case["hq"], n_q, c["d"])


def _plain_bounds(s):
    """The smallest and largest value of each channel over a block's tokens, in 8 bits, rounded outwards; one scale a block."""
    case, c = s["case"], s["cache"]
    lens = s["seq_lens"].long()[:, None]
    last = (lens - 1) // TOKENS
    i = (lens - case["fresh"]).clamp(min=0) // TOKENS + torch.arange((case["fresh"] + 2 * TOKENS - 2) // TOKENS, device="cuda")
    i = torch.minimum(i, last)                      # [B][blocks that the newest `fresh` tokens touch]
    t = i[:, None, :, None] * TOKENS + torch.arange(TOKENS, device="cuda")
    x = _values(c, c["k"], _where(c, t))            # [B][H][blocks][64][D]
    dead = (t >= lens[:, :, None, None])[..., None]
    lo, hi = x.masked_fill(dead, math.inf).amin(3), x.masked_fill(dead, -math.inf).amax(3)
    scale = torch.maximum(lo.abs(), hi.abs()).amax(-1)
    scale = scale / torch.full_like(scale, 127.0)
    by = torch.where(scale > 0, scale, 1.0)[..., None]
    codes = torch.stack(((lo / by).floor(), (hi / by).ceil()), 3).clamp(-127, 127).to(torch.int8)
    page, h, row = _where(c, i[:, None] * TOKENS)
    s["codes"][page, h, row // TOKENS], s["scale"][page, h, row // TOKENS] = codes, scale


def _plain_scores(s):
    """Each block's score for each query: the largest product that its bounds allow, over the query heads of a kv head."""
    case, c = s["case"], s["cache"]
    n, g = (max(s["lens"]) + TOKENS - 1) // TOKENS, case["hq"] // case["hkv"]
    page, h, row = _where(c, (torch.arange(n, device="cuda") * TOKENS).expand(c["b"], 1, n))
    codes, scale = s["codes"][page, h, row // TOKENS].float(), s["scale"][page, h, row // TOKENS]
    q = s["q"].float().reshape(c["b"], c["h"], g * case["n_q"], c["d"])
    top = q.abs().amax(-1, keepdim=True)
    step = top / torch.full_like(top, 127.0)
    q = torch.where(step > 0, (q / torch.where(step > 0, step, 1.0)).round().clamp(-127, 127), 0.0)
    dots = q.clamp(min=0) @ codes[..., 1, :].transpose(-1, -2) + q.clamp(max=0) @ codes[..., 0, :].transpose(-1, -2)   # whole numbers below 2^24
    return (dots * step * scale[:, :, None]).reshape(c["b"], c["h"], g, case["n_q"], n).amax(2)


def _top(x, limits, n_sel):
    """Ascending block lists [B][H][n_q][n_sel]: the first block, the newest one, then the highest scores, ties to the lowest
    index; a row that sees at most n_sel blocks keeps all of them, and -1 fills the rest."""
    n = x.shape[-1]
    size = torch.div(limits + TOKENS, TOKENS, rounding_mode="floor").clamp(min=0)[..., None]
    i = torch.arange(n, device="cuda")
    rank = torch.where(i < size, ((i < 1) | (i == size - 1)).int(), -1).expand(x.shape)
    by = x.sort(dim=-1, descending=True, stable=True).indices
    by = by.gather(-1, rank.gather(-1, by).sort(dim=-1, descending=True, stable=True).indices)[..., :n_sel]
    by = torch.nn.functional.pad(by, (0, n_sel - by.shape[-1]), value=n)
    by = torch.where(by < size, by, n).sort(dim=-1).values
    return torch.where(by < size, by, -1).to(torch.int32)


def _plain_sparse(s):
    case, c = s["case"], s["cache"]
    g, n_q = case["hq"] // case["hkv"], case["n_q"]
    sel = s["sel"].long()[..., None]
    t = sel * TOKENS + torch.arange(TOKENS, device="cuda")              # [B][H][n_q][n_sel][64]
    sees = ((sel >= 0) & (t <= _limits(s)[..., None, None])).flatten(3)
    at = _where(c, t.clamp(min=0).flatten(3))
    q = s["q"].float().reshape(c["b"], c["h"], g, n_q, c["d"]).transpose(2, 3)
    x = torch.where(sees[:, :, :, None], q @ _values(c, c["k"], at).transpose(-1, -2) / math.sqrt(c["d"]), -math.inf)
    out = _softmax(x) @ _values(c, c["v"], at)                          # [B][H][n_q][g][D]
    return out.transpose(2, 3).reshape(c["b"], case["hq"], n_q, c["d"])


# ------------------------------------------------------------------------------------------- one call
def run(s):
    kind = s["kind"]
    if own:
        return _own(s, s["case"], kind)
    if kind == "plan":
        return _plain_plan(s)
    if kind == "append":
        return _plain_append(s)
    if kind == "attend":
        return _plain_attend(s)
    if kind == "select":
        _plain_bounds(s)
        return {"codes": s["codes"], "scale": s["scale"], "sel": _top(_plain_scores(s), _limits(s), s["case"]["n_sel"])}
    return _plain_sparse(s)


def _own(s, case, kind):
    import sub_byte_quantized_gb300 as kvq
    if kind == "plan":
        p = kvq.page_plan(s["seq_lens"], s["new_lens"], s["table"], case["page"], s["free"], s["n_free"], case["tokens"])
        return {"lens": p.lens, "granted": p.granted, "n_free": p.n_free, "cu_new": p.cu_new, "slots": p.slots, "positions": p.positions,
                "table": s["table"], "free": s["free"]}
    c = s["cache"]
    cache = c["handle"]
    if kind == "append":
        if case["by_slots"]:
            k, v = s["kv"].view(-1, 2, c["h"], c["d"]).unbind(1)
            kvq.paged_store_slots(cache, k, v, s["slots"])
        elif case["page"]:
            kvq.paged_store(cache, s["k_new"], s["v_new"], s["positions"])
        else:
            kvq.store(cache, s["k_new"], s["v_new"], s["pos0"])
        return {"k": c["k"], "v": c["v"]}
    n, q, causal = max(s["lens"]), s["q"], case["causal"]
    q_pos0 = n - case["n_q"] if causal else 0
    if kind == "attend":
        if case["page"]:
            return kvq.paged_decode_attend(cache, q, s["seq_lens"], n, causal=causal)
        return kvq.decode_attend(cache, q, n, causal=causal, q_pos0=q_pos0)
    if kind == "select":
        if case["page"]:
            kvq.paged_block_bounds(cache, s["bounds"], s["seq_lens"], case["fresh"])
            sel = kvq.paged_block_select(cache, s["bounds"], q, s["seq_lens"], n, case["n_sel"], n_sink=1, n_recent=1, causal=causal)
        else:
            kvq.block_bounds(cache, s["bounds"], n - case["fresh"], n)
            sel = kvq.block_select(cache, s["bounds"], q, n, case["n_sel"], n_sink=1, n_recent=1, causal=causal, q_pos0=q_pos0)
        return {"codes": s["codes"], "scale": s["scale"], "sel": sel}
    if case["page"]:
        return kvq.paged_sparse_attend(cache, q, s["sel"], s["seq_lens"], n, causal=causal)
    return kvq.sparse_attend(cache, q, s["sel"], n, causal=causal, q_pos0=q_pos0)


# ------------------------------------------------------------------------------------------- the work
def _token_bytes(layout, d):
    """Bytes of one token of one head in one plane: codes, and its share of the scales."""
    return _row_bytes(layout, d) + (4 / TOKENS if layout in TOP else d // 16)


def work(case):
    kind = case["kind"]
    if kind == "plan":                              # lengths in, lengths out, new table entries, the map of the tokens
        b, page = case["batch"], case["page"]
        new = min(case["tokens"], b * (case["new_lo"] + case["new_hi"]) // 2)
        return {"bytes": 24 * b + 8 * (new // page + 1) + 12 * case["tokens"], "flops": 0}
    h, d = case["hkv"], case["d"]
    size = 4 if case["dtype"] == "f32" else 2
    if kind == "append":                            # k and v read, their codes and scales written
        rows = sum(_lens(case)) * h
        return {"bytes": 2 * rows * (d * size + _token_bytes(case["layout"], d)), "flops": 6 * rows * d}
    lens, b, rows = _lens(case), case["batch"], case["hq"] * case["n_q"]
    q_out = b * rows * d * (4 + size)
    if kind == "attend":                            # both planes once, q and out; two products of what each row sees
        n_q = case["n_q"]
        pairs = sum(n_q * x - (n_q * (n_q - 1) // 2 if case["causal"] else 0) for x in lens)
        return {"bytes": 2 * h * sum(lens) * _token_bytes(case["layout"], d) + q_out, "flops": 4 * pairs * case["hq"] * d}
    blocks = sum((x + TOKENS - 1) // TOKENS for x in lens)
    if kind == "select":                            # the fresh tokens' keys, the bounds, q; the lists written
        fresh = sum(min(x, case["fresh"]) for x in lens)
        return {"bytes": h * (fresh * _token_bytes(case["layout"], d) + (blocks + fresh // TOKENS + b) * (2 * d + 4)) + b * rows * d * size
                + 4 * b * h * case["n_q"] * case["n_sel"], "flops": h * fresh * 2 * d + 4 * blocks * rows * d}
    # each list's blocks, those that several rows of a sequence share once
    lists = sum(min(x, TOKENS * case["n_sel"]) for x in lens)
    some = sum(min(x, TOKENS * case["n_sel"] * case["n_q"]) for x in lens)
    return {"bytes": 2 * h * some * _token_bytes(case["layout"], d) + q_out + 4 * b * h * case["n_q"] * case["n_sel"], "flops": 4 * lists * rows * d}


# ------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    """Whole numbers and codes are bits by definition: no value in 64 bits. Attention: one sequence and kv head at a time."""
    kind = case["kind"]
    if kind == "plan":
        return None
    if kind == "append":
        return {"k": {"payload": None, "scale": _exact_scales(case, seed, "k")}, "v": {"payload": None, "scale": _exact_scales(case, seed, "v")}}
    s = prepare(case, seed)
    c = s["cache"]
    if kind == "select":
        return {"codes": None, "scale": _exact_bound_scales(s), "sel": None}
    g, n_q, d = case["hq"] // case["hkv"], case["n_q"], c["d"]
    out = torch.zeros((c["b"], case["hq"], n_q, d), device="cuda", dtype=torch.float64)
    for b, size in enumerate(s["lens"]):
        rows = torch.arange(n_q, device="cuda")
        last = size - n_q + rows if case["causal"] else torch.full_like(rows, size - 1)
        t = torch.arange(size, device="cuda")
        for h in range(c["h"]):
            k, v = (_rows64(c, p, b, h, t) for p in ("k", "v"))
            seen = t[None] <= last[:, None]
            if kind == "sparse":
                listed_blocks = torch.zeros((n_q, (size + TOKENS - 1) // TOKENS + 1), device="cuda", dtype=torch.bool)
                listed_blocks.scatter_(1, s["sel"][b, h].long() % listed_blocks.shape[1], True)     # -1 falls into the last column
                seen &= listed_blocks[:, :-1].repeat_interleave(TOKENS, 1)[:, :size]
            for head in range(h * g, (h + 1) * g):
                x = (s["q"][b, head].double() @ k.T) / math.sqrt(d)
                p = torch.softmax(x.masked_fill(~seen, -math.inf), -1).nan_to_num(0.0)
                out[b, head] = p @ v
    return out


def _rows64(c, name, b, h, t):
    page = c["table"][b].long()[t // c["page"]]
    row = t % c["page"]
    x, s = c[name]["payload"][page, h, row], c[name]["scale"]
    if c["layout"] in TOP:
        x = x.view(torch.float8_e4m3fn if c["layout"] == "e4m3_b64" else torch.int8).double()
        return x * s[page, h, row // TOKENS].double()[:, None]
    s = s[page, h, row].double().repeat_interleave(32, -1)
    if c["layout"] == "q8_0":
        return x.view(torch.int8).double() * s
    y = torch.empty_like(s)
    y[:, 0::2], y[:, 1::2] = (x % 16).double(), (x // 16).double()
    return torch.where(y > 7, y - 16, y) * s


def _exact_bound_scales(s):
    c, case = s["cache"], s["case"]
    out = s["scale"].double().clone()
    for b, size in enumerate(s["lens"]):
        first = max(0, size - case["fresh"]) // TOKENS * TOKENS
        t = torch.arange(first, size, device="cuda")
        for h in range(c["h"]):
            top = _rows64(c, "k", b, h, t).abs().amax(1)
            top = torch.nn.functional.pad(top, (0, -size % TOKENS)).view(-1, TOKENS).amax(1) / 127.0
            t0 = t[::TOKENS]
            out[c["table"][b].long()[t0 // c["page"]], h, t0 % c["page"] // TOKENS] = top
    return out


def _exact_scales(case, seed, name):
    """Scales of the blocks after one append, by their definition: one block and head after the other on the host."""
    s = prepare(case, seed)
    c, top = s["cache"], TOP[case["layout"]]
    scale = c[name]["scale"].double().cpu()
    if case["by_slots"]:
        x = s["kv"].view(-1, 2, c["h"], c["d"])[:, 0 if name == "k" else 1]
        slots = s["slots"].tolist()
    else:
        x = s[name + "_new"].transpose(1, 2).flatten(0, 1)
        first = s["positions"].tolist() if case["page"] else [s["pos0"]] * c["b"]
        table = c["table"].tolist()
        slots = [table[b][t // c["page"]] * c["page"] + t % c["page"] for b in range(c["b"]) for t in range(first[b], first[b] + case["hi"])]
    amax = x.double().abs().amax(-1).cpu().tolist()
    new = {}
    for slot, row in zip(slots, amax):
        block = slot // TOKENS
        begin, most = new.get(block, (slot % TOKENS, [0.0] * c["h"]))
        new[block] = (min(begin, slot % TOKENS), [max(a, b) for a, b in zip(most, row)])
    per = c["page"] // TOKENS
    for block, (begin, most) in new.items():
        for h in range(c["h"]):
            now, need = float(scale[block // per, h, block % per]) if begin else 0.0, most[h] / top
            while 0.0 < now < need:
                now *= 2.0
            scale[block // per, h, block % per] = now if now >= need else need
    return scale
