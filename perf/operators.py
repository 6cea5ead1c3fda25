"""The operators around a packed K/V cache that are measured here, each in its plain form (elementary
torch operations) and as a user's calls of the library:

  table    cos / sin table of the rotary positions, for scaled frequencies and far positions
  append   rotary positions applied to q and k, and the quantised append of the rotated k and of v
  weights  decode attention that also adds every token's attention weight to a running score
  select   the tokens a cache keeps: the highest running scores, with protected first and last ones
  compact  the kept tokens' packed rows moved together (inside the cache, or into a smaller one)

`listed()` and `draw()` give the cases, `prepare()` what a program holds before the call, `run()` one
call and its outputs, `work()` the bytes and operations it cannot do without, `exact()` the outputs
from the definition in 64 bits.
"""
import functools
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HADAMARD = ("had_int4", "had_int2")
LAYOUTS = ("q4_0", "q6_0", "q8_0", "asym4_g32") + HADAMARD


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a short table for a partly rotated head, remade when a program sets its context length
        {"name": "table 8K, 32 dims", "kind": "table", "rot": 32, "n_pos": 8192, "scaling": "none", "factor": 1.0},
        # the table of a 128K context, made once at start: frequencies scaled to four times the trained length
        {"name": "table 128K, 128 dims, yarn", "kind": "table", "rot": 128, "n_pos": 131072, "scaling": "yarn", "factor": 4.0},
        # the decode step of a serving batch: one new token for each of 64 sequences of a paged pool
        {"name": "append 1 token x 64, paged q4_0", "kind": "append", "layout": "q4_0", "batch": 64, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "interleaved": False, "n_new": 1, "cap": 2048, "page": 64, "dtype": "bf16", "n_recent": 0},
        # a prefill chunk of 255 rows into the Hadamard cache with its exact window
        {"name": "append 255 rows x 8, had_int4", "kind": "append", "layout": "had_int4", "batch": 8, "hq": 16, "hkv": 8, "d": 128,
         "rot": 128, "interleaved": False, "n_new": 255, "cap": 1024, "page": 0, "dtype": "f32", "n_recent": 64},
        # a whole prompt, 256-wide heads of which 64 dims are rotated in neighbouring pairs
        {"name": "append 8192 rows, asym4, d256", "kind": "append", "layout": "asym4_g32", "batch": 1, "hq": 16, "hkv": 8, "d": 256,
         "rot": 64, "interleaved": True, "n_new": 8192, "cap": 8192, "page": 0, "dtype": "f16", "n_recent": 0},
        # one decode step at 128K tokens with 64 query heads on 8 kv heads
        {"name": "weights 1 row, 128K, q4_0", "kind": "weights", "layout": "q4_0", "batch": 1, "hq": 64, "hkv": 8, "d": 128, "n_q": 1,
         "lo": 131072, "hi": 131072, "page": 0, "dtype": "bf16", "causal": False, "n_recent": 0, "decay": 1.0},
        # one decode step of a ragged serving batch
        {"name": "weights 1 row, ragged x 16, q8_0", "kind": "weights", "layout": "q8_0", "batch": 16, "hq": 32, "hkv": 8, "d": 128, "n_q": 1,
         "lo": 1021, "hi": 16379, "page": 64, "dtype": "bf16", "causal": False, "n_recent": 0, "decay": 0.95},
        # the last 32 rows of a prompt score the whole of it before the first eviction
        {"name": "weights 32 rows, 32K, had_int4", "kind": "weights", "layout": "had_int4", "batch": 1, "hq": 32, "hkv": 8, "d": 128, "n_q": 32,
         "lo": 32749, "hi": 32749, "page": 0, "dtype": "bf16", "causal": True, "n_recent": 64, "decay": 0.0},
        # a 128K cache cut to a quarter
        {"name": "select 32K of 128K", "kind": "select", "batch": 1, "hkv": 8, "lo": 131072, "hi": 131072, "keep": 32768, "sink": 4, "recent": 256},
        # a ragged batch cut to one budget; some sequences are shorter than it
        {"name": "select 1021 of up to 4099 x 32", "kind": "select", "batch": 32, "hkv": 8, "lo": 700, "hi": 4099, "keep": 1021, "sink": 4, "recent": 64},
        # after the prompt: the kept quarter moves into a cache of the decode budget's size
        {"name": "compact 128K to 32K, q4_0, new cache", "kind": "compact", "layout": "q4_0", "batch": 1, "hkv": 8, "d": 128,
         "lo": 131072, "hi": 131072, "keep": 32768, "page": 0, "n_recent": 0, "in_place": False},
        # during decoding: every sequence of a paged pool is cut in place
        {"name": "compact ragged x 16 in place, q8_0", "kind": "compact", "layout": "q8_0", "batch": 16, "hkv": 8, "d": 128,
         "lo": 3001, "hi": 8190, "keep": 2999, "page": 64, "n_recent": 0, "in_place": True},
    ]


def _log(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("table", "append", "append", "weights", "weights", "select", "compact", "compact"))
    if kind == "table":
        return {"kind": kind, "rot": 16 * rng.randint(1, 16), "n_pos": _log(rng, 1, 60000),
                "scaling": rng.choice(("none", "linear", "ntk", "banded", "yarn")), "factor": rng.choice((2.0, 4.0, 8.0))}
    hkv = rng.choice((1, 2, 4, 8))
    if kind == "select":
        batch, hi = _log(rng, 1, 32), _log(rng, 40, 30000)
        keep = rng.randint(8, hi)
        return {"kind": kind, "batch": batch, "hkv": hkv, "lo": rng.randint(1, hi), "hi": hi, "keep": keep,
                "sink": rng.randint(0, 4), "recent": rng.randint(0, keep - 4)}
    d = rng.choice((128, 128, 256))
    layout = rng.choice(LAYOUTS)
    page = rng.choice((0, 64, 128))
    n_recent = rng.choice((0, 32, 100)) if layout in HADAMARD else 0
    if kind == "append":
        n_new = rng.choice((1, 1, 2, _log(rng, 3, 1500)))
        batch = _log(rng, 1, 32 if n_new < 10 else 4)
        return {"kind": kind, "layout": layout, "batch": batch, "hq": hkv * rng.choice((1, 2, 4, 8)), "hkv": hkv, "d": d,
                "rot": 16 * rng.randint(1, d // 16), "interleaved": rng.random() < 0.5, "n_new": n_new,
                "cap": 64 * ((n_new + rng.randint(0, 500) + 63) // 64 + 1), "page": page, "dtype": rng.choice(tuple(DTYPES)), "n_recent": n_recent}
    batch, hi = _log(rng, 1, 8), _log(rng, 130, 8000)
    lo = rng.randint(129, hi) if page else hi
    if kind == "weights":
        n_q = rng.choice((1, 1, 1, 2, _log(rng, 3, 48)))
        return {"kind": kind, "layout": layout, "batch": batch, "hq": hkv * rng.choice((1, 2, 4, 8)), "hkv": hkv, "d": d, "n_q": n_q,
                "lo": lo, "hi": hi, "page": page, "dtype": rng.choice(tuple(DTYPES)), "causal": n_q > 1, "n_recent": n_recent,
                "decay": rng.choice((0.0, 0.9, 1.0))}
    return {"kind": kind, "layout": layout, "batch": batch, "hkv": hkv, "d": d, "lo": lo, "hi": hi, "keep": rng.randint(110, hi - 1),
            "page": page, "n_recent": n_recent, "in_place": bool(page) or rng.random() < 0.5}


# ------------------------------------------------------------------------------- the packed layouts
def _row_bytes(layout, d):
    return {"q4_0": d // 2, "q6_0": 3 * d // 4, "q8_0": d, "asym4_g32": d // 2, "had_int4": d // 2, "had_int2": d // 4}[layout]


def _fields(bits, u):
    """Unsigned fields of `bits` bits, the first in a byte's lowest bits."""
    n = 8 // bits
    u = u.reshape(u.shape[:-1] + (-1, n)) << torch.arange(0, 8, bits, device=u.device, dtype=torch.int32)
    return u.sum(-1).to(torch.uint8)


def _unfields(bits, b):
    u = b.to(torch.int32).unsqueeze(-1) >> torch.arange(0, 8, bits, device=b.device, dtype=torch.int32)
    return (u & (2 ** bits - 1)).flatten(-2)


def _butterfly(y, h):
    s = y.shape
    y = y.reshape(s[:-1] + (s[-1] // (2 * h), 2, h))
    a, b = y[..., 0, :], y[..., 1, :]
    return torch.stack((a + b, a - b), -2).reshape(s)


def _rotate(x):
    """The orthonormal Hadamard rotation in float32, one rounded operation at a time."""
    d = x.shape[-1]
    steps = [2 ** k for k in range(int(math.log2(d)))]
    return functools.reduce(_butterfly, steps, x) * float(np.float32(1.0 / math.sqrt(d)))


def _codes(x, s, lo, hi):
    """rint(x / s) in [lo, hi], 0 where the scale is 0 (divisions by tensors: correctly rounded)."""
    return torch.where(s > 0, torch.round(x / torch.where(s > 0, s, 1.0)).clamp(lo, hi), 0.0).to(torch.int32)


def _half(x):
    return x.clamp(-65504.0, 65504.0).half()


def _pack(layout, x):
    """float32 rows [..., D] -> (payload, scale, zero or None, rotated rows or None) of a layout."""
    d = x.shape[-1]
    if layout in HADAMARD:
        y, top = _rotate(x), 7.0 if layout == "had_int4" else 1.0
        amax = y.abs().amax(-1, keepdim=True)
        s = amax / torch.full_like(amax, top)
        bits = 4 if layout == "had_int4" else 2
        return _fields(bits, _codes(y, s, -top, top) & (2 ** bits - 1)), s[..., 0], None, y
    b = x.reshape(x.shape[:-1] + (d // 32, 32))
    if layout == "asym4_g32":
        lo, hi = b.amin(-1, keepdim=True), b.amax(-1, keepdim=True)
        span = hi - lo
        s, z = _half(span / torch.full_like(span, 15.0)), _half(lo)
        return _fields(4, _codes(b - z.float(), s.float(), 0, 15)).flatten(-2), s[..., 0], z[..., 0], None
    top = {"q4_0": 8, "q6_0": 32, "q8_0": 128}[layout]
    s = _half(b.abs().amax(-1, keepdim=True) / float(top))            # a power of two: the reciprocal is exact
    c = _codes(b, s.float(), -top, top - 1)
    if layout == "q4_0":
        p = _fields(4, c & 15)
    elif layout == "q6_0":
        p = torch.cat((_fields(4, c & 15), _fields(2, (c >> 4) & 3)), -1)
    else:
        p = (c & 255).to(torch.uint8)
    return p.flatten(-2), s[..., 0], None, None


def _signed(u, bits):
    return ((u ^ (1 << (bits - 1))) - (1 << (bits - 1))).float()


def _unpack(layout, payload, scale, zero, d, to=torch.float32):
    """The values a plane's rows stand for (Hadamard layouts: in the rotated basis)."""
    if layout == "had_int4" or layout == "had_int2":
        bits = 4 if layout == "had_int4" else 2
        return _signed(_unfields(bits, payload), bits).to(to) * scale.to(to).unsqueeze(-1)
    p = payload.reshape(payload.shape[:-1] + (d // 32, -1))
    if layout == "asym4_g32":
        v = _unfields(4, p).to(to) * scale.to(to).unsqueeze(-1) + zero.to(to).unsqueeze(-1)
    elif layout == "q4_0":
        v = _signed(_unfields(4, p), 4).to(to) * scale.to(to).unsqueeze(-1)
    elif layout == "q6_0":
        v = _signed(_unfields(4, p[..., :16]) | (_unfields(2, p[..., 16:]) << 4), 6).to(to) * scale.to(to).unsqueeze(-1)
    else:
        v = _signed(p.to(torch.int32), 8).to(to) * scale.to(to).unsqueeze(-1)
    return v.flatten(-2)


# ------------------------------------------------------------------------------------------ prepare
def _lens(case):
    """The batch's lengths: spread evenly over the case's range, so that the work is the case's own."""
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    return [hi - (hi - lo) * i // max(1, b - 1) for i in range(b)]


def _planes(case, rows, gen, lead):
    """One plane's tensors for token rows of lead + (D,), a few channels far larger than the rest."""
    d, layout = case["d"], case["layout"]
    x = torch.randn(rows + (d,), device="cuda", generator=gen)
    x[..., torch.randperm(d, device="cuda", generator=gen)[:4]] *= 6.0
    payload, scale, zero, _ = _pack(layout, x)
    p = {"payload": payload.reshape(lead + (-1,)), "scale": scale.reshape(lead + ((d // 32,) if layout not in HADAMARD else ()))}
    if zero is not None:
        p["zero"] = zero.reshape(lead + (-1,))
    if case["n_recent"]:
        p["recent"] = torch.randn((case["batch"], case["hkv"], case["n_recent"], d), device="cuda", generator=gen)
    return p


def _make_cache(case, cap, gen):
    """The cache's planes as tensors: contiguous [B][H][cap], or a pool of pages with a shuffled table."""
    b, h, page = case["batch"], case["hkv"], case.get("page", 0)
    c = {"layout": case["layout"], "b": b, "h": h, "d": case["d"], "cap": cap, "page": page, "n_recent": case["n_recent"]}
    if page:
        per = (cap + page - 1) // page
        c["cap"] = per * page
        c["table"] = torch.randperm(b * per, device="cuda", generator=gen).to(torch.int32).reshape(b, per)
        lead = (b * per, h, page)
    else:
        lead = (b, h, cap)
    c["k"], c["v"] = _planes(case, lead, gen, lead), _planes(case, lead, gen, lead)
    if own:
        c["handle"] = _handle(c)
    return c


def _handle(c):
    """The library's cache object for the same planes."""
    import sub_byte_quantized_gb300 as kvq
    if c["page"]:
        h = kvq.PagedKVCache(c["layout"], c["b"], c["h"], c["d"], c["page"], c["table"].numel(), c["table"].shape[1], n_recent=c["n_recent"])
        h.set_block_table(c["table"])
    else:
        h = kvq.KVCache(c["layout"], c["b"], c["h"], c["d"], c["cap"], n_recent=c["n_recent"])
    for t in ("k", "v"):
        for name, x in c[t].items():
            h.planes[t][name].copy_(x)
        c[t] = h.planes[t]
    return h


def _frequencies(rot, base, scaling, factor, length):
    """Rotary frequencies in 64 bits, and the magnitude of the table, for the scalings the library has."""
    i = np.arange(0, rot, 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f, mag = base ** (-i / rot), 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "banded":                       # long wavelengths divided, short ones kept, a ramp between
        turns = length * f / (2 * math.pi)          # turns within the trained length
        keep = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        f = f * keep + f / factor * (1 - keep)
    elif scaling == "yarn":
        at = [rot * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        lo, hi = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
        ramp = np.clip((np.arange(rot // 2) - lo) / (hi - lo if hi != lo else 0.001), 0.0, 1.0)
        f, mag = f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, mag


def _table(freq, mag, pos0, n_pos):
    """cos then sin of every position's angles, formed in 64 bits and rounded once."""
    a = torch.arange(pos0, pos0 + n_pos, device="cuda", dtype=torch.float64)[:, None] * torch.as_tensor(freq, device="cuda")
    return torch.cat((a.cos() * mag, a.sin() * mag), 1).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind = case["kind"]
    s = {"case": case, "kind": kind}
    if kind == "table":
        s["base"], s["pos0"] = 10000.0 + 17.0 * (seed % 1009), seed % 4099
        return s
    b, h = case["batch"], case["hkv"]
    if kind == "append":
        n, d = case["n_new"], case["d"]
        s["cache"] = _make_cache(case, case["cap"], gen)
        # the projection's output, token-major: q, k and v heads side by side
        s["qkv"] = torch.randn((b, n, (case["hq"] + 2 * h) * d), device="cuda", generator=gen).to(DTYPES[case["dtype"]])
        freq, mag = _frequencies(case["rot"], 500000.0, "none", 1.0, 0)
        s["table"] = _table(freq, mag, 0, 4 * case["cap"])
        # the cache has been cut before: positions run ahead of the slots
        room = case["cap"] - n
        s["pos0"] = seed % (room + 1)
        s["slots"] = torch.randint(0, room + 1, (b,), device="cuda", generator=gen, dtype=torch.int32)
        first = torch.randint(room, 3 * case["cap"], (b, 1), device="cuda", generator=gen, dtype=torch.int32)
        s["positions"] = (first + torch.arange(n, device="cuda", dtype=torch.int32)).contiguous()
        return s
    s["lens"] = _lens(case)
    s["seq_lens"] = torch.tensor(s["lens"], device="cuda", dtype=torch.int32)
    cap = max(s["lens"])
    # running scores: attention mass is spread over orders of magnitude; a part has none at all
    s["scores"] = torch.randn((b, h, cap), device="cuda", generator=gen).mul_(2.5).exp_().mul_(1e-4)
    s["scores"][torch.rand((b, h, cap), device="cuda", generator=gen) < 0.1] = 0.0
    if kind == "select":
        return s
    s["cache"] = _make_cache(case, cap, gen)
    if kind == "weights":
        s["q"] = torch.randn((b, case["hq"], case["n_q"], case["d"]), device="cuda", generator=gen).to(DTYPES[case["dtype"]])
        s["scores_out"] = torch.zeros_like(s["scores"])
        return s
    s["keep"] = _select(s["scores"], s["lens"], s["seq_lens"], case["keep"], 4, max(32, case["n_recent"]))
    if not case["in_place"]:
        s["dst"] = _make_cache(dict(case, page=0), case["keep"], gen)
        s["scores_out"] = torch.zeros((b, h, case["keep"]), device="cuda")
    return s


# ---------------------------------------------------------------------------------- the plain forms
def _apply_rope(x, cs, rot, interleaved):
    """x [B][H][n][D] rotated by the table rows cs [B][1][n][rot] (cos, then sin), in float32."""
    h = rot // 2
    c, s = cs[..., :h], cs[..., h:]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        r = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h:rot]
        r = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((r, x[..., rot:]), -1)


def _heads(s):
    """The q, k and v views [B][heads][n][D] of the projection's output."""
    case, x = s["case"], s["qkv"]
    x = x.view(x.shape[0], x.shape[1], -1, case["d"]).transpose(1, 2)
    hq, h = case["hq"], case["hkv"]
    return x[:, :hq], x[:, hq:hq + h], x[:, hq + h:]


def _where(c, t):
    """Indexes of the logical token rows t [B][n] in the planes: [B][H][n] each."""
    b, h = torch.arange(c["b"], device="cuda"), torch.arange(c["h"], device="cuda")[None, :, None]
    if not c["page"]:
        return b[:, None, None], h, t[:, None, :]
    pages = torch.gather(c["table"].long(), 1, t // c["page"])
    return pages[:, None, :], h, (t % c["page"])[:, None, :]


def _plain_append(s):
    case, c = s["case"], s["cache"]
    q, k, v = (x.float() for x in _heads(s))
    cs = s["table"][s["positions"].long()][:, None]
    q, k = (_apply_rope(x, cs, case["rot"], case["interleaved"]) for x in (q, k))
    n = case["n_new"]
    first = s["slots"].long()[:, None] if c["page"] else torch.full((c["b"], 1), s["pos0"], device="cuda", dtype=torch.int64)
    t = first + torch.arange(n, device="cuda")
    _put(c["k"], c, t, k)
    _put(c["v"], c, t, v)
    return {"q": q.to(DTYPES[case["dtype"]]), "k": c["k"], "v": c["v"]}


def _put(plane, c, t, x):
    at = _where(c, t)
    payload, scale, zero, y = _pack(c["layout"], x)
    plane["payload"][at], plane["scale"][at] = payload, scale
    if zero is not None:
        plane["zero"][at] = zero
    if c["n_recent"]:                               # the exact window holds the newest rows, slot = position mod its size
        m = min(x.shape[2], c["n_recent"])
        b, h = torch.arange(c["b"], device="cuda")[:, None, None], torch.arange(c["h"], device="cuda")[None, :, None]
        plane["recent"][b, h, (t[:, -m:] % c["n_recent"])[:, None, :]] = y[:, :, -m:]


def _rows(plane, c, n, name):
    """A plane's rows of the logical tokens [0, n): [B][H][n][...]."""
    x = plane[name]
    if not c["page"]:
        return x[:, :, :n]
    x = x[c["table"][:, :(n + c["page"] - 1) // c["page"]].long()].transpose(1, 2).flatten(2, 3)
    return x[:, :, :n]


def _values(plane, c, n, to=torch.float32):
    zero = _rows(plane, c, n, "zero") if "zero" in plane else None
    return _unpack(c["layout"], _rows(plane, c, n, "payload"), _rows(plane, c, n, "scale"), zero, c["d"], to)


def _visible(s, n):
    """[B][1][rows of a kv head][n]: the tokens each query row sees, and where its length ends."""
    case = s["case"]
    lens, t = s["seq_lens"].long()[:, None, None, None], torch.arange(n, device="cuda")
    if not case["causal"]:
        return (t < lens).expand(-1, 1, case["hq"] // case["hkv"] * case["n_q"], -1)
    i = torch.arange(case["n_q"], device="cuda").repeat(case["hq"] // case["hkv"])[:, None]
    return t <= lens - case["n_q"] + i


def _in_window(s, n):
    lens, t = s["seq_lens"].long()[:, None], torch.arange(n, device="cuda")
    return (t >= lens - s["cache"]["n_recent"]) & (t < lens)


def _plain_weights(s):
    case, c = s["case"], s["cache"]
    n, g = max(s["lens"]), case["hq"] // case["hkv"]
    q = s["q"].float().reshape(c["b"], c["h"], g * case["n_q"], c["d"])
    k, v = _values(c["k"], c, n), _values(c["v"], c, n)
    if c["layout"] in HADAMARD:
        q = _rotate(q)
        amax = q.abs().amax(-1, keepdim=True)
        sq = amax / torch.full_like(amax, 127.0)
        q8 = _codes(q, sq, -127, 127).float()
        bits = 4 if c["layout"] == "had_int4" else 2
        codes = _signed(_unfields(bits, _rows(c["k"], c, n, "payload")), bits)
        dots = (q8 @ codes.transpose(-1, -2)) * sq * _rows(c["k"], c, n, "scale")[:, :, None, :]
        if c["n_recent"]:
            slot = torch.arange(n, device="cuda") % c["n_recent"]
            win = _in_window(s, n)
            dots = torch.where(win[:, None, None, :], q @ c["k"]["recent"][:, :, slot].transpose(-1, -2), dots)
            v = torch.where(win[:, None, :, None], c["v"]["recent"][:, :, slot], v)
    else:
        dots = q @ k.transpose(-1, -2)
    x = torch.where(_visible(s, n), dots / math.sqrt(c["d"]), -math.inf)
    p = (x - x.amax(-1, keepdim=True)).exp()
    p = p / p.sum(-1, keepdim=True)
    out = p @ v
    if c["layout"] in HADAMARD:
        out = _rotate(out)
    got = p.sum(2) + (case["decay"] * s["scores"] if case["decay"] else 0.0)
    s["scores_out"].copy_(torch.where(torch.arange(n, device="cuda") < s["seq_lens"].long()[:, None, None], got, s["scores_out"]))
    return {"out": out.reshape(c["b"], case["hq"], case["n_q"], c["d"]), "scores": s["scores_out"]}


def _select(scores, lens, seq_lens, n_keep, sink, recent):
    """Ascending kept tokens [B][H][n_keep]: protected ones, then the highest scores, ties to the lowest
    index; sequences of at most n_keep tokens keep all, and -1 fills the rest."""
    n = max(lens)
    t, size = torch.arange(n, device="cuda"), seq_lens.long()[:, None, None]
    x = torch.nan_to_num(scores[..., :n], nan=-math.inf, posinf=math.inf, neginf=-math.inf)
    rank = torch.where(t < size, ((t < sink) | (t >= size - recent)).int(), -1).expand(x.shape)
    by = x.sort(dim=-1, descending=True, stable=True).indices
    by = by.gather(-1, rank.gather(-1, by).sort(dim=-1, descending=True, stable=True).indices)[..., :n_keep]
    by = torch.nn.functional.pad(by, (0, n_keep - by.shape[-1]), value=n)
    by = torch.where(by < size, by, n).sort(dim=-1).values
    return torch.where(by < size, by, -1).to(torch.int32)


def _plain_compact(s):
    case, c = s["case"], s["cache"]
    n, n_keep, keep = max(s["lens"]), case["keep"], s["keep"].long()
    new = s["seq_lens"].long().clamp(max=n_keep)[:, None, None]
    dst, out = s.get("dst", c), s.get("scores_out", s["scores"])
    b, h = torch.arange(c["b"], device="cuda")[:, None, None], torch.arange(c["h"], device="cuda")[None, :, None]
    src = keep.clamp(min=0)
    m = min(n_keep, n)
    to = _where(dst, torch.arange(m, device="cuda").expand(c["b"], -1))
    live = torch.arange(m, device="cuda") < new
    cut = s["seq_lens"].long()[:, None, None] - new
    _move(c, dst, "k", n, b, h, src[..., :m], to, live, cut)
    _move(c, dst, "v", n, b, h, src[..., :m], to, live, cut)
    got = torch.zeros_like(out)
    got[..., :m] = torch.where(live, s["scores"][b, h, src[..., :m]], 0.0)
    got[..., n:] = out[..., n:]
    out.copy_(got)
    return {"k": dst["k"], "v": dst["v"], "scores": out}


def _move(c, dst, name, n, b, h, src, to, live, cut):
    a, z, r = c[name], dst[name], c["n_recent"]
    x = _rows(a, c, n, "payload")[b, h, src]
    z["payload"][to] = torch.where(live[..., None], x, z["payload"][to])
    x = _rows(a, c, n, "scale")[b, h, src]
    z["scale"][to] = torch.where(live if x.dim() == 3 else live[..., None], x, z["scale"][to])
    if "zero" in a:
        x = _rows(a, c, n, "zero")[b, h, src]
        z["zero"][to] = torch.where(live[..., None], x, z["zero"][to])
    if r:                                           # a window row's slot is its token's index mod the window's size
        z["recent"].copy_(a["recent"][b, h, (torch.arange(r, device="cuda") + cut) % r])


# ------------------------------------------------------------------------------------------- one call
def run(s):
    case, kind = s["case"], s["kind"]
    if own:
        return _own(s, case, kind)
    if kind == "table":
        freq, mag = _frequencies(case["rot"], s["base"], case["scaling"], case["factor"], 32768)
        return _table(freq, mag, s["pos0"], case["n_pos"])
    if kind == "append":
        return _plain_append(s)
    if kind == "weights":
        return _plain_weights(s)
    if kind == "select":
        return _select(s["scores"], s["lens"], s["seq_lens"], case["keep"], *_protected(case))
    return _plain_compact(s)


def _protected(case):
    return min(case["sink"], case["keep"]), min(case["recent"], case["keep"] - min(case["sink"], case["keep"]))


def _own(s, case, kind):
    import sub_byte_quantized_gb300 as kvq
    if kind == "table":
        freq, mag = kvq.rope_frequencies(case["rot"], s["base"], case["scaling"], case["factor"], 32768)
        return kvq.rope_table(freq, case["n_pos"], pos0=s["pos0"], magnitude=mag)
    if kind == "select":
        sink, recent = _protected(case)
        return kvq.evict_select(s["scores"], max(s["lens"]), case["keep"], n_sink=sink, n_recent=recent, seq_lens=s["seq_lens"])
    c = s["cache"]
    cache = c["handle"]
    if kind == "append":
        q, k, v = _heads(s)
        if c["page"]:
            q = kvq.paged_rope_store(cache, s["table"], k, v, s["slots"], q=q, positions=s["positions"], interleaved=case["interleaved"])
        else:
            q = kvq.rope_store(cache, s["table"], k, v, s["pos0"], q=q, positions=s["positions"], interleaved=case["interleaved"])
        return {"q": q, "k": c["k"], "v": c["v"]}
    n = max(s["lens"])
    if kind == "weights":
        if c["page"]:
            out, scores = kvq.paged_decode_attend_weights(cache, s["q"], s["seq_lens"], n, s["scores"], scores_out=s["scores_out"],
                                                          decay=case["decay"], causal=case["causal"])
        else:
            out, scores = kvq.decode_attend_weights(cache, s["q"], n, s["scores"], scores_out=s["scores_out"], decay=case["decay"],
                                                    causal=case["causal"], q_pos0=n - case["n_q"] if case["causal"] else 0)
        return {"out": out, "scores": scores}
    if c["page"]:
        kvq.paged_evict_compact(cache, s["keep"], s["seq_lens"], n, scores=s["scores"])
        return {"k": c["k"], "v": c["v"], "scores": s["scores"]}
    if case["in_place"]:
        kvq.evict_compact(cache, s["keep"], n, scores=s["scores"])
        return {"k": c["k"], "v": c["v"], "scores": s["scores"]}
    dst = s["dst"]
    kvq.evict_compact(cache, s["keep"], n, dst=dst["handle"], scores=s["scores"], scores_out=s["scores_out"])
    return {"k": dst["k"], "v": dst["v"], "scores": s["scores_out"]}


# ------------------------------------------------------------------------------------------- the work
def _token_bytes(layout, d):
    """Bytes of one token of one head in one plane: codes, scales and zero-points."""
    return _row_bytes(layout, d) + (4 if layout in HADAMARD else d // 16 * (2 if layout == "asym4_g32" else 1))


def work(case):
    kind = case["kind"]
    if kind == "table":                             # the table written; an angle, its sine and its cosine
        e = case["n_pos"] * case["rot"]
        return {"bytes": 4 * e, "flops": 20 * e}
    b, h = case["batch"], case["hkv"]
    if kind == "append":                            # q, k, v read, q written, k and v written packed, the table's rows
        size = 4 if case["dtype"] == "f32" else 2
        rows, d = b * case["n_new"], case["d"]
        per = 2 * case["hq"] * d * size + 2 * h * (d * size + _token_bytes(case["layout"], d)) + 4 * case["rot"]
        ring = 2 * b * h * min(case["n_new"], case["n_recent"]) * d * 4
        return {"bytes": rows * per + ring, "flops": rows * (3 * (case["hq"] + h) * case["rot"] + 2 * h * d * (4 if case["layout"] not in HADAMARD else 11))}
    total = sum(_lens(case))
    if kind == "weights":                           # both planes once, the scores in and out, q and out
        d, rows = case["d"], case["hq"] * case["n_q"]
        win = sum(min(x, case["n_recent"]) for x in _lens(case))
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * h * ((total - win) * _token_bytes(case["layout"], d) + win * d * 4) + total * h * (8 if case["decay"] else 4)
                + b * rows * d * (4 + size), "flops": 4 * total * rows * d}
    if kind == "select":                            # the scores read, the list written
        return {"bytes": 4 * h * (total + b * case["keep"]), "flops": h * total}
    kept = sum(min(x, case["keep"]) for x in _lens(case))
    moved = 2 * 2 * kept * h * _token_bytes(case["layout"], case["d"])
    ring = 2 * 2 * b * h * case["n_recent"] * case["d"] * 4
    return {"bytes": moved + ring + h * (4 * total + 4 * kept + 4 * b * case["keep"]), "flops": 0}


# ------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "table":
        freq, mag = _frequencies(case["rot"], s["base"], case["scaling"], case["factor"], 32768)
        angle = np.outer(np.arange(s["pos0"], s["pos0"] + case["n_pos"], dtype=np.float64), freq)
        return np.concatenate((np.cos(angle), np.sin(angle)), 1) * mag
    if kind == "append":                            # codes and scales are bits by definition: no value in 64 bits
        q = _heads(s)[0].double()
        at = s["table"].double()[s["positions"].long()]
        half = case["rot"] // 2
        i = torch.arange(half, device="cuda")
        first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        z = torch.complex(q[..., first], q[..., second]) * torch.complex(at[:, None, :, :half], at[:, None, :, half:])
        q[..., first], q[..., second] = z.real, z.imag
        planes = {n: None for n in ("payload", "scale", "zero", "recent")}
        return {"q": q, "k": dict(planes), "v": dict(planes)}
    if kind == "weights":
        return _exact_weights(s)
    if kind == "select":
        return None
    return {"k": None, "v": None, "scores": _exact_scores(s)}


def _exact_scores(s):
    out, n = s.get("scores_out", s["scores"]).double().cpu().numpy().copy(), max(s["lens"])
    old, keep = s["scores"].double().cpu().numpy(), s["keep"].cpu().numpy()
    for b, size in enumerate(s["lens"]):
        m = min(size, s["case"]["keep"])
        for h in range(out.shape[1]):
            out[b, h, :n] = 0.0
            out[b, h, :m] = old[b, h, keep[b, h, :m]]
    return out


def _exact_weights(s):
    """One sequence and kv head at a time; the Hadamard query's 8-bit codes are bits by definition and
    come from float32 steps, everything after them is in 64 bits."""
    case, c = s["case"], s["cache"]
    g, d, n_q, had = case["hq"] // case["hkv"], c["d"], case["n_q"], c["layout"] in HADAMARD
    out = torch.zeros((c["b"], case["hq"], n_q, d), device="cuda", dtype=torch.float64)
    scores = s["scores_out"].double()
    basis = None
    if had:
        m = torch.ones((1, 1), dtype=torch.float64, device="cuda")
        while m.shape[0] < d:
            m = torch.cat((torch.cat((m, m), 1), torch.cat((m, -m), 1)), 0)
        basis = m / math.sqrt(d)
    for b, size in enumerate(s["lens"]):
        t = torch.arange(size, device="cuda")
        for h in range(c["h"]):
            rows = {}
            for name in ("k", "v"):
                p = c[name]
                at = (c["table"][b].long()[t // c["page"]], h, t % c["page"]) if c["page"] else (b, h, t)
                rows[name] = _unpack(c["layout"], p["payload"][at], p["scale"][at], p["zero"][at] if "zero" in p else None, d, torch.float64)
            q = s["q"][b, h * g:(h + 1) * g].reshape(g * n_q, d)
            x = q.double()
            if had:
                y = _rotate(q.float())
                top = y.abs().amax(-1, keepdim=True)
                step = top / torch.full_like(top, 127.0)
                x = _codes(y, step, -127, 127).double() * step.double()
            dots = x @ rows["k"].T
            if c["n_recent"]:
                w = min(c["n_recent"], size)
                slot = t[-w:] % c["n_recent"]
                dots[:, -w:] = (q.double() @ basis) @ c["k"]["recent"][b, h, slot].double().T
                rows["v"][-w:] = c["v"]["recent"][b, h, slot].double()
            dots = dots / math.sqrt(d)
            if case["causal"]:
                row = torch.arange(g * n_q, device="cuda") % n_q
                dots.masked_fill_(t[None] > (size - n_q + row)[:, None], -math.inf)
            p = torch.softmax(dots, -1)
            o = p @ rows["v"]
            out[b, h * g:(h + 1) * g] = (o @ basis if had else o).reshape(g, n_q, d)
            scores[b, h, :size] = p.sum(0) + (case["decay"] * s["scores"][b, h, :size].double() if case["decay"] else 0.0)
    return {"out": out, "scores": scores}
