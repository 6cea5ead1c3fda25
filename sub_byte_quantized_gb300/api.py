"""Thin torch-facing wrappers over the C ABI: they check tensor placement/shape, pass raw
pointers and the current CUDA stream, and nothing else. Every computation runs in libkvq.so.

torch is used for device memory (cache planes, workspace) and streams only. A call given a `stream` makes the
buffers that the caller leaves to it (workspace, outputs) on that stream; a caller that reads such an output on
the current stream orders the two, and may then drop it like any tensor of that stream.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import math
from typing import NamedTuple

import torch

from . import _lib as L

_DTYPES = {torch.float32: L.KVQ_F32, torch.bfloat16: L.KVQ_BF16, torch.float16: L.KVQ_F16}
_STORE_FN = {L.KVQ_Q4_0: "kvq_store_q4_0", L.KVQ_Q6_0: "kvq_store_q6_0",
             L.KVQ_HAD_INT4: "kvq_store_hadamard_int4", L.KVQ_ASYM4_G32: "kvq_store_asym4_g32",
             L.KVQ_Q8_0: "kvq_store_q8_0", L.KVQ_HAD_INT2: "kvq_store_hadamard_int2"}


def _layout_id(layout) -> int:
    """Layout value of a name ("q4_0", or "k+v" such as "q4_0+q8_0" for mixed K/V precision) or id."""
    if isinstance(layout, str):
        k, _, v = layout.partition("+")
        return L.mixed(L.LAYOUT_IDS[k], L.LAYOUT_IDS[v]) if v and v != k else L.LAYOUT_IDS[k]
    return int(layout)


def _plane_tensors(layout: int, lead: tuple, head_dim: int, dev, n_recent: int, ring_lead: tuple) -> dict:
    """Zeroed device planes of one of K or V in a plain layout: payload, scale [, zero] [, recent]."""
    rb = row_bytes(layout, head_dim)
    nb = head_dim // 32
    pl = {"payload": torch.zeros(lead + (rb,), dtype=torch.uint8, device=dev)}
    if layout in L.HADAMARD_IDS:
        pl["scale"] = torch.zeros(lead, dtype=torch.float32, device=dev)
        if n_recent:
            pl["recent"] = torch.zeros(ring_lead + (n_recent, head_dim), dtype=torch.float32, device=dev)
    elif layout in L.BLOCK_IDS:
        pl["scale"] = torch.zeros(lead[:-1] + (lead[-1] // 64,), dtype=torch.float32, device=dev)
    else:
        pl["scale"] = torch.zeros(lead + (nb,), dtype=torch.float16, device=dev)
        if layout == L.KVQ_ASYM4_G32:
            pl["zero"] = torch.zeros(lead + (nb,), dtype=torch.float16, device=dev)
    return pl


def _plane_read_bytes(layout: int, head_dim: int, n_tokens: int, n_recent: int) -> int:
    """Packed bytes one plane of one (batch, kv head) reads over n_tokens tokens."""
    per_tok = row_bytes(layout, head_dim)
    if layout in L.HADAMARD_IDS:
        n_w = min(n_recent, n_tokens)
        return (n_tokens - n_w) * (per_tok + 4) + n_w * head_dim * 4
    if layout in L.BLOCK_IDS:
        return n_tokens * per_tok + (n_tokens + 63) // 64 * 4
    return n_tokens * (per_tok + 2 * (head_dim // 32) * (2 if layout == L.KVQ_ASYM4_G32 else 1))


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


_DEVICE, _RAW_STREAM = (getattr(torch._C, n, None) for n in ("_cuda_getDevice", "_cuda_getCurrentRawStream"))


def _stream(stream) -> int | None:
    if stream is None:
        return _RAW_STREAM(_DEVICE())
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


_CURRENT = contextlib.nullcontext()


def _made_on(stream):
    """Context in which a call makes its own buffers: the stream it launches on. The allocator orders a buffer's
    memory by the stream that it was made on, so one made on the current stream could still be in use there when
    another stream's kernels write it, and a workspace, dropped on return, be handed out again while they run."""
    if stream is None:
        return _CURRENT
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream)))


def _output(stream, shape, dtype, device) -> torch.Tensor:
    """A buffer for a call's output, made on its stream. The caller reads it on the current stream as a rule and may
    drop it there while that is still to come: its memory waits for both."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _made_on(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _workspace(stream, nbytes: int, device) -> torch.Tensor:
    """A call's workspace, made on its stream."""
    if stream is None:
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    with _made_on(stream):
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _sized(cache, fn, *args) -> int:
    """fn(cache, *args), a workspace's bytes, remembered with the cache: a decode loop asks for the same again and again."""
    known = cache.__dict__.setdefault("_sizes", {})
    key = (fn, _DEVICE(), *args)
    n = known.get(key)
    if n is None:
        if len(known) >= 256:
            known.clear()
        n = known[key] = fn(cache, *args)
    return n


def _need_cuda(name: str, t: torch.Tensor) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def row_bytes(layout, head_dim: int) -> int:
    return int(L.lib().kvq_row_bytes(_layout_id(layout), head_dim))


def cache_plane_bytes(layout, batch, n_kv_heads, head_dim, capacity, n_recent=0) -> dict:
    out = (C.c_size_t * 4)()
    L.check(L.lib().kvq_cache_bytes(_layout_id(layout), batch, n_kv_heads, head_dim, capacity, n_recent, out),
            "kvq_cache_bytes")
    return {"payload": out[0], "scale": out[1], "zero": out[2], "recent": out[3]}


class KVCache:
    """Device planes of one layer's packed cache plus the C struct describing them.

    Planes (K and V each): payload u8 [B][H_kv][cap][row_bytes]; scale f16 [B][H_kv][cap][D/32]
    (f32 [B][H_kv][cap] for had_int4 / had_int2, f32 [B][H_kv][cap/64] for int8_b64 / e4m3_b64); zero f16 (asym4_g32); recent f32 [B][H_kv][n_recent][D]
    (the Hadamard layouts with n_recent > 0).
    """

    def __init__(self, layout, batch: int, n_kv_heads: int, head_dim: int, capacity: int, n_recent: int = 0,
                 device="cuda"):
        self.layout = _layout_id(layout)
        self.plane_layouts = dict(zip(("k", "v"), L.plane_ids(self.layout)))
        self.batch, self.n_kv_heads, self.head_dim, self.capacity = batch, n_kv_heads, head_dim, capacity
        self.n_recent = n_recent if self.plane_layouts["k"] in L.HADAMARD_IDS else 0
        dev = torch.device(device)
        shp = (batch, n_kv_heads, capacity)
        self.planes = {}
        for t in ("k", "v"):
            lt = self.plane_layouts[t]
            sizes = cache_plane_bytes(lt, batch, n_kv_heads, head_dim, capacity, self.n_recent)
            pl = _plane_tensors(lt, shp, head_dim, dev, self.n_recent, (batch, n_kv_heads))
            assert pl["payload"].numel() == sizes["payload"]
            self.planes[t] = pl
        self.struct = L.KvqCache(
            self.layout, batch, n_kv_heads, head_dim, capacity, self.n_recent,
            _ptr(self.planes["k"]["payload"]), _ptr(self.planes["v"]["payload"]),
            _ptr(self.planes["k"]["scale"]), _ptr(self.planes["v"]["scale"]),
            _ptr(self.planes["k"].get("zero")), _ptr(self.planes["v"].get("zero")),
            _ptr(self.planes["k"].get("recent")), _ptr(self.planes["v"].get("recent")))

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for pl in self.planes.values() for t in pl.values())

    def read_bytes(self, kv_len: int) -> int:
        """Packed bytes (payload + scales [+ zeros] [+ window]) one attention call reads."""
        return self.batch * self.n_kv_heads * sum(
            _plane_read_bytes(self.plane_layouts[t], self.head_dim, kv_len, self.n_recent) for t in ("k", "v"))


def store(cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor, pos0: int, stream=None) -> None:
    """Append k_new/v_new [B][H_kv][n_new][D] at positions [pos0, pos0 + n_new)."""
    _need_cuda("k_new", k_new)
    _need_cuda("v_new", v_new)
    if k_new.shape != v_new.shape or k_new.dtype != v_new.dtype:
        raise ValueError("k_new and v_new must have the same shape and dtype")
    B, H, n_new, D = k_new.shape
    if (B, H, D) != (cache.batch, cache.n_kv_heads, cache.head_dim):
        raise ValueError("k_new shape does not match the cache")
    name = _STORE_FN.get(cache.layout, "kvq_store")       # mixed K/V layouts: the generic store
    fn = getattr(L.lib(), name)
    L.check(fn(C.byref(cache.struct), k_new.data_ptr(), v_new.data_ptr(), _DTYPES[k_new.dtype], n_new, pos0,
               _stream(stream)), name)


def attend_workspace_bytes(cache: KVCache, n_q_heads: int, n_q: int, kv_len: int, chunk: int = 0) -> int:
    return int(L.lib().kvq_attend_workspace_bytes(C.byref(cache.struct), n_q_heads, n_q, kv_len, chunk))


def attend_chunk(cache: KVCache, n_q_heads: int, n_q: int, kv_len: int, chunk: int = 0) -> int:
    """The split-K chunk length a decode_attend call with these arguments uses (0 -> automatic)."""
    return int(L.lib().kvq_attend_chunk(C.byref(cache.struct), n_q_heads, n_q, kv_len, chunk))


def decode_attend(cache: KVCache, q: torch.Tensor, kv_len: int, causal: bool = False, q_pos0: int = 0,
                  attn_scale: float | None = None, chunk: int = 0, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Split-K attention of q [B][H_q][n_q][D] over the first kv_len cached tokens -> f32 out."""
    _need_cuda("q", q)
    B, Hq, n_q, D = q.shape
    if B != cache.batch or D != cache.head_dim:
        raise ValueError("q shape does not match the cache")
    if attn_scale is None:
        attn_scale = 1.0 / math.sqrt(D)
    if out is None:
        out = _output(stream, (B, Hq, n_q, D), torch.float32, q.device)
    _need_cuda("out", out)
    if workspace is None:
        workspace = _workspace(stream, _sized(cache, attend_workspace_bytes, Hq, n_q, kv_len, chunk), q.device)
    _need_cuda("workspace", workspace)
    L.check(L.lib().kvq_decode_attend(C.byref(cache.struct), q.data_ptr(), _DTYPES[q.dtype], Hq, n_q, kv_len,
                                      int(bool(causal)), q_pos0, float(attn_scale), chunk, out.data_ptr(),
                                      workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                      _stream(stream)), "kvq_decode_attend")
    return out


def append_decode_attend(cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor, pos0: int, q: torch.Tensor,
                         kv_len: int, causal: bool = False, q_pos0: int = 0, attn_scale: float | None = None,
                         chunk: int = 0, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """store(cache, k_new, v_new, pos0) then decode_attend(cache, q, kv_len, ...) in one library
    call (same results; the attention work that does not read the appended rows overlaps the
    append)."""
    _need_cuda("k_new", k_new)
    _need_cuda("v_new", v_new)
    _need_cuda("q", q)
    if k_new.shape != v_new.shape or k_new.dtype != v_new.dtype:
        raise ValueError("k_new and v_new must have the same shape and dtype")
    Bk, H, n_new, Dk = k_new.shape
    B, Hq, n_q, D = q.shape
    if (Bk, H, Dk) != (cache.batch, cache.n_kv_heads, cache.head_dim) or B != cache.batch or D != cache.head_dim:
        raise ValueError("k_new/q shape does not match the cache")
    if attn_scale is None:
        attn_scale = 1.0 / math.sqrt(D)
    if out is None:
        out = _output(stream, (B, Hq, n_q, D), torch.float32, q.device)
    _need_cuda("out", out)
    if workspace is None:
        workspace = _workspace(stream, _sized(cache, attend_workspace_bytes, Hq, n_q, kv_len, chunk), q.device)
    _need_cuda("workspace", workspace)
    L.check(L.lib().kvq_append_decode_attend(
        C.byref(cache.struct), k_new.data_ptr(), v_new.data_ptr(), _DTYPES[k_new.dtype], n_new, pos0, q.data_ptr(),
        _DTYPES[q.dtype], Hq, n_q, kv_len, int(bool(causal)), q_pos0, float(attn_scale), chunk, out.data_ptr(),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream(stream)),
        "kvq_append_decode_attend")
    return out


def decode_attend_static(cache: KVCache, q: torch.Tensor, kv_len: int, causal: bool = False, q_pos0: int = 0,
                         attn_scale: float | None = None, chunk: int = 0, out: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """decode_attend without a workspace: the library's built-in device scratch holds the partials.

    For callers that cannot allocate device memory of their own. Calls share that scratch, so
    calls that overlap on the GPU race; the first call on a device must precede stream capture.
    """
    _need_cuda("q", q)
    B, Hq, n_q, D = q.shape
    if B != cache.batch or D != cache.head_dim:
        raise ValueError("q shape does not match the cache")
    if attn_scale is None:
        attn_scale = 1.0 / math.sqrt(D)
    if out is None:
        out = _output(stream, (B, Hq, n_q, D), torch.float32, q.device)
    _need_cuda("out", out)
    L.check(L.lib().kvq_decode_attend_static(C.byref(cache.struct), q.data_ptr(), _DTYPES[q.dtype], Hq, n_q,
                                             kv_len, int(bool(causal)), q_pos0, float(attn_scale), chunk,
                                             out.data_ptr(), _stream(stream)), "kvq_decode_attend_static")
    return out


def debug_scores_i32(cache: KVCache, q: torch.Tensor, kv_len: int, stream=None):
    """Hadamard-int4 exact integer body scores [B][H_q][n_q][kv_len - n_window] and the int8 row scales."""
    _need_cuda("q", q)
    B, Hq, n_q, D = q.shape
    n_body = kv_len - min(cache.n_recent, kv_len)
    buf = _output(stream, B * Hq * n_q * max(n_body, 1), torch.int32, q.device)
    s_q = _output(stream, (B, Hq, n_q), torch.float32, q.device)
    L.check(L.lib().kvq_debug_scores_i32(C.byref(cache.struct), q.data_ptr(), _DTYPES[q.dtype], Hq, n_q, kv_len,
                                         buf.data_ptr(), s_q.data_ptr(), _stream(stream)),
            "kvq_debug_scores_i32")
    return buf[:B * Hq * n_q * n_body].view(B, Hq, n_q, n_body), s_q


def debug_attend_scores_i32(cache: KVCache, q: torch.Tensor, kv_len: int, causal: bool = False, q_pos0: int = 0,
                            attn_scale: float | None = None, chunk: int = 0, fill: int = -(2 ** 31), stream=None):
    """decode_attend on the production kernels, with the tensor-core kernel that scores the body also
    writing its exact integer scores: returns (out, scores [B][H_q][n_q][n_body] int32, s_q [B][H_q][n_q]).
    Score entries the kernels did not compute keep `fill`."""
    _need_cuda("q", q)
    B, Hq, n_q, D = q.shape
    if B != cache.batch or D != cache.head_dim:
        raise ValueError("q shape does not match the cache")
    if attn_scale is None:
        attn_scale = 1.0 / math.sqrt(D)
    n_body = kv_len - min(cache.n_recent, kv_len)
    need = attend_workspace_bytes(cache, Hq, n_q, kv_len, chunk)
    out = _output(stream, (B, Hq, n_q, D), torch.float32, q.device)
    scores = _output(stream, B * Hq * n_q * max(n_body, 1), torch.int32, q.device)
    s_q = _output(stream, (B, Hq, n_q), torch.float32, q.device)
    with _made_on(stream):
        scores.fill_(fill)
        s_q.zero_()
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    L.check(L.lib().kvq_debug_attend_scores_i32(
        C.byref(cache.struct), q.data_ptr(), _DTYPES[q.dtype], Hq, n_q, kv_len, int(bool(causal)), q_pos0,
        float(attn_scale), chunk, out.data_ptr(), workspace.data_ptr(), workspace.numel(), scores.data_ptr(),
        s_q.data_ptr(), _stream(stream)), "kvq_debug_attend_scores_i32")
    return out, scores[:B * Hq * n_q * n_body].view(B, Hq, n_q, n_body), s_q


# ------------------------------------------------------------------ paged pool
class PagedKVCache:
    """Device planes of one layer's paged pool, its block table and the C struct describing them.

    Planes (K and V each): payload u8 [n_pages][H_kv][page_size][row_bytes]; scale f16
    [n_pages][H_kv][page_size][D/32] (f32 [n_pages][H_kv][page_size] for had_int4, f32
    [n_pages][H_kv][page_size/64] for int8_b64 / e4m3_b64); zero f16
    (asym4_g32); recent f32 [batch][H_kv][n_recent][D] (had_int4 with n_recent > 0, one ring per
    sequence). block_table: int32 [batch][max_pages_per_seq] (pool page of each logical page),
    owned by this object; the caller fills it (set_block_table) before storing.
    """

    def __init__(self, layout, batch: int, n_kv_heads: int, head_dim: int, page_size: int, n_pages: int,
                 max_pages_per_seq: int, n_recent: int = 0, device="cuda"):
        self.layout = _layout_id(layout)
        self.batch, self.n_kv_heads, self.head_dim = batch, n_kv_heads, head_dim
        self.page_size, self.n_pages, self.max_pages_per_seq = page_size, n_pages, max_pages_per_seq
        self.capacity = page_size * max_pages_per_seq
        self.plane_layouts = dict(zip(("k", "v"), L.plane_ids(self.layout)))
        self.n_recent = n_recent if self.plane_layouts["k"] in L.HADAMARD_IDS else 0
        dev = torch.device(device)
        shp = (n_pages, n_kv_heads, page_size)
        self.planes = {}
        for t in ("k", "v"):
            lt = self.plane_layouts[t]
            out = (C.c_size_t * 4)()
            L.check(L.lib().kvq_paged_cache_bytes(lt, n_pages, n_kv_heads, head_dim, page_size, batch,
                                                  self.n_recent, out), "kvq_paged_cache_bytes")
            pl = _plane_tensors(lt, shp, head_dim, dev, self.n_recent, (batch, n_kv_heads))
            assert pl["payload"].numel() == out[0]
            self.planes[t] = pl
        self.block_table = torch.zeros((batch, max_pages_per_seq), dtype=torch.int32, device=dev)
        self.struct = L.KvqPagedCache(
            self.layout, batch, n_kv_heads, head_dim, page_size, n_pages, max_pages_per_seq, self.n_recent,
            _ptr(self.planes["k"]["payload"]), _ptr(self.planes["v"]["payload"]),
            _ptr(self.planes["k"]["scale"]), _ptr(self.planes["v"]["scale"]),
            _ptr(self.planes["k"].get("zero")), _ptr(self.planes["v"].get("zero")),
            _ptr(self.planes["k"].get("recent")), _ptr(self.planes["v"].get("recent")),
            _ptr(self.block_table))

    def set_block_table(self, table) -> None:
        """Copy an int [batch][max_pages_per_seq] table (pool page of each logical page)."""
        t = torch.as_tensor(table, dtype=torch.int32)
        if tuple(t.shape) != (self.batch, self.max_pages_per_seq):
            raise ValueError("block table shape does not match the cache")
        self.block_table.copy_(t)

    def read_bytes(self, seq_lens) -> int:
        """Packed bytes (payload + scales [+ zeros] [+ window]) one attention call reads."""
        return self.n_kv_heads * sum(_plane_read_bytes(self.plane_layouts[t], self.head_dim, int(n), self.n_recent)
                                     for n in seq_lens for t in ("k", "v"))


def _i32_vec(name: str, t: torch.Tensor, n: int) -> None:
    _need_cuda(name, t)
    if t.dtype != torch.int32 or t.numel() != n:
        raise ValueError(f"{name} must be a CUDA int32 tensor of {n} entries")


def paged_store(cache: PagedKVCache, k_new: torch.Tensor, v_new: torch.Tensor, positions: torch.Tensor,
                stream=None) -> None:
    """Append k_new/v_new [B][H_kv][n_new][D]: sequence b's rows at [positions[b], positions[b] + n_new)."""
    _need_cuda("k_new", k_new)
    _need_cuda("v_new", v_new)
    _i32_vec("positions", positions, cache.batch)
    if k_new.shape != v_new.shape or k_new.dtype != v_new.dtype:
        raise ValueError("k_new and v_new must have the same shape and dtype")
    B, H, n_new, D = k_new.shape
    if (B, H, D) != (cache.batch, cache.n_kv_heads, cache.head_dim):
        raise ValueError("k_new shape does not match the cache")
    L.check(L.lib().kvq_paged_store(C.byref(cache.struct), k_new.data_ptr(), v_new.data_ptr(), _DTYPES[k_new.dtype],
                                    n_new, positions.data_ptr(), _stream(stream)), "kvq_paged_store")


def paged_attend_workspace_bytes(cache: PagedKVCache, n_q_heads: int, n_q: int, max_kv_len: int,
                                 chunk: int = 0) -> int:
    return int(L.lib().kvq_paged_attend_workspace_bytes(C.byref(cache.struct), n_q_heads, n_q, max_kv_len, chunk))


def paged_attend_chunk(cache: PagedKVCache, n_q_heads: int, n_q: int, max_kv_len: int, total_kv_len: int = 0,
                       chunk: int = 0) -> int:
    """The split-K chunk of a paged call (0 -> automatic); total_kv_len = the sum of the sequence
    lengths (0: every sequence at max_kv_len) balances a ragged batch."""
    return int(L.lib().kvq_paged_attend_chunk(C.byref(cache.struct), n_q_heads, n_q, max_kv_len, total_kv_len,
                                              chunk))


def paged_attend_plan_chunk(cache: PagedKVCache, n_q_heads: int, n_q: int, seq_lens, q_dtype=torch.bfloat16) -> int:
    """A balanced split-K chunk for this batch from the host copy of its sequence lengths."""
    import numpy as np
    lens = np.ascontiguousarray(np.asarray(seq_lens, dtype=np.int32))
    if lens.size != cache.batch:
        raise ValueError("seq_lens must have one entry per sequence")
    return int(L.lib().kvq_paged_attend_plan_chunk(C.byref(cache.struct), n_q_heads, n_q, _DTYPES[q_dtype],
                                                   lens.ctypes.data))


def _paged_out_ws(cache, q, max_kv_len, chunk, out, workspace, stream):
    B, Hq, n_q, D = q.shape
    if B != cache.batch or D != cache.head_dim:
        raise ValueError("q shape does not match the cache")
    if out is None:
        out = _output(stream, (B, Hq, n_q, D), torch.float32, q.device)
    _need_cuda("out", out)
    if workspace is None:
        workspace = _workspace(stream, _sized(cache, paged_attend_workspace_bytes, Hq, n_q, max_kv_len, chunk), q.device)
    _need_cuda("workspace", workspace)
    return out, workspace


def paged_decode_attend(cache: PagedKVCache, q: torch.Tensor, seq_lens: torch.Tensor, max_kv_len: int,
                        causal: bool = False, attn_scale: float | None = None, chunk: int = 0,
                        out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """Split-K attention of q [B][H_q][n_q][D] over each sequence's seq_lens[b] tokens -> f32 out
    (causal rows are each sequence's newest n_q tokens)."""
    _need_cuda("q", q)
    _i32_vec("seq_lens", seq_lens, cache.batch)
    Hq, n_q, D = q.shape[1], q.shape[2], q.shape[3]
    if attn_scale is None:
        attn_scale = 1.0 / math.sqrt(D)
    out, workspace = _paged_out_ws(cache, q, max_kv_len, chunk, out, workspace, stream)
    L.check(L.lib().kvq_paged_decode_attend(
        C.byref(cache.struct), q.data_ptr(), _DTYPES[q.dtype], Hq, n_q, seq_lens.data_ptr(), max_kv_len,
        int(bool(causal)), float(attn_scale), chunk, out.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream(stream)), "kvq_paged_decode_attend")
    return out


def paged_append_decode_attend(cache: PagedKVCache, k_new: torch.Tensor, v_new: torch.Tensor, q: torch.Tensor,
                               seq_lens: torch.Tensor, max_kv_len: int, causal: bool = False,
                               attn_scale: float | None = None, chunk: int = 0, out: torch.Tensor | None = None,
                               workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """paged_store at [seq_lens[b] - n_new, seq_lens[b]) then paged_decode_attend, in one call."""
    _need_cuda("k_new", k_new)
    _need_cuda("v_new", v_new)
    _need_cuda("q", q)
    _i32_vec("seq_lens", seq_lens, cache.batch)
    if k_new.shape != v_new.shape or k_new.dtype != v_new.dtype:
        raise ValueError("k_new and v_new must have the same shape and dtype")
    Bk, H, n_new, Dk = k_new.shape
    if (Bk, H, Dk) != (cache.batch, cache.n_kv_heads, cache.head_dim):
        raise ValueError("k_new shape does not match the cache")
    Hq, n_q, D = q.shape[1], q.shape[2], q.shape[3]
    if attn_scale is None:
        attn_scale = 1.0 / math.sqrt(D)
    out, workspace = _paged_out_ws(cache, q, max_kv_len, chunk, out, workspace, stream)
    L.check(L.lib().kvq_paged_append_decode_attend(
        C.byref(cache.struct), k_new.data_ptr(), v_new.data_ptr(), _DTYPES[k_new.dtype], n_new, q.data_ptr(),
        _DTYPES[q.dtype], Hq, n_q, seq_lens.data_ptr(), max_kv_len, int(bool(causal)), float(attn_scale), chunk,
        out.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream(stream)),
        "kvq_paged_append_decode_attend")
    return out


def _need_host(name: str, t: torch.Tensor) -> None:
    if t.is_cuda:
        raise ValueError(f"{name} must be a host tensor for the host-buffer call")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _host_out_ws(q, device, need, out, workspace, stream):
    B, Hq, n_q, D = q.shape
    if out is None:
        out = torch.empty((B, Hq, n_q, D), dtype=torch.float32, pin_memory=True)
    _need_host("out", out)
    if out.dtype != torch.float32 or tuple(out.shape) != (B, Hq, n_q, D):
        raise ValueError("out must be a float32 host tensor of q's shape")
    if workspace is None:
        with _made_on(stream):
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    _need_cuda("workspace", workspace)
    return out, workspace


def append_decode_attend_host_workspace_bytes(cache: KVCache, kv_dtype, n_new: int, q_dtype, n_q_heads: int,
                                              n_q: int, kv_len: int, chunk: int = 0) -> int:
    return L.lib().kvq_append_decode_attend_host_workspace_bytes(C.byref(cache.struct), _DTYPES[kv_dtype], n_new,
                                                                 _DTYPES[q_dtype], n_q_heads, n_q, kv_len, chunk)


def append_decode_attend_host(cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor, pos0: int, q: torch.Tensor,
                              kv_len: int, causal: bool = False, q_pos0: int = 0, attn_scale: float | None = None,
                              chunk: int = 0, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                              stream=None) -> torch.Tensor:
    """append_decode_attend with host tensors (ideally pinned): the library copies k_new, v_new and
    q to device staging in the workspace, runs the step and copies the f32 result back into the
    host tensor `out`, returning once it is filled."""
    for n, t in (("k_new", k_new), ("v_new", v_new), ("q", q)):
        _need_host(n, t)
    if k_new.shape != v_new.shape or k_new.dtype != v_new.dtype:
        raise ValueError("k_new and v_new must have the same shape and dtype")
    Bk, H, n_new, Dk = k_new.shape
    B, Hq, n_q, D = q.shape
    if (Bk, H, Dk) != (cache.batch, cache.n_kv_heads, cache.head_dim) or B != cache.batch or D != cache.head_dim:
        raise ValueError("k_new/q shape does not match the cache")
    if attn_scale is None:
        attn_scale = 1.0 / math.sqrt(D)
    need = 0 if workspace is not None else \
        append_decode_attend_host_workspace_bytes(cache, k_new.dtype, n_new, q.dtype, Hq, n_q, kv_len, chunk)
    out, workspace = _host_out_ws(q, cache.planes["k"]["payload"].device, need, out, workspace, stream)
    L.check(L.lib().kvq_append_decode_attend_host(
        C.byref(cache.struct), k_new.data_ptr(), v_new.data_ptr(), _DTYPES[k_new.dtype], n_new, pos0, q.data_ptr(),
        _DTYPES[q.dtype], Hq, n_q, kv_len, int(bool(causal)), q_pos0, float(attn_scale), chunk, out.data_ptr(),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream(stream)),
        "kvq_append_decode_attend_host")
    return out


def paged_append_decode_attend_host_workspace_bytes(cache: PagedKVCache, kv_dtype, n_new: int, q_dtype,
                                                    n_q_heads: int, n_q: int, max_kv_len: int, chunk: int = 0) -> int:
    return L.lib().kvq_paged_append_decode_attend_host_workspace_bytes(
        C.byref(cache.struct), _DTYPES[kv_dtype], n_new, _DTYPES[q_dtype], n_q_heads, n_q, max_kv_len, chunk)


def paged_append_decode_attend_host(cache: PagedKVCache, k_new: torch.Tensor, v_new: torch.Tensor, q: torch.Tensor,
                                    seq_lens: torch.Tensor, max_kv_len: int, causal: bool = False,
                                    attn_scale: float | None = None, chunk: int = 0,
                                    out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                                    stream=None) -> torch.Tensor:
    """paged_append_decode_attend with host tensors (seq_lens: host int32 [batch]); returns once the
    host tensor `out` holds the result."""
    for n, t in (("k_new", k_new), ("v_new", v_new), ("q", q), ("seq_lens", seq_lens)):
        _need_host(n, t)
    if seq_lens.dtype != torch.int32 or seq_lens.numel() != cache.batch:
        raise ValueError(f"seq_lens must be a host int32 tensor of {cache.batch} entries")
    if k_new.shape != v_new.shape or k_new.dtype != v_new.dtype:
        raise ValueError("k_new and v_new must have the same shape and dtype")
    Bk, H, n_new, Dk = k_new.shape
    B, Hq, n_q, D = q.shape
    if (Bk, H, Dk) != (cache.batch, cache.n_kv_heads, cache.head_dim) or B != cache.batch or D != cache.head_dim:
        raise ValueError("k_new/q shape does not match the cache")
    if attn_scale is None:
        attn_scale = 1.0 / math.sqrt(D)
    need = 0 if workspace is not None else \
        paged_append_decode_attend_host_workspace_bytes(cache, k_new.dtype, n_new, q.dtype, Hq, n_q, max_kv_len, chunk)
    out, workspace = _host_out_ws(q, cache.planes["k"]["payload"].device, need, out, workspace, stream)
    L.check(L.lib().kvq_paged_append_decode_attend_host(
        C.byref(cache.struct), k_new.data_ptr(), v_new.data_ptr(), _DTYPES[k_new.dtype], n_new, q.data_ptr(),
        _DTYPES[q.dtype], Hq, n_q, seq_lens.data_ptr(), max_kv_len, int(bool(causal)), float(attn_scale), chunk,
        out.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream(stream)),
        "kvq_paged_append_decode_attend_host")
    return out


# ------------------------------------------------------------------ rotary positions
# The calls below check with few torch calls: a decode step makes them once per layer, and their kernels
# take a few microseconds.
def _here(*named) -> int:
    """The current device, which every one of the (name, tensor) pairs has to live on (None passes)."""
    dev = _DEVICE()
    for name, t in named:
        if t is not None and t.get_device() != dev:               # -1 for a host tensor
            if not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
            raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{dev}")
    return dev


def _stream_of(stream, dev: int) -> int:
    return _RAW_STREAM(dev) if stream is None else _stream(stream)


def _dense(name: str, t: torch.Tensor, dtype, shape=None) -> None:
    """Checks a contiguous tensor of a type (and shape, where given)."""
    if t.dtype is not dtype or not t.is_contiguous() or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor" + (f" of shape {tuple(shape)}" if shape is not None else ""))


def _ints(name: str, t: torch.Tensor | None, n: int) -> None:
    if t is not None and (t.dtype is not torch.int32 or t.numel() != n or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} entries")


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_len: float = 0.0, low: float | None = None, high: float | None = None):
    """Rotary frequencies (float64 CPU tensor [rot_dim / 2], radians per position) and the magnitude of
    their table. scaling: "none", "linear", "ntk", "banded" (low / high turns 1 / 4 within original_len
    by default) or "yarn" (1 / 32); see kvq_rope_scaling in include/kvq.h for the formulas."""
    if scaling not in L.ROPE_SCALINGS:
        raise ValueError(f"unknown rotary scaling {scaling!r}")
    lo = 1.0 if low is None else low
    hi = (32.0 if scaling == "yarn" else 4.0) if high is None else high
    cfg = L.KvqRopeConfig(rot_dim, L.ROPE_SCALINGS[scaling], base, factor, original_len, lo, hi)
    out = torch.empty(max(rot_dim // 2, 0), dtype=torch.float64)
    mag = C.c_float()
    L.check(L.lib().kvq_rope_frequencies(C.byref(cfg), out.data_ptr(), C.byref(mag)), "kvq_rope_frequencies")
    return out, mag.value


def rope_table(inv_freq: torch.Tensor, n_pos: int, pos0: int = 0, magnitude: float = 1.0,
               out: torch.Tensor | None = None, device="cuda", stream=None) -> torch.Tensor:
    """Rows [pos0, pos0 + n_pos) of a rotary table: f32 [n_pos][rot_dim], cosines then sines, times
    magnitude. inv_freq: host float64 [rot_dim / 2] (rope_frequencies)."""
    if inv_freq.is_cuda or inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous host float64 vector")
    rot_dim = 2 * inv_freq.numel()
    if out is None:
        out = _output(stream, (max(n_pos, 0), rot_dim), torch.float32, device)
    dev = _here(("out", out))
    _dense("out", out, torch.float32, (n_pos, rot_dim))
    L.check(L.lib().kvq_rope_table(inv_freq.data_ptr(), rot_dim, pos0, n_pos, magnitude, out.data_ptr(),
                                   _stream_of(stream, dev)), "kvq_rope_table")
    return out


def _rows(name: str, t: torch.Tensor) -> L.KvqRows:
    """A [batch][heads][n_new][head_dim] tensor by its strides (the last axis contiguous)."""
    (b, h, n, d), (sb, sh, sn, sd) = t.shape, t.stride()
    if sd != 1 and d > 1:
        raise ValueError(f"{name}: the head_dim axis must be contiguous")
    # the stride of an axis of one entry is never used
    return L.KvqRows(t.data_ptr(), sb if b > 1 else 0, sh if h > 1 else 0, sn if n > 1 else 0)


def _rope_call(cache, table, k_new, v_new, slots, q, positions, interleaved, q_out, stream):
    """The arguments both rotary appends share."""
    shape, dtype = k_new.shape, k_new.dtype
    if len(shape) != 4 or shape[0] != cache.batch or shape[1] != cache.n_kv_heads or shape[3] != cache.head_dim:
        raise ValueError("k_new shape does not match the cache")
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    if v_new.shape != shape or v_new.dtype is not dtype:
        raise ValueError("k_new and v_new must have the same shape and dtype")
    _dense("table", table, torch.float32)
    if table.dim() != 2:
        raise ValueError("table must be float32 [n_pos][rot_dim]")
    B, _, n_new, D = shape
    _ints("positions", positions, B * n_new)
    _ints("slots", slots, B)
    qr, Hq = None, 0
    if q is not None:
        Hq = q.shape[1]
        if q.shape != (B, Hq, n_new, D) or q.dtype is not dtype:
            raise ValueError("q must have k_new's batch, rows, head_dim and dtype")
        if q_out is None:
            q_out = _output(stream, (B, Hq, n_new, D), dtype, q.device)
        else:
            _dense("q_out", q_out, dtype, (B, Hq, n_new, D))
        qr = C.byref(_rows("q", q))
    elif q_out is not None:
        raise ValueError("q_out without q")
    dev = _here(("cache", cache.planes["k"]["payload"]), ("table", table), ("k_new", k_new), ("v_new", v_new), ("q", q),
                ("positions", positions), ("slots", slots), ("q_out", q_out))
    n_pos, rot_dim = table.shape
    rope = L.KvqRope(table.data_ptr(), n_pos, rot_dim, 1 if interleaved else 0, _ptr(positions))
    return (C.byref(cache.struct), C.byref(rope), C.byref(_rows("k_new", k_new)), C.byref(_rows("v_new", v_new)), qr,
            _DTYPES[dtype], Hq, n_new), q_out, _stream_of(stream, dev)


def rope_store(cache: KVCache, table: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, pos0: int,
               q: torch.Tensor | None = None, positions: torch.Tensor | None = None, interleaved: bool = False,
               q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """store() of k_new rotated by the table and of v_new at slots [pos0, pos0 + n_new); returns q rotated
    ([B][H_q][n_new][D], contiguous, q's dtype). k_new, v_new and q may be strided views. positions: int32
    [B][n_new], the rotary positions where they are not the slots."""
    args, q_out, st = _rope_call(cache, table, k_new, v_new, None, q, positions, interleaved, q_out, stream)
    L.check(L.lib().kvq_rope_store(*args, pos0, _ptr(q_out), st), "kvq_rope_store")
    return q_out


def paged_rope_store(cache: PagedKVCache, table: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                     slots: torch.Tensor, q: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                     interleaved: bool = False, q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """rope_store into a paged pool: sequence b's rows at slots [slots[b], slots[b] + n_new)."""
    args, q_out, st = _rope_call(cache, table, k_new, v_new, slots, q, positions, interleaved, q_out, stream)
    L.check(L.lib().kvq_paged_rope_store(*args, slots.data_ptr(), _ptr(q_out), st), "kvq_paged_rope_store")
    return q_out


# ------------------------------------------------------------------ a cache inside a budget
def _scores(name: str, t: torch.Tensor, cache) -> int:
    """Checks running scores f32 [B][H_kv][stride] and returns the stride."""
    shape = t.shape
    if t.dtype is not torch.float32 or len(shape) != 3 or shape[0] != cache.batch or shape[1] != cache.n_kv_heads or \
            not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous float32 [batch][n_kv_heads][tokens]")
    return shape[2]


def attend_weights_workspace_bytes(cache: KVCache, n_q_heads: int, n_q: int, kv_len: int, chunk: int = 0) -> int:
    return L.lib().kvq_attend_weights_workspace_bytes(C.byref(cache.struct), n_q_heads, n_q, kv_len, chunk)


def paged_attend_weights_workspace_bytes(cache: PagedKVCache, n_q_heads: int, n_q: int, max_kv_len: int,
                                         chunk: int = 0) -> int:
    return L.lib().kvq_paged_attend_weights_workspace_bytes(C.byref(cache.struct), n_q_heads, n_q, max_kv_len, chunk)


def _weights_call(cache, need_fn, q, n, seq_lens, scores, scores_out, attn_scale, chunk, out, workspace, stream):
    """The buffers both calls share: (out, scores_out, stride, attn_scale, workspace, its bytes, stream)."""
    shape = q.shape
    if len(shape) != 4 or shape[0] != cache.batch or shape[3] != cache.head_dim:
        raise ValueError("q shape does not match the cache")
    if q.dtype not in _DTYPES or not q.is_contiguous():
        raise ValueError("q must be contiguous f32, bf16 or f16")
    if scores_out is None:
        if scores is None:
            raise ValueError("scores or scores_out is needed")
        scores_out = scores
    stride = _scores("scores_out", scores_out, cache)
    if scores is not None and scores is not scores_out and _scores("scores", scores, cache) != stride:
        raise ValueError("scores and scores_out must have the same shape")
    _ints("seq_lens", seq_lens, cache.batch)
    if out is None:
        out = _output(stream, shape, torch.float32, q.device)
    else:
        _dense("out", out, torch.float32, shape)
    if workspace is None:
        workspace = _workspace(stream, _sized(cache, need_fn, shape[1], shape[2], n, chunk), q.device)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    dev = _here(("cache", cache.planes["k"]["payload"]), ("q", q), ("scores", scores), ("scores_out", scores_out),
                ("seq_lens", seq_lens), ("out", out), ("workspace", workspace))
    return (out, scores_out, stride, 1.0 / math.sqrt(shape[3]) if attn_scale is None else attn_scale, workspace,
            workspace.numel() * workspace.element_size(), _stream_of(stream, dev))


def decode_attend_weights(cache: KVCache, q: torch.Tensor, kv_len: int, scores: torch.Tensor | None,
                          scores_out: torch.Tensor | None = None, decay: float = 1.0, causal: bool = False,
                          q_pos0: int = 0, attn_scale: float | None = None, chunk: int = 0,
                          out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """decode_attend that also updates the tokens' running attention weight: returns (out, scores_out) with
    scores_out[b][h][t] = decay * scores[b][h][t] + the weights of token t summed over the query rows of kv
    head h, t < kv_len. scores: f32 [B][H_kv][tokens >= kv_len] or None; scores_out defaults to scores."""
    out, scores_out, stride, attn_scale, workspace, nbytes, st = _weights_call(
        cache, attend_weights_workspace_bytes, q, kv_len, None, scores, scores_out, attn_scale, chunk, out, workspace, stream)
    L.check(L.lib().kvq_decode_attend_weights(
        C.byref(cache.struct), q.data_ptr(), _DTYPES[q.dtype], q.shape[1], q.shape[2], kv_len, 1 if causal else 0, q_pos0,
        attn_scale, chunk, out.data_ptr(), _ptr(scores), scores_out.data_ptr(), stride, decay, workspace.data_ptr(),
        nbytes, st), "kvq_decode_attend_weights")
    return out, scores_out


def paged_decode_attend_weights(cache: PagedKVCache, q: torch.Tensor, seq_lens: torch.Tensor, max_kv_len: int,
                                scores: torch.Tensor | None, scores_out: torch.Tensor | None = None,
                                decay: float = 1.0, causal: bool = False, attn_scale: float | None = None,
                                chunk: int = 0, out: torch.Tensor | None = None,
                                workspace: torch.Tensor | None = None, stream=None):
    """paged_decode_attend that also updates the tokens' running attention weight (decode_attend_weights);
    scores of sequence b's tokens t < seq_lens[b] are written."""
    out, scores_out, stride, attn_scale, workspace, nbytes, st = _weights_call(
        cache, paged_attend_weights_workspace_bytes, q, max_kv_len, seq_lens, scores, scores_out, attn_scale, chunk, out,
        workspace, stream)
    L.check(L.lib().kvq_paged_decode_attend_weights(
        C.byref(cache.struct), q.data_ptr(), _DTYPES[q.dtype], q.shape[1], q.shape[2], seq_lens.data_ptr(), max_kv_len,
        1 if causal else 0, attn_scale, chunk, out.data_ptr(), _ptr(scores), scores_out.data_ptr(), stride, decay,
        workspace.data_ptr(), nbytes, st), "kvq_paged_decode_attend_weights")
    return out, scores_out


def evict_select(scores: torch.Tensor, kv_len: int, n_keep: int, n_sink: int = 0, n_recent: int = 0,
                 seq_lens: torch.Tensor | None = None, keep: torch.Tensor | None = None,
                 new_lens: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The n_keep tokens each (batch, kv head) keeps, ascending (int32 [B][H_kv][n_keep]): the first n_sink,
    the last n_recent and the highest scores among the others, ties to the lowest index. seq_lens: int32 [B]
    lengths (else kv_len for all); sequences of at most n_keep tokens keep all, -1 fills their lists.
    new_lens: int32 [B], gets min(length, n_keep)."""
    if scores.dtype is not torch.float32 or scores.dim() != 3 or not scores.is_contiguous():
        raise ValueError("scores must be contiguous float32 [batch][n_kv_heads][tokens]")
    B, H, stride = scores.shape
    if keep is None:
        keep = _output(stream, (B, H, max(n_keep, 1)), torch.int32, scores.device)
    else:
        _ints("keep", keep, B * H * max(n_keep, 1))
    _ints("seq_lens", seq_lens, B)
    _ints("new_lens", new_lens, B)
    dev = _here(("scores", scores), ("keep", keep), ("seq_lens", seq_lens), ("new_lens", new_lens))
    L.check(L.lib().kvq_evict_select(scores.data_ptr(), B, H, stride, kv_len, _ptr(seq_lens), n_keep, n_sink, n_recent,
                                     keep.data_ptr(), _ptr(new_lens), _stream_of(stream, dev)), "kvq_evict_select")
    return keep


def _keep_list(keep: torch.Tensor, cache) -> int:
    """Checks a list of kept tokens int32 [B][H_kv][n_keep] and returns n_keep."""
    shape = keep.shape
    if keep.dtype is not torch.int32 or len(shape) != 3 or shape[0] != cache.batch or shape[1] != cache.n_kv_heads or \
            not keep.is_contiguous():
        raise ValueError("keep must be contiguous int32 [batch][n_kv_heads][n_keep]")
    return shape[2]


def evict_compact(cache: KVCache, keep: torch.Tensor, kv_len: int, dst: KVCache | None = None,
                  scores: torch.Tensor | None = None, scores_out: torch.Tensor | None = None, stream=None) -> int:
    """Move the kept tokens' packed rows together: token keep[b][h][i] becomes token i, in place or into dst;
    returns the new length min(kv_len, n_keep). scores (f32 [B][H_kv][tokens]) move likewise, in place or, with
    a dst, into scores_out; entries behind the kept ones become 0."""
    n_keep = _keep_list(keep, cache)
    stride = _scores("scores", scores, cache) if scores is not None else 0
    out_stride = _scores("scores_out", scores_out, cache) if scores_out is not None else stride
    dev = _here(("cache", cache.planes["k"]["payload"]), ("keep", keep), ("scores", scores), ("scores_out", scores_out),
                ("dst", None if dst is None else dst.planes["k"]["payload"]))
    L.check(L.lib().kvq_evict_compact(C.byref(cache.struct), None if dst is None else C.byref(dst.struct),
                                      keep.data_ptr(), n_keep, kv_len, _ptr(scores), stride, _ptr(scores_out),
                                      out_stride, _stream_of(stream, dev)), "kvq_evict_compact")
    return min(kv_len, n_keep)


def paged_evict_compact(cache: PagedKVCache, keep: torch.Tensor, seq_lens: torch.Tensor, max_kv_len: int,
                        scores: torch.Tensor | None = None, stream=None) -> None:
    """evict_compact in place in a paged pool, every sequence by its own length (seq_lens: the lengths before)."""
    n_keep = _keep_list(keep, cache)
    _ints("seq_lens", seq_lens, cache.batch)
    stride = _scores("scores", scores, cache) if scores is not None else 0
    dev = _here(("cache", cache.planes["k"]["payload"]), ("keep", keep), ("seq_lens", seq_lens), ("scores", scores))
    L.check(L.lib().kvq_paged_evict_compact(C.byref(cache.struct), keep.data_ptr(), n_keep, seq_lens.data_ptr(),
                                            max_kv_len, _ptr(scores), stride, _stream_of(stream, dev)),
            "kvq_paged_evict_compact")


# ------------------------------------------------------------------ steps planned on the device
class PagePlan(NamedTuple):
    """What page_plan writes: int32 lens [batch], granted [batch], n_free [1], cu_new [batch + 1], positions
    [max_tokens] and int64 slots [max_tokens]."""
    lens: torch.Tensor
    granted: torch.Tensor
    n_free: torch.Tensor
    cu_new: torch.Tensor
    slots: torch.Tensor
    positions: torch.Tensor


def page_plan(seq_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor, page_size: int,
              free_pages: torch.Tensor, n_free: torch.Tensor, max_tokens: int, lens_out: torch.Tensor | None = None,
              granted: torch.Tensor | None = None, n_free_out: torch.Tensor | None = None,
              cu_new: torch.Tensor | None = None, slots: torch.Tensor | None = None,
              positions: torch.Tensor | None = None, stream=None) -> PagePlan:
    """Pages, table entries and slot map of a step: request b holds seq_lens[b] tokens and asks for new_lens[b]
    more (negative: it has ended, its pages go back to free_pages). In the requests' order, those are granted that
    the table, the free pages and max_tokens have room for. block_table (int32 [batch][max_pages_per_seq]) and
    free_pages (int32, n_free [1] of them free) are updated in place; lens_out, granted and n_free_out may be
    seq_lens, new_lens and n_free. Token i of the step goes to pool row slots[i], at positions[i] of its sequence
    (-1 behind the last of cu_new[batch] tokens)."""
    if block_table.dim() != 2:
        raise ValueError("block_table must be int32 [batch][max_pages_per_seq]")
    B, per = block_table.shape
    n_tok = max(max_tokens, 0)
    out = {"lens_out": lens_out, "granted": granted, "n_free_out": n_free_out, "cu_new": cu_new, "slots": slots, "positions": positions}
    for (name, t), n in zip(out.items(), (B, B, 1, B + 1, n_tok, n_tok)):
        dtype = torch.int64 if name == "slots" else torch.int32
        if t is None:
            out[name] = _output(stream, n, dtype, seq_lens.device)
        else:
            _dense(name, t, dtype)
            if t.numel() != n:
                raise ValueError(f"{name} must have {n} entries")
    _ints("seq_lens", seq_lens, B)
    _ints("new_lens", new_lens, B)
    _ints("n_free", n_free, 1)
    _dense("block_table", block_table, torch.int32)
    _dense("free_pages", free_pages, torch.int32)
    here = _here(("seq_lens", seq_lens), ("new_lens", new_lens), ("block_table", block_table), ("free_pages", free_pages),
                 ("n_free", n_free), *out.items())
    L.check(L.lib().kvq_page_plan(B, page_size, per, seq_lens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(),
                                  free_pages.data_ptr(), free_pages.numel(), n_free.data_ptr(), max_tokens,
                                  *(t.data_ptr() for t in out.values()), _stream_of(stream, here)), "kvq_page_plan")
    return PagePlan(*out.values())


def paged_store_slots(cache: PagedKVCache, k_new: torch.Tensor, v_new: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
    """Append a ragged run of tokens k_new / v_new [n_tokens][H_kv][D] (strided views allowed): token t's rows go to
    pool row slots[t] (int64, as page_plan writes them; -1: nowhere)."""
    shape, dtype = k_new.shape, k_new.dtype
    if len(shape) != 3 or shape[1] != cache.n_kv_heads or shape[2] != cache.head_dim:
        raise ValueError("k_new must be [n_tokens][n_kv_heads][head_dim] of the cache")
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    if v_new.shape != shape or v_new.dtype is not dtype:
        raise ValueError("k_new and v_new must have the same shape and dtype")
    if slots.dtype is not torch.int64 or slots.numel() != shape[0] or not slots.is_contiguous():
        raise ValueError(f"slots must be a contiguous int64 tensor of {shape[0]} entries")
    dev = _here(("cache", cache.planes["k"]["payload"]), ("k_new", k_new), ("v_new", v_new), ("slots", slots))
    k, v = (_rows(name, t.transpose(0, 1).unsqueeze(0)) for name, t in (("k_new", k_new), ("v_new", v_new)))
    L.check(L.lib().kvq_paged_store_slots(C.byref(cache.struct), C.byref(k), C.byref(v), _DTYPES[dtype], shape[0],
                                          slots.data_ptr(), _stream_of(stream, dev)), "kvq_paged_store_slots")


# ------------------------------------------------------------------ attention over selected blocks
class BlockBounds:
    """Bounds of a cache's keys per block of 64 tokens and kv head: codes int8 [B][H_kv][cap/64][2][D] (smallest, then
    largest value of each channel) and scale f32 [B][H_kv][cap/64]; of a paged pool [n_pages][H_kv][page_size/64]..."""

    def __init__(self, cache):
        payload = cache.planes["k"]["payload"]
        lead = payload.shape[:2] + ((payload.shape[2] + 63) // 64,)
        self.codes = torch.zeros(lead + (2, cache.head_dim), dtype=torch.int8, device=payload.device)
        self.scale = torch.zeros(lead, dtype=torch.float32, device=payload.device)
        self.struct = L.KvqBlockBounds(self.codes.data_ptr(), self.scale.data_ptr())

    def fits(self, cache) -> None:
        shape = cache.planes["k"]["payload"].shape
        if self.scale.shape != shape[:2] + ((shape[2] + 63) // 64,) or self.codes.shape[-1] != cache.head_dim:
            raise ValueError("the bounds belong to a cache of another shape")


def block_bounds(cache: KVCache, bounds: BlockBounds, first: int, kv_len: int, stream=None) -> None:
    """Renew the bounds of every block that holds a token of [first, kv_len) (after an append at `first`)."""
    bounds.fits(cache)
    dev = _here(("cache", cache.planes["k"]["payload"]), ("bounds", bounds.codes))
    L.check(L.lib().kvq_block_bounds_update(C.byref(cache.struct), C.byref(bounds.struct), first, kv_len, _stream_of(stream, dev)),
            "kvq_block_bounds_update")


def paged_block_bounds(cache: PagedKVCache, bounds: BlockBounds, seq_lens: torch.Tensor, n_fresh: int, stream=None) -> None:
    """Renew the bounds of the blocks that hold each sequence's newest n_fresh tokens (seq_lens: the lengths with them)."""
    bounds.fits(cache)
    _ints("seq_lens", seq_lens, cache.batch)
    dev = _here(("cache", cache.planes["k"]["payload"]), ("bounds", bounds.codes), ("seq_lens", seq_lens))
    L.check(L.lib().kvq_paged_block_bounds_update(C.byref(cache.struct), C.byref(bounds.struct), seq_lens.data_ptr(), n_fresh,
                                                  _stream_of(stream, dev)), "kvq_paged_block_bounds_update")


def sparse_attend_workspace_bytes(cache: KVCache, n_q_heads: int, n_q: int, n_sel: int, chunk: int = 0) -> int:
    return L.lib().kvq_sparse_attend_workspace_bytes(C.byref(cache.struct), n_q_heads, n_q, n_sel, chunk)


def paged_sparse_attend_workspace_bytes(cache: PagedKVCache, n_q_heads: int, n_q: int, n_sel: int, chunk: int = 0) -> int:
    return L.lib().kvq_paged_sparse_attend_workspace_bytes(C.byref(cache.struct), n_q_heads, n_q, n_sel, chunk)


def _blocks_call(cache, q, seq_lens) -> None:
    """The checks that the calls below share."""
    shape = q.shape
    if len(shape) != 4 or shape[0] != cache.batch or shape[3] != cache.head_dim:
        raise ValueError("q shape does not match the cache")
    if q.dtype not in _DTYPES or not q.is_contiguous():
        raise ValueError("q must be contiguous f32, bf16 or f16")
    if seq_lens is not None:
        _ints("seq_lens", seq_lens, cache.batch)


def _select_call(fn, cache, bounds, q, seq_lens, lengths, n_sel, n_sink, n_recent, sel, stream):
    bounds.fits(cache)
    _blocks_call(cache, q, seq_lens)
    shape = (cache.batch, cache.n_kv_heads, q.shape[2], max(n_sel, 1))
    if sel is None:
        sel = _output(stream, shape, torch.int32, q.device)
    else:
        _dense("sel", sel, torch.int32, shape)
    dev = _here(("cache", cache.planes["k"]["payload"]), ("bounds", bounds.codes), ("q", q), ("seq_lens", seq_lens), ("sel", sel))
    L.check(getattr(L.lib(), fn)(C.byref(cache.struct), C.byref(bounds.struct), q.data_ptr(), _DTYPES[q.dtype], q.shape[1], q.shape[2],
                                 *lengths, n_sel, n_sink, n_recent, sel.data_ptr(), _stream_of(stream, dev)), fn)
    return sel


def block_select(cache: KVCache, bounds: BlockBounds, q: torch.Tensor, kv_len: int, n_sel: int, n_sink: int = 1, n_recent: int = 1,
                 causal: bool = False, q_pos0: int = 0, sel: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The n_sel blocks of 64 tokens for each query row and kv head, ascending (int32 [B][H_kv][n_q][n_sel]): the first n_sink, the
    last n_recent that the row sees, and those whose bounds allow the largest scores, ties to the lowest index; -1 behind the
    blocks of a row that sees fewer."""
    return _select_call("kvq_block_select", cache, bounds, q, None, (kv_len, 1 if causal else 0, q_pos0), n_sel, n_sink, n_recent, sel,
                        stream)


def paged_block_select(cache: PagedKVCache, bounds: BlockBounds, q: torch.Tensor, seq_lens: torch.Tensor, max_kv_len: int, n_sel: int,
                       n_sink: int = 1, n_recent: int = 1, causal: bool = False, sel: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """block_select over a paged pool, each sequence by its own length (causal rows are its newest n_q tokens)."""
    return _select_call("kvq_paged_block_select", cache, bounds, q, seq_lens, (seq_lens.data_ptr(), max_kv_len, 1 if causal else 0),
                        n_sel, n_sink, n_recent, sel, stream)


def _sparse_call(fn, need, cache, q, sel, seq_lens, lengths, attn_scale, chunk, out, workspace, stream):
    shape = q.shape
    if sel.dtype is not torch.int32 or sel.dim() != 4 or len(shape) != 4 or sel.shape[:3] != (cache.batch, cache.n_kv_heads, shape[2]) or \
            not sel.is_contiguous():
        raise ValueError("sel must be contiguous int32 [batch][n_kv_heads][n_q][n_sel]")
    _blocks_call(cache, q, seq_lens)
    if workspace is None:
        workspace = _workspace(stream, _sized(cache, need, shape[1], shape[2], sel.shape[3], chunk), q.device)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    nbytes = workspace.numel() * workspace.element_size()
    if out is None:
        out = _output(stream, shape, torch.float32, q.device)
    else:
        _dense("out", out, torch.float32, shape)
    dev = _here(("cache", cache.planes["k"]["payload"]), ("q", q), ("sel", sel), ("seq_lens", seq_lens), ("out", out), ("workspace", workspace))
    L.check(getattr(L.lib(), fn)(C.byref(cache.struct), q.data_ptr(), _DTYPES[q.dtype], shape[1], shape[2], *lengths,
                                 1.0 / math.sqrt(shape[3]) if attn_scale is None else attn_scale, sel.data_ptr(), sel.shape[3], chunk,
                                 out.data_ptr(), workspace.data_ptr(), nbytes, _stream_of(stream, dev)), fn)
    return out


def sparse_attend(cache: KVCache, q: torch.Tensor, sel: torch.Tensor, kv_len: int, causal: bool = False, q_pos0: int = 0,
                  attn_scale: float | None = None, chunk: int = 0, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """decode_attend in which each query row sees only the blocks of 64 tokens in its list sel [B][H_kv][n_q][n_sel] (block_select's,
    or any ascending one) -> f32 out [B][H_q][n_q][D]."""
    return _sparse_call("kvq_sparse_attend", sparse_attend_workspace_bytes, cache, q, sel, None, (kv_len, 1 if causal else 0, q_pos0),
                        attn_scale, chunk, out, workspace, stream)


def paged_sparse_attend(cache: PagedKVCache, q: torch.Tensor, sel: torch.Tensor, seq_lens: torch.Tensor, max_kv_len: int,
                        causal: bool = False, attn_scale: float | None = None, chunk: int = 0, out: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """sparse_attend over a paged pool, each sequence by its own length."""
    return _sparse_call("kvq_paged_sparse_attend", paged_sparse_attend_workspace_bytes, cache, q, sel, seq_lens,
                        (seq_lens.data_ptr(), max_kv_len, 1 if causal else 0), attn_scale, chunk, out, workspace, stream)
