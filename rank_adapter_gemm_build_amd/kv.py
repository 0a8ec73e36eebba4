"""Binding of the paged-cache operators (page plan, rotary append, paged attention): what a
layer does between its packed q/k/v projection and its o projection.

    plan = PagePlan(device, max_seqs, max_tokens)
    page_plan(plan, past_lens, new_lens, T, free_pages, cursor, block_table, page_size)     # once a step
    rotary_append(rotary, qkv, num_q_heads, plan.positions, plan.slots, q, cache)           # per layer
    paged_attention(attention, q, cache, block_table, plan.seq_lens, plan.query_start, out)

Imported by the package itself; argument checks and marshalling only."""
from __future__ import annotations

import ctypes as C
import math
from typing import Optional, Sequence

from . import (LORA_BF16, LORA_F32, LORA_FP8E4M3, _check, _CKVCache, _dt, lib)

LORA_MAX_SEQS, LORA_MAX_HEAD_DIM, LORA_PLAN_META = 4096, 256, 8
LORA_ROPE_PLAIN, LORA_ROPE_LINEAR, LORA_ROPE_WAVELENGTH, LORA_ROPE_DIM = 0, 1, 2, 3
_SCALINGS = {"plain": LORA_ROPE_PLAIN, "linear": LORA_ROPE_LINEAR, "wavelength": LORA_ROPE_WAVELENGTH, "dim": LORA_ROPE_DIM}

__all__ = ["LORA_MAX_SEQS", "LORA_MAX_HEAD_DIM", "LORA_PLAN_META", "LORA_ROPE_PLAIN", "LORA_ROPE_LINEAR",
           "LORA_ROPE_WAVELENGTH", "LORA_ROPE_DIM", "PagePlan", "KVCache", "Rotary", "Attention", "rotary_frequencies",
           "page_plan", "rotary_append", "paged_attention"]


# A call of a small step costs the host more than the GPU, so the checks read each property of a
# tensor once and torch is looked up once.
torch = None          # the module, from the first object or call on
_raw_stream = None    # device -> raw handle of its current stream


def _load() -> None:
    global torch, _raw_stream
    import torch as module

    def public(device):
        return module.cuda.current_stream(device).cuda_stream
    _raw_stream = getattr(module._C, "_cuda_getCurrentRawStream", public)
    torch = module


def _stream_on(device: int, stream) -> Optional[int]:
    """Raw stream: the given one, or `device`'s current stream."""
    if stream is None:
        return _raw_stream(device) or None
    return (stream if isinstance(stream, int) else stream.cuda_stream) or None


def _elsewhere(device: int, *named) -> None:
    """The device rule's error, for the first tensor that breaks it."""
    for what, t in named:
        if t.get_device() != device:
            raise ValueError(f"{what} must be a tensor on cuda:{device}")


def _c_int(value: int, what: str) -> None:
    """A number that the C interface takes as an int (it would wrap)."""
    if not -2 ** 31 <= value < 2 ** 31:
        raise ValueError(f"{what} = {value} does not fit 32 bits")


def _vec(t, least: int, what: str) -> int:
    """Address of a contiguous int32 vector of at least `least` entries."""
    try:
        if t.dtype is not torch.int32:
            raise TypeError(f"{what} must be an int32 torch tensor (got {t.dtype})")
        shape = t.shape
        if len(shape) != 1 or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous 1-D tensor")
        if shape[0] < least:
            raise ValueError(f"{what} must have at least {least} entries (got {shape[0]})")
        return t.data_ptr()
    except AttributeError:
        raise TypeError(f"{what} must be a torch tensor") from None


def _table(t, rows: int) -> tuple:
    """(address, row stride, columns) of a block table."""
    try:
        if t.dtype is not torch.int32:
            raise TypeError(f"block_table must be an int32 torch tensor (got {t.dtype})")
        shape = t.shape
        if len(shape) != 2 or shape[0] < rows or shape[1] < 1:
            raise ValueError(f"block_table must be 2-D with at least {rows} rows and a column (got {tuple(shape)})")
        cols = shape[1]
        ld, unit = t.stride()
        if cols > 1 and unit != 1:
            raise ValueError("block_table must have unit column stride")
        if shape[0] == 1:
            ld = cols   # the stride of a single row is never used
        elif not cols <= ld < 2 ** 31:
            raise ValueError(f"block_table: row stride {ld} is not in [{cols} (its width), 2^31)")
        return t.data_ptr(), ld, cols
    except AttributeError:
        raise TypeError("block_table must be a torch tensor") from None


def _rows(t, dtype, rows: int, width: int, what: str) -> tuple:
    """(address, row stride) of a row-major [rows, width] matrix."""
    try:
        if t.dtype is not dtype:
            raise TypeError(f"{what} must be a torch tensor of {dtype} (got {t.dtype})")
        if t.shape != (rows, width):
            raise ValueError(f"{what} must have shape ({rows}, {width}) (got {tuple(t.shape)})")
        ld, unit = t.stride()
        if unit != 1 and width > 1:
            raise ValueError(f"{what} must have unit column stride (got stride {t.stride()})")
        if rows <= 1:
            ld = -(-width // 8) * 8   # the stride of a single row is never used
        elif not width <= ld < 2 ** 31:
            raise ValueError(f"{what}: row stride {ld} is not in [{width} (its width), 2^31)")
        return t.data_ptr(), ld
    except AttributeError:
        raise TypeError(f"{what} must be a torch tensor") from None


class KVCache:
    """One layer's paged cache: k and v [num_pages, page_size, num_heads, head_dim], any order
    of the first three axes in memory (the last has unit stride); float32, bfloat16 or
    e4m3 (torch.float8_e4m3fn or uint8; values are stored divided by k_scale / v_scale).
    Holds references to the tensors; see lora_kv_cache for the rules."""

    def __init__(self, k, v, k_scale: float = 1.0, v_scale: float = 1.0):
        if torch is None:
            _load()
        for t, what in ((k, "k"), (v, "v")):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{what} must be a torch tensor")
            if t.dim() != 4:
                raise ValueError(f"{what} must be [num_pages, page_size, num_heads, head_dim] (got {tuple(t.shape)})")
        if k.dtype != v.dtype or k.shape != v.shape or k.get_device() != v.get_device():
            raise ValueError("k and v must have the same dtype, shape and device")
        dtype = _dt(k)
        pages, size, heads, dim = k.shape
        if size < 16 or size > 1024 or size & (size - 1):
            raise ValueError(f"page_size must be a power of two in [16, 1024] (got {size})")
        if dim < 16 or dim % 16 or dim > LORA_MAX_HEAD_DIM:
            raise ValueError(f"head_dim must be a multiple of 16 up to {LORA_MAX_HEAD_DIM} (got {dim})")
        strides = []
        for t in (k, v):
            if t.stride(3) != 1:
                raise ValueError("the last axis must have unit stride")
            strides.append([0 if n == 1 else s for s, n in zip(t.stride()[:3], t.shape[:3])])
        if strides[0] != strides[1]:
            raise ValueError("k and v must have the same strides")
        if dtype == LORA_FP8E4M3 and not all(math.isfinite(s) and s > 0 for s in (k_scale, v_scale)):
            raise ValueError("k_scale and v_scale must be positive and finite")
        self.k, self.v, self.dtype, self.device = k, v, dtype, k.get_device()
        self.num_pages, self.page_size, self.num_heads, self.head_dim = pages, size, heads, dim
        self.act = torch.float32 if dtype == LORA_F32 else torch.bfloat16   # the activations it takes
        self.act_code = LORA_F32 if dtype == LORA_F32 else LORA_BF16
        self.c = _CKVCache(k.data_ptr(), v.data_ptr(), *strides[0], pages, size, heads, dim, dtype, k_scale, v_scale)
        self.ref = C.byref(self.c)


class PagePlan:
    """Output vectors of page_plan for steps of up to max_seqs requests and max_tokens tokens,
    at fixed addresses: seq_lens, query_start (one longer), positions, slots, meta (int32)."""

    META = ("tokens", "pages_taken", "pages_returned", "refused", "invalid", "free_pages")

    def __init__(self, device: int, max_seqs: int, max_tokens: int):
        if torch is None:
            _load()
        if not 0 <= max_seqs <= LORA_MAX_SEQS or max_tokens < 0:
            raise ValueError(f"max_seqs must be in [0, {LORA_MAX_SEQS}] and max_tokens not negative")
        self.device, self.max_seqs, self.max_tokens = device, max_seqs, max_tokens

        def vec(n):
            return torch.zeros(max(1, n), dtype=torch.int32, device=f"cuda:{device}")
        self.seq_lens, self.query_start = vec(max_seqs), vec(max_seqs + 1)
        self.positions, self.slots, self.meta = vec(max_tokens), vec(max_tokens), vec(LORA_PLAN_META)
        if not torch.cuda.is_current_stream_capturing():      # the vectors are ready for steps on any stream
            torch.cuda.current_stream(device).synchronize()
        self._out = [t.data_ptr() for t in (self.seq_lens, self.query_start, self.positions, self.slots, self.meta)]

    def query(self) -> dict:
        """The last step's counts (synchronous; for tests and a host that wants to know)."""
        return dict(zip(self.META, self.meta.tolist()))


def page_plan(plan: PagePlan, past_lens, new_lens, num_tokens: int, free_pages, cursor, block_table, page_size: int,
              cursor_out=None, stream=None) -> None:
    """Block table, slot map and positions of a step from the request lengths (see
    lora_page_plan).  past_lens, new_lens: int32 [requests]; num_tokens: entries of
    plan.positions and plan.slots to fill (the batch's tokens, or more for a padded step);
    free_pages: int32 ring [num_pages]; cursor: int32 [4] (first free place, free pages, 0,
    0); cursor_out: where the advanced cursor goes (default: cursor itself).  Nothing the call
    writes may overlap its other vectors: past_lens is not plan.seq_lens, but a copy of it."""
    if torch is None:
        _load()
    dev = plan.device
    past = _vec(past_lens, 0, "past_lens")
    n = past_lens.numel()
    new = _vec(new_lens, n, "new_lens")
    if new_lens.numel() != n:
        raise ValueError("past_lens and new_lens must have one entry per request")
    if n > plan.max_seqs:
        raise ValueError(f"{n} requests, the plan holds {plan.max_seqs}")
    if not 0 <= num_tokens <= plan.max_tokens:
        raise ValueError(f"num_tokens = {num_tokens} outside [0, {plan.max_tokens}]")
    ring, cur = _vec(free_pages, 1, "free_pages"), _vec(cursor, 4, "cursor")
    cur_out = cur if cursor_out is None else _vec(cursor_out, 2, "cursor_out")
    table, ld, cols = _table(block_table, n)
    _c_int(page_size, "page_size")
    lens, starts, positions, slots, meta = plan._out
    if lens - 4 * n < past < lens + 4 * n or lens - 4 * n < new < lens + 4 * n:
        raise ValueError("past_lens and new_lens must not overlap plan.seq_lens, which the call writes")
    if (past_lens.get_device() != dev or new_lens.get_device() != dev or free_pages.get_device() != dev or
            cursor.get_device() != dev or block_table.get_device() != dev or
            (cursor_out is not None and cursor_out.get_device() != dev)):
        _elsewhere(dev, ("past_lens", past_lens), ("new_lens", new_lens), ("free_pages", free_pages), ("cursor", cursor),
                   ("block_table", block_table), ("cursor_out", cursor_out))
    _check(lib.lora_page_plan(dev, past, new, n, num_tokens, page_size, free_pages.numel(), ring, cur, cur_out, table, ld,
                              cols, lens, starts, positions, slots, meta, _stream_on(dev, stream)), "lora_page_plan")


def rotary_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                       original_len: float = 0.0, low: float = 0.0, high: float = 0.0) -> list:
    """Rotary frequencies (radians a position) of rot_dim / 2 pairs; scaling "plain",
    "linear", "wavelength" or "dim" (see lora_rotary_frequencies)."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)} (got {scaling!r})")
    out = (C.c_double * max(1, rot_dim // 2))()
    _check(lib.lora_rotary_frequencies(rot_dim, base, _SCALINGS[scaling], factor, original_len, low, high, out),
           "lora_rotary_frequencies")
    return list(out)


class Rotary:
    """A rotary embedding of the first rot_dim values of a head (owns its device table);
    freqs: rot_dim / 2 frequencies (rotary_frequencies, or any others)."""

    def __init__(self, device: int, rot_dim: int, freqs: Sequence[float], interleaved: bool = False,
                 amplitude: float = 1.0):
        freqs = [float(f) for f in freqs]
        if len(freqs) != rot_dim // 2:
            raise ValueError(f"rot_dim {rot_dim} takes {rot_dim // 2} frequencies (got {len(freqs)})")
        self.handle = 0
        self.device, self.rot_dim, self.interleaved = device, rot_dim, bool(interleaved)
        h = C.c_void_p()
        _check(lib.lora_rotary_create(C.byref(h), device, rot_dim, int(self.interleaved),
                                      (C.c_double * max(1, len(freqs)))(*freqs), amplitude), "lora_rotary_create")
        self.handle = h.value

    def close(self) -> None:
        if self.handle:
            _check(lib.lora_rotary_destroy(self.handle), "lora_rotary_destroy")
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def rotary_append(rotary: Rotary, qkv, num_q_heads: int, positions, slots, q_out, cache: KVCache, stream=None) -> None:
    """q_out = the turned q heads of the packed rows qkv [T, (num_q_heads + 2 num_heads) *
    head_dim]; the turned k heads and the v heads go to the cache at `slots` (see
    lora_rotary_append).  q_out [T, num_q_heads * head_dim] may be qkv's own first columns."""
    if torch is None:
        _load()
    dev, dim = rotary.device, cache.head_dim
    T = qkv.shape[0] if hasattr(qkv, "shape") and len(qkv.shape) else 0
    x, ldx = _rows(qkv, cache.act, T, (num_q_heads + 2 * cache.num_heads) * dim, "qkv")
    q, ldq = _rows(q_out, cache.act, T, num_q_heads * dim, "q_out")
    pos, sl = _vec(positions, T, "positions"), _vec(slots, T, "slots")
    if (qkv.get_device() != dev or q_out.get_device() != dev or positions.get_device() != dev or
            slots.get_device() != dev or cache.device != dev):
        _elsewhere(dev, ("qkv", qkv), ("q_out", q_out), ("positions", positions), ("slots", slots), ("the cache", cache.k))
    _check(lib.lora_rotary_append(rotary.handle, x or None, ldx, cache.act_code, num_q_heads, pos or None, sl or None, T,
                                  q or None, ldq, cache.ref, _stream_on(dev, stream)), "lora_rotary_append")


class Attention:
    """Paged attention of up to max_seqs sequences and max_tokens new tokens (owns its workspace)."""

    def __init__(self, device: int, max_seqs: int, max_tokens: int, num_q_heads: int, num_kv_heads: int, head_dim: int):
        self.handle = 0
        for value, what in ((max_seqs, "max_seqs"), (max_tokens, "max_tokens"), (num_q_heads, "num_q_heads"),
                            (num_kv_heads, "num_kv_heads"), (head_dim, "head_dim")):
            _c_int(value, what)
        self.device, self.max_seqs, self.max_tokens = device, max_seqs, max_tokens
        self.num_q_heads, self.num_kv_heads, self.head_dim = num_q_heads, num_kv_heads, head_dim
        h = C.c_void_p()
        _check(lib.lora_attention_create(C.byref(h), device, max_seqs, max_tokens, num_q_heads, num_kv_heads, head_dim),
               "lora_attention_create")
        self.handle = h.value

    def close(self) -> None:
        if self.handle:
            _check(lib.lora_attention_destroy(self.handle), "lora_attention_destroy")
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def paged_attention(attention: Attention, q, cache: KVCache, block_table, seq_lens, query_start, out,
                    scale: Optional[float] = None, window: int = 0, lse=None, stream=None) -> None:
    """out [T, num_q_heads * head_dim] = attention of the new tokens' queries q over the cache
    (see lora_paged_attention).  block_table, seq_lens, query_start: of the page plan or
    the caller's own, one row (entry) per sequence, query_start one longer; scale: default
    1 / sqrt(head_dim); window: keys a token sees, 0 for all; lse: float32 [T, num_q_heads]."""
    if torch is None:
        _load()
    dev = attention.device
    n = query_start.numel() - 1 if hasattr(query_start, "numel") else 0
    starts, lens = _vec(query_start, 1, "query_start"), _vec(seq_lens, n, "seq_lens")
    table, ld, cols = _table(block_table, n)
    T = q.shape[0] if hasattr(q, "shape") and len(q.shape) else 0
    width = attention.num_q_heads * attention.head_dim
    _c_int(window, "window")
    qp, ldq = _rows(q, cache.act, T, width, "q")
    op, ldo = _rows(out, cache.act, T, width, "out")
    lp = None
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.shape != (T, attention.num_q_heads) or not lse.is_contiguous():
            raise ValueError(f"lse must be a contiguous float32 tensor of shape ({T}, {attention.num_q_heads})")
        if lse.get_device() != dev:
            _elsewhere(dev, ("lse", lse))
        lp = lse.data_ptr()
    if (q.get_device() != dev or out.get_device() != dev or block_table.get_device() != dev or
            seq_lens.get_device() != dev or query_start.get_device() != dev or cache.device != dev):
        _elsewhere(dev, ("q", q), ("out", out), ("block_table", block_table), ("seq_lens", seq_lens),
                   ("query_start", query_start), ("the cache", cache.k))
    _check(lib.lora_paged_attention(attention.handle, qp or None, ldq, cache.act_code, cache.ref, table, ld, cols,
                                    lens, starts, n, T, 1.0 / math.sqrt(attention.head_dim) if scale is None else scale,
                                    window, op or None, ldo, lp or None, _stream_on(dev, stream)), "lora_paged_attention")
