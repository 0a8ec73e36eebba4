"""Binding of the operators of beam search, and of batches with common tokens, over the paged cache: what a step
does between the logits and the next step's page plan, and the attention that reads common pages once.

    beams, plan, layers = Beams(device, requests, width, vocab), ForkPlan(device, rows, num_pages), KVLayers(caches)
    beam_select(beams, logits, scores, parents, tokens, scores)                           # once a step
    page_fork(plan, parents, lens, free_pages, cursor, shares, block_table, page_size)
    page_copy(layers, plan.copy_src[:rows], plan.copy_dst[:rows], plan.copy_tokens[:rows])
    shared_attention(attention, q, cache, block_table, seq_lens, query_start, group_start, common_lens, out)   # per layer

Imported by the package itself; argument checks and marshalling only."""
from __future__ import annotations

import ctypes as C
import math
from typing import Optional

from . import LORA_BF16, LORA_F32, _check, _CKVCache, lib
from . import kv
from .kv import KVCache, _c_int, _elsewhere, _rows, _stream_on, _table, _vec

LORA_MAX_BEAMS, LORA_MAX_VOCAB, LORA_FORK_META, LORA_MAX_LAYERS = 64, 1 << 24, 8, 128

__all__ = ["LORA_MAX_BEAMS", "LORA_MAX_VOCAB", "LORA_FORK_META", "LORA_MAX_LAYERS", "Beams", "ForkPlan", "KVLayers",
           "SharedAttention", "beam_select", "page_fork", "page_copy", "shared_attention"]


def _floats(t, least: int, what: str) -> int:
    """Address of a contiguous float32 vector of at least `least` entries."""
    try:
        if t.dtype is not kv.torch.float32:
            raise TypeError(f"{what} must be a float32 torch tensor (got {t.dtype})")
        shape = t.shape
        if len(shape) != 1 or not t.is_contiguous() or shape[0] < least:
            raise ValueError(f"{what} must be a contiguous 1-D tensor of at least {least} entries (got {tuple(shape)})")
        return t.data_ptr()
    except AttributeError:
        raise TypeError(f"{what} must be a torch tensor") from None


class Beams:
    """Beam selection for up to max_requests requests of `beams` beams each, over `vocab` tokens; `candidates`: the
    continuations that each request gets (default: as many as beams).  Owns its workspace."""

    def __init__(self, device: int, max_requests: int, beams: int, vocab: int, candidates: int = 0):
        self.handle = 0
        candidates = candidates or beams
        for value, what in ((max_requests, "max_requests"), (beams, "beams"), (vocab, "vocab"), (candidates, "candidates")):
            _c_int(value, what)
        self.device, self.max_requests, self.beams, self.vocab, self.candidates = device, max_requests, beams, vocab, candidates
        h = C.c_void_p()
        _check(lib.lora_beams_create(C.byref(h), device, max_requests, beams, vocab, candidates), "lora_beams_create")
        self.handle = h.value

    def close(self) -> None:
        if self.handle:
            _check(lib.lora_beams_destroy(self.handle), "lora_beams_destroy")
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def beam_select(beams: Beams, logits, scores, parents, tokens, scores_out, ended=None, end_token: int = -1, ended_out=None,
                weights=None, stream=None) -> None:
    """Every request's best continuations over its beams and the vocabulary (see lora_beam_select).  logits [requests *
    beams, vocab], bfloat16 or float32, unit column stride; scores: float32 [requests * beams]; parents, tokens
    (int32) and scores_out (float32): [requests * candidates]; ended, ended_out: int32, one entry a row and a candidate;
    weights: float32 [requests * beams], what scores are multiplied by to rank.  With as many candidates as
    beams scores_out may be scores itself, and ended_out may be ended."""
    if kv.torch is None:
        kv._load()
    dev = beams.device
    rows = logits.shape[0] if hasattr(logits, "shape") and len(logits.shape) == 2 else -1
    if rows < 0 or rows % beams.beams or logits.shape[1] != beams.vocab:
        raise ValueError(f"logits must be [requests * {beams.beams}, {beams.vocab}]")
    requests = rows // beams.beams
    dtype = logits.dtype
    if dtype is not kv.torch.bfloat16 and dtype is not kv.torch.float32:
        raise TypeError(f"logits must be a torch tensor of bfloat16 or float32 (got {dtype})")
    ld, unit = logits.stride()
    if unit != 1 and beams.vocab > 1:
        raise ValueError("logits must have unit column stride")
    if rows <= 1:
        ld = beams.vocab   # the stride of a single row is never used
    elif not beams.vocab <= ld < 2 ** 31:
        raise ValueError(f"logits: row stride {ld} is not in [{beams.vocab} (its width), 2^31)")
    n = requests * beams.candidates
    sc, par, tok, out = _floats(scores, rows, "scores"), _vec(parents, n, "parents"), _vec(tokens, n, "tokens"), _floats(scores_out, n, "scores_out")
    end = None if ended is None else _vec(ended, rows, "ended")
    end_out = None if ended_out is None else _vec(ended_out, n, "ended_out")
    wt = None if weights is None else _floats(weights, rows, "weights")
    _c_int(end_token, "end_token")
    if (logits.get_device() != dev or scores.get_device() != dev or parents.get_device() != dev or tokens.get_device() != dev or
            scores_out.get_device() != dev or (ended is not None and ended.get_device() != dev) or
            (ended_out is not None and ended_out.get_device() != dev) or (weights is not None and weights.get_device() != dev)):
        _elsewhere(dev, ("logits", logits), ("scores", scores), ("parents", parents), ("tokens", tokens), ("scores_out", scores_out),
                   *[(what, t) for what, t in (("ended", ended), ("ended_out", ended_out), ("weights", weights)) if t is not None])
    _check(lib.lora_beam_select(beams.handle, logits.data_ptr() or None, ld, LORA_F32 if dtype is kv.torch.float32 else LORA_BF16, sc or None,
                                end, end_token, wt, requests, par or None, tok or None, out or None, end_out, _stream_on(dev, stream)),
           "lora_beam_select")


class ForkPlan:
    """Output vectors and scratch words of page_fork for up to max_rows rows over num_pages pages, at fixed addresses: copy_src,
    copy_dst, copy_tokens (one entry a row; what page_copy takes), meta (int32)."""

    META = ("pages_drawn", "pages_returned", "refused", "invalid", "free_pages")

    def __init__(self, device: int, max_rows: int, num_pages: int):
        if kv.torch is None:
            kv._load()
        if not 0 <= max_rows <= kv.LORA_MAX_SEQS or not 1 <= num_pages < 2 ** 31:
            raise ValueError(f"max_rows must be in [0, {kv.LORA_MAX_SEQS}] and num_pages positive")
        self.device, self.max_rows, self.num_pages = device, max_rows, num_pages

        def vec(n, value=0):
            return kv.torch.full((max(1, n),), value, dtype=kv.torch.int32, device=f"cuda:{device}")
        self.copy_src, self.copy_dst, self.copy_tokens = vec(max_rows, -1), vec(max_rows, -1), vec(max_rows)
        self.meta, self._scratch = vec(LORA_FORK_META), vec((num_pages + 31) // 32)
        if not kv.torch.cuda.is_current_stream_capturing():      # the vectors are ready for steps on any stream
            kv.torch.cuda.current_stream(device).synchronize()
        self._out = [t.data_ptr() for t in (self.copy_src, self.copy_dst, self.copy_tokens, self._scratch, self.meta)]

    def query(self) -> dict:
        """The last fork's counts (synchronous; for tests and a host that wants to know)."""
        return dict(zip(self.META, self.meta.tolist()))


def page_fork(plan: ForkPlan, parents, lens, free_pages, cursor, shares, block_table, page_size: int, stream=None) -> None:
    """Block table rows continue the rows that `parents` names, with pages shared, copied where partly filled, and freed
    (see lora_page_fork).  parents, lens: int32 [rows], lens changes in place; free_pages: int32 ring [num_pages], cursor: int32
    [4], as page_plan takes them; shares: int32 [num_pages], holders of each page beyond the first.  The entries
    of plan.copy_src, copy_dst and copy_tokens past the rows are left as they were, with the pairs of an earlier call of more rows
    among them: page_copy is given the first `rows` of each."""
    if kv.torch is None:
        kv._load()
    dev = plan.device
    par = _vec(parents, 0, "parents")
    n = parents.numel()
    ln = _vec(lens, n, "lens")
    if lens.numel() != n:
        raise ValueError("parents and lens must have one entry per row")
    if n > plan.max_rows:
        raise ValueError(f"{n} rows, the plan holds {plan.max_rows}")
    ring, cur = _vec(free_pages, plan.num_pages, "free_pages"), _vec(cursor, 4, "cursor")
    sh = _vec(shares, plan.num_pages, "shares")
    if free_pages.numel() != plan.num_pages or shares.numel() != plan.num_pages:
        raise ValueError(f"free_pages and shares must have the plan's {plan.num_pages} entries")
    table, ld, cols = _table(block_table, n)
    _c_int(page_size, "page_size")
    src, dst, tokens, scratch, meta = plan._out
    if (parents.get_device() != dev or lens.get_device() != dev or free_pages.get_device() != dev or cursor.get_device() != dev or
            shares.get_device() != dev or block_table.get_device() != dev):
        _elsewhere(dev, ("parents", parents), ("lens", lens), ("free_pages", free_pages), ("cursor", cursor), ("shares", shares),
                   ("block_table", block_table))
    _check(lib.lora_page_fork(dev, par, n, ln, page_size, plan.num_pages, ring, cur, sh, table, ld, cols, src, dst, tokens, scratch,
                              meta, _stream_on(dev, stream)), "lora_page_fork")


class KVLayers:
    """The caches of several layers (KVCache), alike but for their tensors, for calls that take them all."""

    def __init__(self, caches):
        caches = list(caches)
        if not 1 <= len(caches) <= LORA_MAX_LAYERS or not all(isinstance(c, KVCache) for c in caches):
            raise ValueError(f"give 1..{LORA_MAX_LAYERS} KVCache objects")
        if len({c.device for c in caches}) != 1:
            raise ValueError("the caches must be on one device")
        self.caches, self.device = caches, caches[0].device
        self.c = (_CKVCache * len(caches))(*[c.c for c in caches])


def page_copy(caches, src, dst, tokens=None, stream=None) -> None:
    """The first tokens[i] tokens (all without `tokens`) of page src[i] go to page dst[i], in every layer (see
    lora_page_copy).  caches: a KVCache or a KVLayers; src, dst, tokens: int32 [pairs]."""
    if kv.torch is None:
        kv._load()
    if isinstance(caches, KVCache):
        dev, layers, count = caches.device, caches.ref, 1
    elif isinstance(caches, KVLayers):
        dev, layers, count = caches.device, caches.c, len(caches.caches)
    else:
        raise TypeError("caches must be a KVCache or a KVLayers")
    s = _vec(src, 0, "src")
    n = src.numel()
    d = _vec(dst, n, "dst")
    t = None if tokens is None else _vec(tokens, n, "tokens")
    if dst.numel() != n or (tokens is not None and tokens.numel() != n):
        raise ValueError("src, dst and tokens must have one entry per pair")
    if src.get_device() != dev or dst.get_device() != dev or (tokens is not None and tokens.get_device() != dev):
        _elsewhere(dev, ("src", src), ("dst", dst), *([("tokens", tokens)] if tokens is not None else []))
    _check(lib.lora_page_copy(dev, layers, count, s or None, d or None, t or None, n, _stream_on(dev, stream)), "lora_page_copy")


class SharedAttention:
    """Attention over common pages of up to max_seqs sequences and max_tokens new tokens (owns its workspace)."""

    def __init__(self, device: int, max_seqs: int, max_tokens: int, num_q_heads: int, num_kv_heads: int, head_dim: int):
        self.handle = 0
        for value, what in ((max_seqs, "max_seqs"), (max_tokens, "max_tokens"), (num_q_heads, "num_q_heads"),
                            (num_kv_heads, "num_kv_heads"), (head_dim, "head_dim")):
            _c_int(value, what)
        self.device, self.max_seqs, self.max_tokens = device, max_seqs, max_tokens
        self.num_q_heads, self.num_kv_heads, self.head_dim = num_q_heads, num_kv_heads, head_dim
        h = C.c_void_p()
        _check(lib.lora_shared_create(C.byref(h), device, max_seqs, max_tokens, num_q_heads, num_kv_heads, head_dim),
               "lora_shared_create")
        self.handle = h.value

    def close(self) -> None:
        if self.handle:
            _check(lib.lora_shared_destroy(self.handle), "lora_shared_destroy")
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def shared_attention(attention: SharedAttention, q, cache: KVCache, block_table, seq_lens, query_start, group_start, common_lens, out,
                     scale: Optional[float] = None, lse=None, stream=None) -> None:
    """paged_attention of sequences whose first tokens lie in common pages, which are read once for all of a group (see
    lora_shared_attention, which also says from how many common tokens on that pays).  group_start: int32 [groups + 1], the first sequence of each group; common_lens: int32
    [groups], the tokens that its sequences have in common.  The other arguments are paged_attention's."""
    if kv.torch is None:
        kv._load()
    dev = attention.device
    n = query_start.numel() - 1 if hasattr(query_start, "numel") else 0
    groups = group_start.numel() - 1 if hasattr(group_start, "numel") else 0
    starts, lens = _vec(query_start, 1, "query_start"), _vec(seq_lens, n, "seq_lens")
    first, common = _vec(group_start, 1, "group_start"), _vec(common_lens, groups, "common_lens")
    if common_lens.numel() != groups:
        raise ValueError("group_start must have one entry more than common_lens")
    table, ld, cols = _table(block_table, n)
    T = q.shape[0] if hasattr(q, "shape") and len(q.shape) else 0
    width = attention.num_q_heads * attention.head_dim
    qp, ldq = _rows(q, cache.act, T, width, "q")
    op, ldo = _rows(out, cache.act, T, width, "out")
    lp = None
    if lse is not None:
        if lse.dtype is not kv.torch.float32 or lse.shape != (T, attention.num_q_heads) or not lse.is_contiguous():
            raise ValueError(f"lse must be a contiguous float32 tensor of shape ({T}, {attention.num_q_heads})")
        if lse.get_device() != dev:
            _elsewhere(dev, ("lse", lse))
        lp = lse.data_ptr()
    if (q.get_device() != dev or out.get_device() != dev or block_table.get_device() != dev or seq_lens.get_device() != dev or
            query_start.get_device() != dev or group_start.get_device() != dev or common_lens.get_device() != dev or cache.device != dev):
        _elsewhere(dev, ("q", q), ("out", out), ("block_table", block_table), ("seq_lens", seq_lens), ("query_start", query_start),
                   ("group_start", group_start), ("common_lens", common_lens), ("the cache", cache.k))
    _check(lib.lora_shared_attention(attention.handle, qp or None, ldq, cache.act_code, cache.ref, table, ld, cols, lens, starts, n, T,
                                         first, common or None, groups, 1.0 / math.sqrt(attention.head_dim) if scale is None else scale,
                                         op or None, ldo, lp or None, _stream_on(dev, stream)), "lora_shared_attention")
