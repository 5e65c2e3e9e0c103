"""Attention on packed prompts and on batches that share a prefix.

The cascade softmax(scale * Q K^T + mask) V in one kernel, for grouped heads
(``include/b2b.h``, section "attention"): :class:`PromptAttentionPlan` for
whole prompts of different lengths, :class:`SharedPrefixAttentionPlan` for the
new tokens of a batch of requests that share one long prefix.  A plan holds
the head layout; a run takes tensors of any length, with any strides whose
last one is 1.  Inference only.  There is no CPU path.
"""
from __future__ import annotations

import ctypes

import torch

from . import DTYPES, _check, _current_device, _lib

__all__ = ["PromptAttentionPlan", "SharedPrefixAttentionPlan"]

_TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}
_P, _I = ctypes.c_void_p, ctypes.c_int64


def _rows(*names):
    """Fields of one b2b_attn_rows_t for each name."""
    return [(f"{n}_{f}", t) for n in names
            for f, t in (("data", _P), ("row_stride", _I), ("head_stride", _I), ("block_stride", _I))]


class _PromptRun(ctypes.Structure):  # b2b_prompt_attention_t
    _fields_ = ([(n, _I) for n in ("batch", "tokens", "key_rows", "causal")] + _rows("q", "k", "v", "out") +
                [(n, _P) for n in ("cu_q", "cu_k", "lse", "workspace")] + [("workspace_bytes", ctypes.c_size_t)])


class _SharedRun(ctypes.Structure):  # b2b_shared_attention_t
    _fields_ = ([(n, _I) for n in ("batch", "fresh", "prefix", "cache_rows", "cache_blocks", "table_width")] +
                _rows("q", "prefix_k", "prefix_v", "cache_k", "cache_v", "out") +
                [(n, _P) for n in ("lengths", "page_table", "lse", "workspace")] +
                [("workspace_bytes", ctypes.c_size_t)])


def _packed(t):
    """Arguments of a [rows][heads][dim] tensor."""
    s = t.stride()
    return t.data_ptr(), s[0], s[1], 0


def _blocks(t):
    """Arguments of a [blocks][rows][heads][dim] tensor."""
    s = t.stride()
    return t.data_ptr(), s[1], s[2], s[0]


class _AttentionPlan:
    """Head layout, scale and status word of one kind of attention.

    ``dtype`` is "f16" or "bf16"; ``q_heads`` a multiple of ``kv_heads``;
    ``head_dim`` a multiple of 8 up to 128; ``scale`` defaults to
    1 / sqrt(head_dim).  Bound to the GPU that is current now.
    """

    def __init__(self, dtype: str, q_heads: int, kv_heads: int, head_dim: int, scale: float | None = None):
        if dtype not in DTYPES:
            raise ValueError(f"unknown dtype {dtype!r}; one of {sorted(_TORCH)}")
        if scale is not None and not scale > 0:
            raise ValueError(f"scale {scale!r}: a positive number is expected")
        self.dtype, self.q_heads, self.kv_heads, self.head_dim = dtype, q_heads, kv_heads, head_dim
        h = ctypes.c_void_p()
        _check(_lib.b2b_attn_plan_create(ctypes.byref(h), DTYPES[dtype], q_heads, kv_heads, head_dim, scale or 0.0),
               "b2b_attn_plan_create")
        self._h = h
        self._torch_dtype = _TORCH[dtype]
        self.device_index = _current_device()
        self._workspace_sizes = {}

    # -- checks ------------------------------------------------------------
    def _tensor(self, name, t, heads, dims):
        if t.dtype is not self._torch_dtype:
            raise TypeError(f"{name}: {t.dtype} given, {self._torch_dtype} expected")
        shape = t.shape
        if len(shape) != dims or shape[-2] != heads or shape[-1] != self.head_dim:
            raise ValueError(f"{name}: shape {tuple(shape)} given, {'[blocks, ' if dims == 4 else '['}rows, {heads}, "
                             f"{self.head_dim}] expected")
        if t.stride(-1) != 1:
            raise ValueError(f"{name}: the elements of a head must be consecutive (last stride {t.stride(-1)})")
        self._placed(name, t)

    def _placed(self, name, t):
        if t.get_device() != self.device_index:  # (-1 for a CPU tensor)
            raise ValueError(f"{name} is on {t.device}, the plan on cuda:{self.device_index}")

    def _counts(self, name, t, n, width=None):
        """A dense int32 array of n entries (or n rows of any width)."""
        if t.dtype is not torch.int32:
            raise TypeError(f"{name}: {t.dtype} given, torch.int32 expected")
        if t.dim() != (1 if width is None else 2) or (n is not None and t.shape[0] != n) or not t.is_contiguous():
            raise ValueError(f"{name}: shape {tuple(t.shape)} given, a contiguous array of "
                             f"{n if width is None else f'{n} rows'} expected")
        self._placed(name, t)

    def _results(self, q, out, lse, return_lse, sizes, query):
        """Output, LSE and workspace of one run, in the pool of the current stream."""
        tokens = q.shape[0]
        if out is None:
            out = torch.empty((tokens, self.q_heads, self.head_dim), dtype=self._torch_dtype, device=q.device)
        else:
            self._tensor("out", out, self.q_heads, 3)
            if out.shape[0] != tokens:
                raise ValueError(f"out: {out.shape[0]} rows given, {tokens} expected")
        if lse is not None:
            if lse.dtype is not torch.float32:
                raise TypeError(f"lse: {lse.dtype} given, torch.float32 expected")
            if tuple(lse.shape) != (tokens, self.q_heads) or not lse.is_contiguous():
                raise ValueError(f"lse: shape {tuple(lse.shape)} given, contiguous {(tokens, self.q_heads)} expected")
            self._placed("lse", lse)
        elif return_lse:
            lse = torch.empty((tokens, self.q_heads), dtype=torch.float32, device=q.device)
        need = self._workspace_sizes.get(sizes)
        if need is None:
            n = ctypes.c_size_t()
            _check(query(self._h, *sizes, ctypes.byref(n)), query.__name__)
            if len(self._workspace_sizes) >= 4096:
                self._workspace_sizes.clear()
            need = self._workspace_sizes[sizes] = n.value
        ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
        return out, lse, ws, need

    # -- as the chain plans ------------------------------------------------
    def status(self, stream=None) -> int:
        """Synchronise and return the device status word (0 = OK)."""
        stream = torch.cuda.current_stream() if stream is None else stream
        return int(_lib.b2b_attn_plan_device_status(self._h, stream.cuda_stream or None))

    def set_wait_budget(self, ns: int) -> None:
        _check(_lib.b2b_attn_plan_set_wait_budget(self._h, int(ns)), "b2b_attn_plan_set_wait_budget")

    def set_debug(self, flags: int) -> None:
        """Test support (see b2b_plan_set_debug in include/b2b.h)."""
        _check(_lib.b2b_attn_plan_set_debug(self._h, int(flags)), "b2b_attn_plan_set_debug")

    def close(self) -> None:
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            _lib.b2b_attn_plan_destroy(h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class PromptAttentionPlan(_AttentionPlan):
    """Attention over whole prompts, packed one after the other."""

    def run(self, q, k, v, cu_q, cu_k=None, causal: bool = True, out=None, lse=None, return_lse: bool = False,
            stream=None):
        """Launch on ``stream`` (default: torch's current stream).

        ``q`` [rows, q_heads, head_dim]; ``k``, ``v`` [key rows, kv_heads,
        head_dim]; ``cu_q``, ``cu_k`` int32 [sequences + 1] on the GPU, the
        offsets of each sequence's rows (``cu_k`` defaults to ``cu_q``).  With
        ``causal`` row i of a sequence sees keys j <= i + (keys - queries).
        Returns ``out``, or ``(out, lse)`` when ``lse`` is given or asked for.
        """
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.run(q, k, v, cu_q, cu_k, causal, out, lse, return_lse)
        if cu_k is None:
            cu_k = cu_q
        self._tensor("q", q, self.q_heads, 3)
        self._tensor("k", k, self.kv_heads, 3)
        self._tensor("v", v, self.kv_heads, 3)
        tokens, key_rows = q.shape[0], k.shape[0]
        if v.shape[0] != key_rows:
            raise ValueError(f"v: {v.shape[0]} rows given, {key_rows} expected as k has")
        self._counts("cu_q", cu_q, None)
        batch = cu_q.shape[0] - 1
        if batch < 0:
            raise ValueError("cu_q: at least one offset is expected")
        self._counts("cu_k", cu_k, batch + 1)
        out, lse, ws, need = self._results(q, out, lse, return_lse, (batch, tokens, key_rows),
                                           _lib.b2b_prompt_attention_workspace)
        r = _PromptRun(batch, tokens, key_rows, bool(causal), *_packed(q), *_packed(k), *_packed(v), *_packed(out),
                       cu_q.data_ptr(), cu_k.data_ptr(), None if lse is None else lse.data_ptr(),
                       None if ws is None else ws.data_ptr(), need)
        _check(_lib.b2b_prompt_attention_run(self._h, ctypes.byref(r), torch.cuda.current_stream().cuda_stream or None),
               "b2b_prompt_attention_run")
        return out if lse is None else (out, lse)


class SharedPrefixAttentionPlan(_AttentionPlan):
    """Attention of a batch of requests that share one prefix, for their new tokens."""

    def run(self, q, prefix_k, prefix_v, cache_k, cache_v, lengths, page_table=None, out=None, lse=None,
            return_lse: bool = False, stream=None):
        """Launch on ``stream`` (default: torch's current stream).

        ``q`` [requests * new tokens, q_heads, head_dim], request after
        request; ``prefix_k``, ``prefix_v`` [prefix rows, kv_heads, head_dim];
        ``cache_k``, ``cache_v`` the requests' own keys and values, the new
        tokens' among them: dense [requests, rows, kv_heads, head_dim], or with
        ``page_table`` (int32 [requests, width]) a pool of pages [pages,
        rows of a page, kv_heads, head_dim]; ``lengths`` int32 [requests], own
        keys of each.  New token t sees the prefix and own keys
        j < length - new tokens + 1 + t.  Returns ``out``, or ``(out, lse)``
        when ``lse`` is given or asked for.
        """
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.run(q, prefix_k, prefix_v, cache_k, cache_v, lengths, page_table, out, lse, return_lse)
        self._tensor("q", q, self.q_heads, 3)
        self._tensor("prefix_k", prefix_k, self.kv_heads, 3)
        self._tensor("prefix_v", prefix_v, self.kv_heads, 3)
        self._tensor("cache_k", cache_k, self.kv_heads, 4)
        self._tensor("cache_v", cache_v, self.kv_heads, 4)
        if prefix_v.shape[0] != prefix_k.shape[0]:
            raise ValueError(f"prefix_v: {prefix_v.shape[0]} rows given, {prefix_k.shape[0]} expected as prefix_k has")
        if cache_v.shape != cache_k.shape:
            raise ValueError(f"cache_v: shape {tuple(cache_v.shape)} given, {tuple(cache_k.shape)} expected as cache_k has")
        self._counts("lengths", lengths, None)
        batch, tokens = lengths.shape[0], q.shape[0]
        if tokens % batch if batch else tokens:
            raise ValueError(f"q: {tokens} rows given, a multiple of the {batch} requests expected")
        fresh = tokens // batch if batch else 0
        blocks, rows = cache_k.shape[:2]
        width = 0
        if page_table is not None:
            self._counts("page_table", page_table, batch, "any")
            width = page_table.shape[1]
        elif blocks != batch:
            raise ValueError(f"cache_k: {blocks} requests given, {batch} expected as lengths has")
        prefix = prefix_k.shape[0]
        room = (width * rows if blocks else 0) if page_table is not None else rows
        out, lse, ws, need = self._results(q, out, lse, return_lse, (batch, fresh, prefix, room),
                                           _lib.b2b_shared_attention_workspace)
        r = _SharedRun(batch, fresh, prefix, rows, blocks, width, *_packed(q), *_packed(prefix_k), *_packed(prefix_v),
                       *_blocks(cache_k), *_blocks(cache_v), *_packed(out), lengths.data_ptr(),
                       None if page_table is None else page_table.data_ptr(), None if lse is None else lse.data_ptr(),
                       None if ws is None else ws.data_ptr(), need)
        _check(_lib.b2b_shared_attention_run(self._h, ctypes.byref(r), torch.cuda.current_stream().cuda_stream or None),
               "b2b_shared_attention_run")
        return out if lse is None else (out, lse)
