"""Attention on packed prompts and on batches that share a prefix.

The cascade softmax(scale * Q K^T + mask) V in one kernel, for grouped heads
(``include/b2b.h``, section "attention"): :class:`PromptAttentionPlan` for
whole prompts of different lengths, :class:`SharedPrefixAttentionPlan` for the
new tokens of a batch of requests that share one long prefix.  A plan holds
the head layout; a run takes tensors of any length on 16-byte boundaries, with
any positive strides that are multiples of 8 elements, the last one 1 (a stride
of 0, as of keys expanded over heads, is refused).  Inference only: inputs that
require a gradient are refused where gradients are recorded.  There is no CPU
path.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import math
import os
import struct
import warnings

from . import DTYPES, _check, _current_device, _lib, _stream_handle, library_path

__all__ = ["PromptAttentionPlan", "SharedPrefixAttentionPlan"]

_LOG2E = 1 / math.log(2)
_TYPES = {"f16": "float16", "bf16": "bfloat16"}

# Set when the first plan is made (_load): the package's other parts need neither torch nor the compiled module.
torch = _raw_stream = _binding = None

# The argument structures, whose members all take eight bytes (b2b_attn_rows_t:
# data, row_stride, head_stride, block_stride), as the C functions read them.
# b2b_prompt_attention_t: batch, tokens, key_rows, causal; q, k, v, out; cu_q, cu_k, lse, workspace, workspace_bytes
_prompt_run = struct.Struct("25q").pack
# b2b_shared_attention_t: batch, fresh, prefix, cache_rows, cache_blocks, table_width; q, prefix_k, prefix_v,
# cache_k, cache_v, out; lengths, page_table, lse, workspace, workspace_bytes
_shared_run = struct.Struct("35q").pack


class _NoBinding:
    """In the compiled module's place where there is none: every call takes the way through Python."""

    @staticmethod
    def bind(*_):
        return None

    prompt = shared = bind


def _load_binding():
    """The module that passes tensors to the C functions (binding/attention.cpp), if it is there for this torch."""
    path = os.path.join(os.path.dirname(library_path()), "attn_binding.so")
    try:
        loader = importlib.machinery.ExtensionFileLoader("attn_binding", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("attn_binding", loader))
        loader.exec_module(module)
        if not torch.__version__.startswith(module.torch_version):
            raise ImportError(f"built for torch {module.torch_version}, this is {torch.__version__}")
    except ImportError as e:
        warnings.warn(f"{path}: {e}; attention calls take some microseconds longer without it "
                      "(python fusion_b2b_gemm_gb300/_build.py)", RuntimeWarning, stacklevel=5)
        return _NoBinding
    module.connect(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
        _lib.b2b_prompt_attention_workspace, _lib.b2b_prompt_attention_run,
        _lib.b2b_shared_attention_workspace, _lib.b2b_shared_attention_run)))
    return module


def _load():
    global torch, _raw_stream, _binding
    if _binding is None:
        import torch
        # (the public torch.cuda.current_stream() builds an object each time, 3 us)
        _raw_stream = torch._C._cuda_getCurrentRawStream
        _binding = _load_binding()


class _AttentionPlan:
    """Head layout, scale and status word of one kind of attention.

    ``dtype`` is "f16" or "bf16"; ``q_heads`` a multiple of ``kv_heads``;
    ``head_dim`` a multiple of 8 up to 128; ``scale`` defaults to
    1 / sqrt(head_dim).  Bound to the GPU that is current now.
    """

    def __init__(self, dtype: str, q_heads: int, kv_heads: int, head_dim: int, scale: float | None = None):
        if dtype not in DTYPES:
            raise ValueError(f"unknown dtype {dtype!r}; one of {sorted(_TYPES)}")
        # (in 32 bits, where the kernel also takes it times log2(e); there 0 would mean the default)
        if scale is not None and not (ctypes.c_float(scale).value > 0 and ctypes.c_float(scale * _LOG2E).value < math.inf):
            raise ValueError(f"scale {scale!r}: a positive number is expected that fp32 holds, also times log2(e)")
        _load()
        self.dtype, self.q_heads, self.kv_heads, self.head_dim = dtype, q_heads, kv_heads, head_dim
        h = ctypes.c_void_p()
        _check(_lib.b2b_attn_plan_create(ctypes.byref(h), DTYPES[dtype], q_heads, kv_heads, head_dim, scale or 0.0),
               "b2b_attn_plan_create")
        self._h = h
        self._torch_dtype = getattr(torch, _TYPES[dtype])
        self.device_index = _current_device()
        self._workspace_sizes = {}
        # What the binding's calls need to know of the plan.  They take the
        # common call, with no tensors for the results and no stream, and return
        # None where anything is not as they want it: the same in Python below
        # finds out what.
        self._bound = _binding.bind(h.value, dtype == "bf16", q_heads, kv_heads, head_dim, self.device_index)

    # -- checks ------------------------------------------------------------
    # The runs test a tensor's type, layout and device in one expression and
    # come here only to say what is wrong: a call's checks cost about as much
    # as its launch.
    def _refuse(self, name, t, heads, dims):
        if t.dtype is not self._torch_dtype:
            raise TypeError(f"{name}: {t.dtype} given, {self._torch_dtype} expected")
        shape = t.shape
        if len(shape) != dims or shape[-2] != heads or shape[-1] != self.head_dim:
            raise ValueError(f"{name}: shape {tuple(shape)} given, {'[blocks, ' if dims == 4 else '['}rows, {heads}, "
                             f"{self.head_dim}] expected")
        self._placed(name, t)
        raise ValueError(f"{name}: the elements of a head must be consecutive (last stride {t.stride(-1)})")

    def _packed(self, name, t, heads):
        """Rows and arguments of a [rows][heads][dim] tensor."""
        shape, stride = t.shape, t.stride()
        if (t.dtype is not self._torch_dtype or len(shape) != 3 or shape[1] != heads or shape[2] != self.head_dim
                or stride[2] != 1 or t.get_device() != self.device_index):
            self._refuse(name, t, heads, 3)
        return shape[0], t.data_ptr(), stride[0], stride[1]

    def _blocks(self, name, t):
        """Blocks, rows and arguments of a [blocks][rows][heads][dim] tensor."""
        shape, stride = t.shape, t.stride()
        if (t.dtype is not self._torch_dtype or len(shape) != 4 or shape[2] != self.kv_heads or shape[3] != self.head_dim
                or stride[3] != 1 or t.get_device() != self.device_index):
            self._refuse(name, t, self.kv_heads, 4)
        return shape[0], shape[1], t.data_ptr(), stride[1], stride[2], stride[0]

    def _no_gradient(self, *inputs):
        if torch.is_grad_enabled() and any(t.requires_grad for t in inputs):
            raise RuntimeError(f"{type(self).__name__} is inference-only: its output has no gradient "
                               "(run it under torch.no_grad())")

    def _placed(self, name, t):
        if t.get_device() != self.device_index:  # (-1 for a CPU tensor)
            raise ValueError(f"{name} is on {t.device}, the plan on cuda:{self.device_index}")

    def _counts(self, name, t, n, dims=1):
        """A dense int32 array of n entries (or n rows of any width); returns its extent and address."""
        shape = t.shape
        if t.dtype is not torch.int32:
            raise TypeError(f"{name}: {t.dtype} given, torch.int32 expected")
        if len(shape) != dims or (n is not None and shape[0] != n) or not t.is_contiguous():
            raise ValueError(f"{name}: shape {tuple(shape)} given, a contiguous array of "
                             f"{n if dims == 1 else f'{n} rows'} expected")
        if t.get_device() != self.device_index:
            self._placed(name, t)
        return shape[-1], t.data_ptr()

    def _results(self, q, tokens, out, lse, return_lse):
        """Output and LSE of one run with the output's arguments and the LSE's address."""
        if out is None:
            out = q.new_empty((tokens, self.q_heads, self.head_dim))
            args = out.data_ptr(), self.q_heads * self.head_dim, self.head_dim
        else:
            rows, *args = self._packed("out", out, self.q_heads)
            if rows != tokens:
                raise ValueError(f"out: {rows} rows given, {tokens} expected")
        if lse is not None:
            if lse.dtype is not torch.float32:
                raise TypeError(f"lse: {lse.dtype} given, torch.float32 expected")
            if tuple(lse.shape) != (tokens, self.q_heads) or not lse.is_contiguous():
                raise ValueError(f"lse: shape {tuple(lse.shape)} given, contiguous {(tokens, self.q_heads)} expected")
            self._placed("lse", lse)
        elif return_lse:
            lse = torch.empty((tokens, self.q_heads), dtype=torch.float32, device=q.device)
        return out, lse, args, 0 if lse is None else lse.data_ptr()

    def _workspace(self, q, sizes, query):
        """Workspace of one run, from the pool of the current stream, and its size."""
        need = self._workspace_sizes.get(sizes)
        if need is None:
            n = ctypes.c_size_t()
            _check(query(self._h, *sizes, ctypes.byref(n)), query.__name__)
            if len(self._workspace_sizes) >= 4096:
                self._workspace_sizes.clear()
            need = self._workspace_sizes[sizes] = n.value
        return (torch.empty(need, dtype=torch.uint8, device=q.device) if need else None), need

    def _kept(self, stream, done, given):
        """Results of a run on `stream`, which is told of the tensors it uses: their memory may belong to another stream,
        and is not handed out anew before `stream` is done with it, even if the caller lets go of them at once.  The
        caller's stream likewise of the results made on `stream`."""
        current = torch.cuda.current_stream(self.device_index)
        if current != stream:
            for t in given:
                if t is not None:
                    t.record_stream(stream)
            for t in done if isinstance(done, tuple) else (done,):
                t.record_stream(current)
        return done

    def _stream(self):
        return _raw_stream(self.device_index) or None

    # -- as the chain plans ------------------------------------------------
    def status(self, stream=None) -> int:
        """Synchronise and return the device status word (0 = OK)."""
        return int(_lib.b2b_attn_plan_device_status(self._h, _stream_handle(stream)))

    def set_wait_budget(self, ns: int) -> None:
        _check(_lib.b2b_attn_plan_set_wait_budget(self._h, int(ns)), "b2b_attn_plan_set_wait_budget")

    def set_debug(self, flags: int) -> None:
        """Test support (see b2b_plan_set_debug in include/b2b.h)."""
        _check(_lib.b2b_attn_plan_set_debug(self._h, int(flags)), "b2b_attn_plan_set_debug")

    def close(self) -> None:
        self._bound = None
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
        Rows of no sequence are not computed: they stay as they are in a given
        ``out`` and are unset in a new one.
        Returns ``out``, or ``(out, lse)`` when ``lse`` is given or asked for.
        """
        if stream is not None:
            with torch.cuda.stream(stream):
                done = self.run(q, k, v, cu_q, cu_k, causal, out, lse, return_lse)
            return self._kept(stream, done, (q, k, v, cu_q, cu_k, out, lse))
        if out is None and lse is None:
            done = _binding.prompt(self._bound, _raw_stream(self.device_index), q, k, v, cu_q, cu_k, causal, return_lse)
            if done is not None:
                return done
        self._no_gradient(q, k, v)
        tokens, *qa = self._packed("q", q, self.q_heads)
        key_rows, *ka = self._packed("k", k, self.kv_heads)
        rows, *va = self._packed("v", v, self.kv_heads)
        if rows != key_rows:
            raise ValueError(f"v: {rows} rows given, {key_rows} expected as k has")
        offsets, cu_qp = self._counts("cu_q", cu_q, None)
        if offsets < 1:
            raise ValueError("cu_q: at least one offset is expected")
        cu_kp = cu_qp if cu_k is None else self._counts("cu_k", cu_k, offsets)[1]
        batch = offsets - 1
        out, lse, oa, lsep = self._results(q, tokens, out, lse, return_lse)
        causal = bool(causal)
        ws, need = self._workspace(q, (batch, tokens, key_rows, causal), _lib.b2b_prompt_attention_workspace)
        r = _prompt_run(batch, tokens, key_rows, causal, *qa, 0, *ka, 0, *va, 0, *oa, 0, cu_qp, cu_kp, lsep,
                        0 if ws is None else ws.data_ptr(), need)
        code = _lib.b2b_prompt_attention_run(self._h, r, self._stream())
        if code:
            _check(code, "b2b_prompt_attention_run")
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
                done = self.run(q, prefix_k, prefix_v, cache_k, cache_v, lengths, page_table, out, lse, return_lse)
            return self._kept(stream, done, (q, prefix_k, prefix_v, cache_k, cache_v, lengths, page_table, out, lse))
        if out is None and lse is None:
            done = _binding.shared(self._bound, _raw_stream(self.device_index), q, prefix_k, prefix_v, cache_k, cache_v,
                                   lengths, page_table, return_lse)
            if done is not None:
                return done
        self._no_gradient(q, prefix_k, prefix_v, cache_k, cache_v)
        tokens, *qa = self._packed("q", q, self.q_heads)
        prefix, *pka = self._packed("prefix_k", prefix_k, self.kv_heads)
        rows, *pva = self._packed("prefix_v", prefix_v, self.kv_heads)
        if rows != prefix:
            raise ValueError(f"prefix_v: {rows} rows given, {prefix} expected as prefix_k has")
        blocks, rows, *cka = self._blocks("cache_k", cache_k)
        vblocks, vrows, *cva = self._blocks("cache_v", cache_v)
        if vblocks != blocks or vrows != rows:
            raise ValueError(f"cache_v: shape {tuple(cache_v.shape)} given, {tuple(cache_k.shape)} expected as cache_k has")
        batch, lengthsp = self._counts("lengths", lengths, None)
        if tokens % batch if batch else tokens:
            raise ValueError(f"q: {tokens} rows given, a multiple of the {batch} requests expected")
        fresh = tokens // batch if batch else 0
        if page_table is None:
            width, tablep, room = 0, 0, rows
            if blocks != batch:
                raise ValueError(f"cache_k: {blocks} requests given, {batch} expected as lengths has")
        else:
            width, tablep = self._counts("page_table", page_table, batch, 2)
            tablep = tablep or lengthsp  # (null means no table, and is the address of one without columns)
            room = width * rows if blocks else 0
        out, lse, oa, lsep = self._results(q, tokens, out, lse, return_lse)
        ws, need = self._workspace(q, (batch, fresh, prefix, room), _lib.b2b_shared_attention_workspace)
        r = _shared_run(batch, fresh, prefix, rows, blocks, width, *qa, 0, *pka, 0, *pva, 0, *cka, *cva, *oa, 0, lengthsp,
                        tablep, lsep, 0 if ws is None else ws.data_ptr(), need)
        code = _lib.b2b_shared_attention_run(self._h, r, self._stream())
        if code:
            _check(code, "b2b_shared_attention_run")
        return out if lse is None else (out, lse)
