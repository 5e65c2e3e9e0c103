"""The gated feed-forward block and the 8-bit matrix product.

``act(x Wg) * (x Wu)`` in one kernel and its product with ``Wd``
(``include/b2b.h``, section "feed-forward"): :class:`GatedFeedForwardPlan` with
16-bit operands, for serving (``run``) and for training (``forward`` and
``backward``); :class:`ScaledFeedForwardPlan` with e4m3 weights that carry a
scale for each block of 128 x 128; :class:`ScaledGemmPlan` for one product of
such operands; :func:`quantize_blocks` brings 16-bit matrices to that form.  A
plan holds the widths; a run takes any number of rows.  Matrices have
consecutive elements in a row (last stride 1), rows on 16-byte boundaries and any
row stride that keeps them there, so a column range of a wider buffer will do.
Gradients are computed by ``backward`` alone: inputs that require a gradient, and
tensors to write into that do, are refused where gradients are recorded, and so
are those with a forward-mode tangent.  There is no CPU path.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import struct
import warnings

from . import DTYPES, _check, _current_device, _differentiated, _lib, _stream_handle, library_path

__all__ = ["GatedFeedForwardPlan", "ScaledFeedForwardPlan", "ScaledGemmPlan", "quantize_blocks", "ACTIVATIONS"]

ACTIVATIONS = {"silu": 0, "gelu": 1}  # b2b_activation_t; gelu in its tanh form
BLOCK = 128
_TYPES = {"f16": "float16", "bf16": "bfloat16"}
_INFERENCE, _TRAINING, _BACKWARD = 0, 1, 2  # B2B_FFN_*

# Set when the first plan is made (_load): the package's other parts need neither torch nor the compiled module.
torch = _raw_stream = _increment_version = _binding = None

# The argument structures, whose members all take eight bytes (b2b_matrix_t: data, row_stride; b2b_scales_t: data,
# row_stride, block_stride), as the C functions read them.
_forward_run = struct.Struct("15q").pack   # tokens; x, w_gate, w_up, w_down, out; kept, bytes; workspace, bytes
_backward_run = struct.Struct("24q").pack  # tokens, accumulate; dy, x, three weights; kept, bytes; four gradients; workspace, bytes
_scaled_run = struct.Struct("22q").pack    # tokens; x, three weights, out; three scales; workspace, bytes
_product_run = struct.Struct("15q").pack   # rows; a, b, out; two scales; workspace, bytes
_matrix = struct.Struct("2q").pack
_scales = struct.Struct("3q").pack


class _NoBinding:
    """In the compiled module's place where there is none: every call takes the way through Python."""

    @staticmethod
    def bind(*_):
        return None

    run = forward = backward = scaled_ffn = scaled_gemm = bind


def _load_binding():
    """The module that passes tensors to the C functions (binding/feedforward.cpp), if it is there for this torch."""
    path = os.path.join(os.path.dirname(library_path()), "ffn_binding.so")
    try:
        loader = importlib.machinery.ExtensionFileLoader("ffn_binding", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("ffn_binding", loader))
        loader.exec_module(module)
        if not torch.__version__.startswith(module.torch_version):
            raise ImportError(f"built for torch {module.torch_version}, this is {torch.__version__}")
    except ImportError as e:
        warnings.warn(f"{path}: {e}; feed-forward calls take some microseconds longer without it "
                      "(python fusion_b2b_gemm_gb300/_build.py)", RuntimeWarning, stacklevel=5)
        return _NoBinding
    module.connect(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
        _lib.b2b_ffn_workspace, _lib.b2b_ffn_kept_bytes, _lib.b2b_ffn_forward, _lib.b2b_ffn_backward, _lib.b2b_scaled_ffn_run,
        _lib.b2b_scaled_gemm_run)))
    return module


def _load():
    global torch, _raw_stream, _increment_version, _binding
    if _binding is None:
        import torch
        # (the public torch.cuda.current_stream() builds an object each time, 3 us)
        _raw_stream = torch._C._cuda_getCurrentRawStream
        _increment_version = torch.autograd.graph.increment_version
        _binding = _load_binding()


def _refuse(name, t, dtype, rows, cols, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: {type(t).__name__} given, a tensor expected")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: {t.dtype} given, {dtype} expected")
    shape = tuple(t.shape)
    if len(shape) != 2 or shape[1] != cols or (rows is not None and shape[0] != rows):
        raise ValueError(f"{name}: shape {shape} given, [{'rows' if rows is None else rows}, {cols}] expected")
    if t.get_device() != device:  # (-1 for a CPU tensor)
        raise ValueError(f"{name} is on {t.device}, the plan on cuda:{device}")
    raise ValueError(f"{name}: the elements of a row must be consecutive (last stride {t.stride(1)})")


def _rows(name, t, dtype, rows, cols, device):
    """Rows, address and row stride of a matrix of so many columns."""
    if t.__class__ is torch.Tensor or isinstance(t, torch.Tensor):
        shape, stride = t.shape, t.stride()
        if (t.dtype is dtype and len(shape) == 2 and shape[1] == cols and (rows is None or shape[0] == rows)
                and (stride[1] == 1 or cols == 1) and t.get_device() == device):
            return shape[0], t.data_ptr(), stride[0]
    _refuse(name, t, dtype, rows, cols, device)


def _scale(name, t, rows, blocks, device):
    """Address and strides of the scales of rows (or row blocks) x blocks; any strides."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or tuple(t.shape) != (rows, blocks) or t.get_device() != device:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: {type(t).__name__} given, a tensor expected")
        if t.dtype is not torch.float32:
            raise TypeError(f"{name}: {t.dtype} given, torch.float32 expected")
        if tuple(t.shape) != (rows, blocks):
            raise ValueError(f"{name}: shape {tuple(t.shape)} given, {(rows, blocks)} expected")
        raise ValueError(f"{name} is on {t.device}, the plan on cuda:{device}")
    return (t.data_ptr(), *t.stride())


def _kept(stream, device, done, given):
    """Results of a run on `stream`, which is told of the tensors it uses: their memory may belong to another stream, and
    is not handed out anew before `stream` is done with it.  The caller's stream likewise of the results made on `stream`."""
    current = torch.cuda.current_stream(device)
    if current != stream:
        for t in given:
            if t is not None:
                t.record_stream(stream)
        for t in done:
            if t is not None:
                t.record_stream(current)


def _written(*given):
    """Tells autograd that a call has changed tensors it was given, so that none of them passes for what was saved of it."""
    changed = [t for t in given if t is not None and not t.is_inference()]
    if changed:
        _increment_version(changed)


_WITHOUT = "(run it under torch.no_grad(), on the primals of dual tensors)"


def _blocks(n):
    return -(-n // BLOCK)


class _Plan:
    """Widths and status word of one kind of operator.  Bound to the GPU that is current now."""

    def __init__(self, dtype, create, sizes, *args):
        if dtype not in _TYPES:
            raise ValueError(f"unknown dtype {dtype!r}; one of {sorted(_TYPES)}")
        _load()
        self.dtype = dtype
        h = ctypes.c_void_p()
        _check(create(ctypes.byref(h), DTYPES[dtype], *(n for n in sizes if n is not None), *args), create.__name__)
        self._h = h
        self._torch_dtype = getattr(torch, _TYPES[dtype])
        self.device_index = _current_device()
        self._bind_args = h.value, dtype == "bf16", *(n or 0 for n in sizes), self.device_index
        self._bind()

    def _bind(self):
        """Without the sizes of workspaces that are known so far, which depend on the plan's flags."""
        self._workspace_sizes = {}
        # What the binding's calls need to know of the plan.  They take the
        # common call, with no tensors for the results and no stream, and return
        # None where anything is not as they want it: the same in Python below
        # finds out what.
        self._bound = _binding.bind(*self._bind_args)

    def _no_gradient(self, *tensors):
        """Of inputs, and of tensors that results are written into."""
        if _differentiated(*tensors):
            raise RuntimeError(f"{type(self).__name__} records no gradient for its outputs {_WITHOUT}")

    def _workspace(self, like, rows, which=_INFERENCE):
        """Workspace of one run, from the pool of the current stream, with its address and size."""
        need = self._workspace_sizes.get((rows, which))
        if need is None:
            n = ctypes.c_size_t()
            _check(_lib.b2b_ffn_workspace(self._h, rows, which, ctypes.byref(n)), "b2b_ffn_workspace")
            if len(self._workspace_sizes) >= 4096:
                self._workspace_sizes.clear()
            need = self._workspace_sizes[rows, which] = n.value
        ws = torch.empty(need, dtype=torch.uint8, device=like.device) if need else None
        return ws, 0 if ws is None else ws.data_ptr(), need

    def _call(self, function, args):
        code = function(self._h, args, _raw_stream(self.device_index) or None)
        if code:
            _check(code, function.__name__)

    def _new(self, like, rows, cols):
        return torch.empty((rows, cols), dtype=self._torch_dtype, device=like.device)

    # -- as the chain plans ------------------------------------------------
    def status(self, stream=None) -> int:
        """Synchronise and return the device status word (0 = OK)."""
        return int(_lib.b2b_ffn_plan_device_status(self._h, _stream_handle(stream)))

    def set_wait_budget(self, ns: int) -> None:
        _check(_lib.b2b_ffn_plan_set_wait_budget(self._h, int(ns)), "b2b_ffn_plan_set_wait_budget")

    def set_debug(self, flags: int) -> None:
        """Test support (see b2b_plan_set_debug and B2B_DEBUG_PAIR_KERNEL in include/b2b.h)."""
        _check(_lib.b2b_ffn_plan_set_debug(self._h, int(flags)), "b2b_ffn_plan_set_debug")
        self._bind()

    def close(self) -> None:
        self._bound = None
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            _lib.b2b_ffn_plan_destroy(h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _activation(name):
    if name not in ACTIVATIONS:
        raise ValueError(f"unknown activation {name!r}; one of {sorted(ACTIVATIONS)}")
    return ACTIVATIONS[name]


class GatedFeedForwardPlan(_Plan):
    """``(act(x Wg) * (x Wu)) Wd`` with 16-bit operands, and its gradients.

    ``dtype`` is "f16" or "bf16"; weights are ``w_gate``, ``w_up`` [width,
    hidden] and ``w_down`` [hidden, out_width] (default: width), all multiples
    of 8; ``activation`` "silu" or "gelu" (tanh form).  Hidden activations, and
    gradients of the projections, are rounded to the plan's type: in "f16" a
    magnitude of 65520 or more becomes an infinity.
    """

    def __init__(self, dtype: str, width: int, hidden: int, out_width: int | None = None, activation: str = "silu"):
        out_width = width if out_width is None else out_width
        super().__init__(dtype, _lib.b2b_ffn_plan_create, (width, hidden, out_width), _activation(activation))
        self.width, self.hidden, self.out_width, self.activation = width, hidden, out_width, activation

    def _operands(self, x, w_gate, w_up, w_down):
        dt, dev = self._torch_dtype, self.device_index
        tokens, *xa = _rows("x", x, dt, None, self.width, dev)
        return tokens, (*xa, *_rows("w_gate", w_gate, dt, self.width, self.hidden, dev)[1:],
                        *_rows("w_up", w_up, dt, self.width, self.hidden, dev)[1:],
                        *_rows("w_down", w_down, dt, self.hidden, self.out_width, dev)[1:])

    def _result(self, x, tokens, out):
        if out is None:
            out = self._new(x, tokens, self.out_width)
        return out, _rows("out", out, self._torch_dtype, tokens, self.out_width, self.device_index)[1:]

    def run(self, x, w_gate, w_up, w_down, out=None, stream=None):
        """The block's output [tokens, out_width] for ``x`` [tokens, width], on ``stream`` (default: torch's current one)."""
        if stream is not None:
            with torch.cuda.stream(stream):
                done = self.run(x, w_gate, w_up, w_down, out)
            _kept(stream, self.device_index, (done,), (x, w_gate, w_up, w_down, out))
            return done
        if out is None:
            done = _binding.run(self._bound, _raw_stream(self.device_index), x, w_gate, w_up, w_down)
            if done is not None:
                return done
        tokens, operands = self._operands(x, w_gate, w_up, w_down)
        given = out
        out, oa = self._result(x, tokens, out)
        self._no_gradient(x, w_gate, w_up, w_down, out)
        ws, wsp, need = self._workspace(x, tokens)
        self._call(_lib.b2b_ffn_forward, _forward_run(tokens, *operands, *oa, 0, 0, wsp, need))
        _written(given)
        return out

    def forward(self, x, w_gate, w_up, w_down, out=None, kept=None, stream=None):
        """As ``run``; returns ``(out, kept)``.  ``kept`` is what ``backward`` needs, a torch.uint8 tensor whose order is the
        kernels' own (10 bytes a token and hidden column); one that an earlier call on as many tokens returned may be given
        to be written again."""
        if stream is not None:
            with torch.cuda.stream(stream):
                done = self.forward(x, w_gate, w_up, w_down, out, kept)
            _kept(stream, self.device_index, done, (x, w_gate, w_up, w_down, out, kept))
            return done
        if out is None and kept is None:
            done = _binding.forward(self._bound, _raw_stream(self.device_index), x, w_gate, w_up, w_down)
            if done is not None:
                return done
        tokens, operands = self._operands(x, w_gate, w_up, w_down)
        given = out, kept
        out, oa = self._result(x, tokens, out)
        self._no_gradient(x, w_gate, w_up, w_down, out)
        if kept is None:
            n = ctypes.c_size_t()
            _check(_lib.b2b_ffn_kept_bytes(self._h, tokens, ctypes.byref(n)), "b2b_ffn_kept_bytes")
            kept = torch.empty(n.value, dtype=torch.uint8, device=x.device)
        ka = self._kept_args(kept)
        if tokens == 0:  # (no address: nothing to keep)
            return out, kept
        ws, wsp, need = self._workspace(x, tokens, _TRAINING)
        self._call(_lib.b2b_ffn_forward, _forward_run(tokens, *operands, *oa, *ka, wsp, need))
        _written(*given)
        return out, kept

    def _kept_args(self, kept):
        if not isinstance(kept, torch.Tensor) or kept.dtype is not torch.uint8:
            raise TypeError(f"kept: {getattr(kept, 'dtype', type(kept).__name__)} given, what forward() returned expected")
        if kept.dim() != 1 or not kept.is_contiguous():
            raise ValueError(f"kept: shape {tuple(kept.shape)} given, what forward() returned expected")
        if kept.get_device() != self.device_index:
            raise ValueError(f"kept is on {kept.device}, the plan on cuda:{self.device_index}")
        return kept.data_ptr(), kept.numel()

    def backward(self, dy, x, w_gate, w_up, w_down, kept, input_grad: bool = True, weight_grads=True, stream=None):
        """Gradients ``(dx, dw_gate, dw_up, dw_down)`` for ``dy``, the gradient of ``forward``'s output.

        ``kept`` is what ``forward`` returned for the same ``x`` and weights.
        Without ``input_grad`` dx is None.  ``weight_grads``: True for new
        tensors of the plan's type, False for none, or three fp32 tensors of the
        weights' shapes, to which the gradients are added (and which are
        returned); a None among them leaves that one out.
        """
        if stream is not None:
            with torch.cuda.stream(stream):
                done = self.backward(dy, x, w_gate, w_up, w_down, kept, input_grad, weight_grads)
            _kept(stream, self.device_index, done,
                  (dy, x, w_gate, w_up, w_down, kept, *(() if isinstance(weight_grads, bool) else done[1:])))
            return done
        if weight_grads is True:
            done = _binding.backward(self._bound, _raw_stream(self.device_index), dy, x, w_gate, w_up, w_down, kept, input_grad)
            if done is not None:
                return done
        tokens, (xp, xs, *weights) = self._operands(x, w_gate, w_up, w_down)
        dya = _rows("dy", dy, self._torch_dtype, tokens, self.out_width, self.device_index)[1:]
        ka = self._kept_args(kept)
        accumulate = not isinstance(weight_grads, bool)
        grads = tuple(weight_grads) if accumulate else ()
        self._no_gradient(dy, x, w_gate, w_up, w_down, *[g for g in grads if isinstance(g, torch.Tensor)])
        dx = self._new(x, tokens, self.width) if input_grad else None
        shapes = (self.width, self.hidden), (self.width, self.hidden), (self.hidden, self.out_width)
        if accumulate:
            if len(grads) != 3:
                raise ValueError(f"weight_grads: {len(grads)} tensors given, three expected")
        elif weight_grads:
            grads = tuple(self._new(x, *shape) for shape in shapes)
        else:
            grads = (None,) * 3
        ga = [] if dx is None else [dx.data_ptr(), dx.stride(0)]
        ga = ga or [0, 0]
        for name, g, shape in zip(("w_gate", "w_up", "w_down"), grads, shapes):
            ga += (0, 0) if g is None else _rows(f"gradient of {name}", g, torch.float32 if accumulate else self._torch_dtype,
                                                 *shape, self.device_index)[1:]
        ws, wsp, need = self._workspace(x, tokens, _BACKWARD)
        self._call(_lib.b2b_ffn_backward, _backward_run(tokens, accumulate, *dya, xp, xs, *weights, *ka, *ga, wsp, need))
        if accumulate:
            _written(*grads)
        return (dx, *grads)


class ScaledFeedForwardPlan(_Plan):
    """``(act(x Wg^T) * (x Wu^T)) Wd^T`` with e4m3 weights, for serving.

    ``dtype`` ("f16" or "bf16") is that of the activations; weights are
    torch.float8_e4m3fn ``w_gate``, ``w_up`` [hidden, width] and ``w_down``
    [out_width, hidden] (default: width), extents multiples of 16.
    """

    def __init__(self, dtype: str, width: int, hidden: int, out_width: int | None = None, activation: str = "silu"):
        out_width = width if out_width is None else out_width
        super().__init__(dtype, _lib.b2b_scaled_ffn_plan_create, (width, hidden, out_width), _activation(activation))
        self.width, self.hidden, self.out_width, self.activation = width, hidden, out_width, activation

    def run(self, x, w_gate, gate_scale, w_up, up_scale, w_down, down_scale, out=None, stream=None):
        """The block's output [tokens, out_width] for 16-bit ``x`` [tokens, width], on ``stream`` (default: torch's current
        one).

        Scales are fp32, one for each block of 128 x 128: ``gate_scale`` and
        ``up_scale`` [hidden / 128, width / 128], ``down_scale`` [out_width /
        128, hidden / 128], rounded up.  ``x`` and the hidden activations are
        quantised as :func:`quantize_blocks` does.
        """
        if stream is not None:
            with torch.cuda.stream(stream):
                done = self.run(x, w_gate, gate_scale, w_up, up_scale, w_down, down_scale, out)
            _kept(stream, self.device_index, (done,), (x, w_gate, gate_scale, w_up, up_scale, w_down, down_scale, out))
            return done
        if out is None:
            done = _binding.scaled_ffn(self._bound, _raw_stream(self.device_index), x, w_gate, gate_scale, w_up, up_scale, w_down,
                                       down_scale)
            if done is not None:
                return done
        dev, f8 = self.device_index, torch.float8_e4m3fn
        d, f, o = self.width, self.hidden, self.out_width
        tokens, *xa = _rows("x", x, self._torch_dtype, None, d, dev)
        weights = (*_rows("w_gate", w_gate, f8, f, d, dev)[1:], *_rows("w_up", w_up, f8, f, d, dev)[1:],
                   *_rows("w_down", w_down, f8, o, f, dev)[1:])
        scales = (*_scale("gate_scale", gate_scale, _blocks(f), _blocks(d), dev),
                  *_scale("up_scale", up_scale, _blocks(f), _blocks(d), dev),
                  *_scale("down_scale", down_scale, _blocks(o), _blocks(f), dev))
        given = out
        if out is None:
            out = self._new(x, tokens, o)
        oa = _rows("out", out, self._torch_dtype, tokens, o, dev)[1:]
        self._no_gradient(x, w_gate, w_up, w_down, gate_scale, up_scale, down_scale, out)
        ws, wsp, need = self._workspace(x, tokens)
        self._call(_lib.b2b_scaled_ffn_run, _scaled_run(tokens, *xa, *weights, *oa, *scales, wsp, need))
        _written(given)
        return out


class ScaledGemmPlan(_Plan):
    """``a b^T`` of e4m3 matrices with scales, ``a`` [rows, k] one for each 128 of a row, ``b`` [n, k] one for each block
    of 128 x 128.  ``dtype`` ("f16" or "bf16") is that of the result; ``k`` is a multiple of 16, ``n`` of 8."""

    def __init__(self, dtype: str, k: int, n: int):
        super().__init__(dtype, _lib.b2b_scaled_gemm_plan_create, (k, None, n))
        self.k, self.n = k, n

    def run(self, a, a_scale, b, b_scale, out=None, stream=None):
        """The product [rows, n], on ``stream`` (default: torch's current one).  ``a_scale`` is fp32 [rows, k / 128],
        ``b_scale`` [n / 128, k / 128], rounded up, with any strides; a column of ``a_scale`` is best consecutive, as
        :func:`quantize_blocks` lays it out.  The two scales of a block are multiplied with each other, in fp32, before
        they are applied."""
        if stream is not None:
            with torch.cuda.stream(stream):
                done = self.run(a, a_scale, b, b_scale, out)
            _kept(stream, self.device_index, (done,), (a, a_scale, b, b_scale, out))
            return done
        if out is None:
            done = _binding.scaled_gemm(self._bound, _raw_stream(self.device_index), a, a_scale, b, b_scale)
            if done is not None:
                return done
        dev, f8 = self.device_index, torch.float8_e4m3fn
        rows, *aa = _rows("a", a, f8, None, self.k, dev)
        ba = _rows("b", b, f8, self.n, self.k, dev)[1:]
        scales = (*_scale("a_scale", a_scale, rows, _blocks(self.k), dev),
                  *_scale("b_scale", b_scale, _blocks(self.n), _blocks(self.k), dev))
        given = out
        if out is None:
            out = self._new(a, rows, self.n)
        oa = _rows("out", out, self._torch_dtype, rows, self.n, dev)[1:]
        self._no_gradient(a, b, a_scale, b_scale, out)
        ws, wsp, need = self._workspace(a, rows)
        self._call(_lib.b2b_scaled_gemm_run, _product_run(rows, *aa, *ba, *oa, *scales, wsp, need))
        _written(given)
        return out


def quantize_blocks(x, block_rows: int = 1, stream=None):
    """``(values, scale)``: a 16-bit matrix as torch.float8_e4m3fn with fp32 scales, one for each block of ``block_rows``
    (1: activations, 128: weights) by 128.

    A scale is the smallest power of two that leaves no magnitude of its block
    above 448; ``values * scale`` stands for x.  ``scale`` is [rows /
    block_rows, columns / 128], rounded up; for single rows its columns are
    consecutive.  A block that holds an infinity or a NaN becomes NaN.  The
    columns are a multiple of 8.
    """
    _load()
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x: a matrix [rows, columns] expected")
    if stream is not None:
        with torch.cuda.stream(stream):
            done = quantize_blocks(x, block_rows)
        _kept(stream, x.get_device(), done, (x,))
        return done
    dtype = {torch.float16: "f16", torch.bfloat16: "bf16"}.get(x.dtype)
    if dtype is None:
        raise TypeError(f"x: {x.dtype} given, torch.float16 or torch.bfloat16 expected")
    if block_rows not in (1, BLOCK):
        raise ValueError(f"block_rows {block_rows!r}: 1 or {BLOCK} expected")
    if _differentiated(x):
        raise RuntimeError(f"quantize_blocks records no gradient for its outputs {_WITHOUT}")
    rows, cols = x.shape
    device = x.get_device()
    if device < 0:
        raise ValueError(f"x is on {x.device}, a GPU expected")
    if cols > 1 and x.stride(1) != 1:
        raise ValueError(f"x: the elements of a row must be consecutive (last stride {x.stride(1)})")
    scale_rows, blocks = -(-rows // block_rows), _blocks(cols)
    q = torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device=x.device)
    if block_rows == 1:
        scale = torch.empty((blocks, rows), dtype=torch.float32, device=x.device).t()
    else:
        scale = torch.empty((scale_rows, blocks), dtype=torch.float32, device=x.device)
    with torch.cuda.device(device):
        _check(_lib.b2b_quantize_blocks(DTYPES[dtype], rows, cols, block_rows, _matrix(x.data_ptr(), x.stride(0)),
                                        _matrix(q.data_ptr(), q.stride(0)), _scales(scale.data_ptr(), *scale.stride()),
                                        _raw_stream(device) or None), "b2b_quantize_blocks")
    return q, scale
