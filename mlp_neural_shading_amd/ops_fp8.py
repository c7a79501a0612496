"""Torch form of the 8-bit operators in ``include/mlp_ops_fp8.h``, beside the 16-bit ones of ``ops``: the norm of
the residual stream (``rms_norm``), the rounding to blocks of E4M3 (``quantize``), one affine layer (``linear``) and
the experts' layers on routed rows (``expert_linear``).

``Quantized`` pairs E4M3 values with an FP32 scale for each block of 128 columns, of one row (activations) or of 128
rows (weights).  As in ``ops``: tensors are checked, outputs and scratch memory come from torch's allocator on the
current stream, nothing here computes or waits, and inputs that require gradients are refused.  The usual call of each
(new outputs, the current device) goes through an extension in C++, ``_torch_fp8``, which leaves any other to the
functions here; where it is not built, they take every call.  A layer of experts with its weights rounded once::

    w1, w2 = ops_fp8.quantize(w1, block_rows=128, gated=True), ops_fp8.quantize(w2, block_rows=128)

    h, q, stream = ops_fp8.rms_norm(y, g, residual=stream, out="both")
    index, weight = ops.route(ops.linear(h, w_router, out_dtype=torch.float32), k)
    plan = ops.dispatch(index, experts)
    a = ops_fp8.expert_linear(q, w1, plan, k=k, act="silu", gated=True, out_dtype=torch.float8_e4m3fn)
    y = ops_fp8.expert_linear(a, w2, plan, k=k, rows="slots", combine=True, weight=weight)
"""
from __future__ import annotations

import ctypes
import warnings
from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad

from .ops import (ACTIVATIONS, DTYPES, Dispatch, _call, _choice, _count, _f32, _FLOATS, _i32, _i64, _matrix, _out_dtype,
                  _p, _packer, _tensor, _u64, _vector, _workspace, _written)

try:
    from . import _torch_fp8 as _usual
except ImportError as e:
    class _usual:
        """In its place: leaves every call to the functions here."""
        rms_norm = quantize = linear = expert_linear = staticmethod(lambda *a: None)
    if not isinstance(e, ModuleNotFoundError):
        warnings.warn("the extension _torch_fp8 does not load, build it again: %s" % e)

MLP_DTYPE_FP8 = 3
BLOCK = 128
FP8 = torch.float8_e4m3fn


class RmsNormArgs(ctypes.Structure):
    _fields_ = [("rows", _i64), ("width", _i32), ("dtype", _i32), ("out_dtype", _i32), ("eps", _f32), ("x", _p),
                ("ldx", _i64), ("residual", _p), ("ldr", _i64), ("weight", _p), ("total", _p), ("ldt", _i64), ("y", _p),
                ("ldy", _i64), ("values", _p), ("ldv", _i64), ("scales", _p), ("lds", _i64)]


class QuantizeArgs(ctypes.Structure):
    _fields_ = [("rows", _i64), ("count", _i32), ("width", _i32), ("dtype", _i32), ("block_rows", _i32), ("x", _p),
                ("ldx", _i64), ("x_stride", _i64), ("values", _p), ("ldv", _i64), ("v_stride", _i64), ("scales", _p),
                ("lds", _i64), ("s_stride", _i64)]


class Fp8LinearArgs(ctypes.Structure):
    _fields_ = [("rows", _i64), ("in_width", _i32), ("out_width", _i32), ("out_dtype", _i32), ("act", _i32),
                ("gated", _i32), ("x", _p), ("ldx", _i64), ("x_scale", _p), ("ldxs", _i64), ("w", _p), ("ldw", _i64),
                ("w_scale", _p), ("ldws", _i64), ("bias", _p), ("residual", _p), ("ldr", _i64), ("y", _p), ("ldy", _i64),
                ("y_scale", _p), ("ldys", _i64), ("workspace", _p), ("workspace_bytes", _u64)]


class Fp8ExpertLinearArgs(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("k", _i32), ("experts", _i32), ("in_width", _i32), ("out_width", _i32),
                ("out_dtype", _i32), ("act", _i32), ("gated", _i32), ("x_slots", _i32), ("combine", _i32), ("x", _p),
                ("ldx", _i64), ("x_scale", _p), ("ldxs", _i64), ("w", _p), ("ldw", _i64), ("w_stride", _i64),
                ("w_scale", _p), ("ldws", _i64), ("ws_stride", _i64), ("bias", _p), ("offsets", _p), ("slots", _p),
                ("places", _p), ("weight", _p), ("residual", _p), ("ldr", _i64), ("y", _p), ("ldy", _i64),
                ("y_scale", _p), ("ldys", _i64), ("workspace", _p), ("workspace_bytes", _u64)]


_norm_args, _quantize_args, _linear_args, _expert_linear_args = map(
    _packer, (RmsNormArgs, QuantizeArgs, Fp8LinearArgs, Fp8ExpertLinearArgs))

_OUT = {**DTYPES, FP8: MLP_DTYPE_FP8}
_CODE = (FP8,)
_SCALE = (torch.float32,)


class Quantized(NamedTuple):
    """``values`` float8_e4m3fn [..., rows, width], rows contiguous; ``scales`` float32 [..., rows, blocks] of
    blocks of 128 columns, or [..., blocks of 128 rows, blocks]."""
    values: torch.Tensor
    scales: torch.Tensor


class Normed(NamedTuple):
    """``y`` in 16 or 32 bits, ``quantized`` in 8, ``total`` = x + residual; None where not asked for."""
    y: Optional[torch.Tensor]
    quantized: Optional[Quantized]
    total: Optional[torch.Tensor]


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _new(rows, width, device):
    """Values in rows of whole 16 bytes, which the products read fastest, and their scales."""
    pad = width + 15 & ~15
    values = torch.empty(rows, pad, dtype=FP8, device=device)
    return values if pad == width else values[:, :width], torch.empty(rows, _blocks(width), dtype=torch.float32, device=device)


def _quantized(name, q):
    if not isinstance(q, tuple) or len(q) != 2:
        raise ValueError("%s must be Quantized" % name)
    return q


def rms_norm(x, weight=None, *, residual=None, total=None, eps=1e-6, out="same", out_dtype=None) -> Normed:
    """``t / sqrt(mean(t^2) + eps) * weight`` of ``t = x + residual``, each row by itself, in FP32 and rounded once.

    ``x`` and ``residual`` [rows, width] and ``weight`` [width] have one type, float16, bfloat16 or float32; their sum
    is rounded to it and comes back as ``total`` (a new tensor, or the one given, which may be x or residual itself).
    ``out``: "same" gives ``y`` in x's type (or ``out_dtype`` float32), "fp8" the normed rows ``quantized``, "both" both."""
    if out not in ("same", "fp8", "both"):
        raise ValueError("out must be same, fp8 or both, got %r" % (out,))
    if total is None and forward_ad._current_level < 0 and (out_dtype is None or out_dtype is torch.float32):
        r = _usual.rms_norm(x, weight, residual, eps, out != "fp8", out != "same", out_dtype is not None)
        if r is not None:
            y, values, scales, total = r
            return Normed(y, None if values is None else Quantized(values, scales), total)
    ldx = _matrix("x", x, _FLOATS)
    rows, width = x.shape
    device, dtype = x.device, x.dtype
    y_dtype = _out_dtype(dtype, out_dtype)
    ldr = ldt = 0
    given = total is not None
    if residual is not None:
        ldr = _matrix("residual", residual, (dtype,), device, rows, width)
        if given:
            ldt = _matrix("total", total, (dtype,), device, rows, width)
        else:
            total = torch.empty(rows, width, dtype=dtype, device=device)
            ldt = width
    elif given:
        raise ValueError("total goes with a residual")
    y = values = scales = None
    if out != "fp8":
        y = torch.empty(rows, width, dtype=y_dtype, device=device)
    if out != "same":
        values, scales = _new(rows, width, device)
    a = _norm_args(rows, width, DTYPES[dtype], DTYPES[y_dtype], eps, x.data_ptr(), ldx,
                   0 if residual is None else residual.data_ptr(), ldr,
                   0 if weight is None else _vector("weight", weight, dtype, device, width),
                   0 if total is None else total.data_ptr(), ldt, 0 if y is None else y.data_ptr(), width,
                   0 if values is None else values.data_ptr(), 0 if values is None else values.stride(0) if rows > 1 else width,
                   0 if scales is None else scales.data_ptr(), _blocks(width))
    _call("mlp_rms_norm", a, device)
    if given:
        _written(total)
    return Normed(y, None if values is None else Quantized(values, scales), total)


def quantize(x, *, block_rows=1, gated=False) -> Quantized:
    """``x`` [rows, width], or several matrices [count, rows, width], in blocks of 8 bits; float16, bfloat16 or float32
    with contiguous rows.

    ``block_rows`` 1: a scale for each row and 128 columns (activations); 128: for 128 rows and 128 columns (weights).
    A value is ``v * (1 / scale)``, both rounded in FP32, to E4M3: next to the middle between two numbers it may go to either.
    ``gated``: the weights of a gated layer, whose two halves of the rows are matrices of their own."""
    if not gated and forward_ad._current_level < 0:
        r = _usual.quantize(x, block_rows)
        if r is not None:
            return Quantized(*r)
    block_rows = _count("block_rows", block_rows)
    if block_rows not in (1, BLOCK):
        raise ValueError("block_rows must be 1 or %d, got %d" % (BLOCK, block_rows))
    if isinstance(x, torch.Tensor) and x.dim() == 3:
        _tensor("x", x, 3, _FLOATS)
        count, rows, width = x.shape
        if x.stride(2) != 1 and width > 1:
            raise ValueError("the rows of x must be contiguous")
        ldx, x_stride = x.stride(1) if rows > 1 else width, x.stride(0)
    else:
        ldx = _matrix("x", x, _FLOATS)
        (rows, width), count, x_stride = x.shape, 1, 0
    device = x.device
    halves = 1
    if gated:
        if rows % 2:
            raise ValueError("a gated layer's w has an even number of rows, got %d" % rows)
        halves = 2
    part = rows // halves
    down = part if block_rows == 1 else _blocks(part)
    values, scales = _new(count * rows, width, device)
    if block_rows != 1:
        scales = torch.empty(count * halves * down, _blocks(width), dtype=torch.float32, device=device)
    ldv, lds = values.stride(0), _blocks(width)
    for h in range(halves):
        a = _quantize_args(part, count, width, DTYPES[x.dtype], block_rows, x.data_ptr() + h * part * ldx * x.element_size(), ldx,
                           x_stride, values.data_ptr() + h * part * ldv, ldv, rows * ldv,
                           scales.data_ptr() + h * down * lds * 4, lds, halves * down * lds)
        _call("mlp_quantize", a, device)
    if x.dim() == 3:
        values, scales = values.unflatten(0, (count, rows)), scales.unflatten(0, (count, halves * down))
    return Quantized(values, scales)


def _layer(x, w, bias, gated, experts):
    """The checked operands: device, rows, in, out, experts, the structs' fields of x, of w, and the bias."""
    x, xs = _quantized("x", x)
    w, ws = _quantized("w", w)
    ldx = _matrix("x", x, _CODE)
    rows, k = x.shape
    device = x.device
    ldxs = _matrix("x.scales", xs, _SCALE, device, rows, _blocks(k))
    if experts:
        _tensor("w", w, 3, _CODE, device)
        if w.shape[2] != k or (w.stride(2) != 1 and k > 1):
            raise ValueError("w must be [experts, out, %d] with contiguous rows" % k)
        _tensor("w.scales", ws, 3, _SCALE, device)
        count, wide = w.shape[:2]
        ldw = w.stride(1) if wide > 1 else k
    else:
        ldw = _matrix("w", w, _CODE, device, cols=k)
        count, wide = 1, w.shape[0]
    if gated and wide % 2:
        raise ValueError("a gated layer's w has an even number of rows, got %d" % wide)
    n = wide // 2 if gated else wide
    down = _blocks(n) * (2 if gated else 1)
    if experts:
        if ws.shape != (count, down, _blocks(k)) or (ws.stride(2) != 1 and k > BLOCK):
            raise ValueError("w.scales must be [%d, %d, %d] with contiguous rows, got %s" % (count, down, _blocks(k), list(ws.shape)))
        weights = (w.data_ptr(), ldw, w.stride(0) if count > 1 else 0, ws.data_ptr(), ws.stride(1) if down > 1 else _blocks(k),
                   ws.stride(0) if count > 1 else 0)
    else:
        ldws = _matrix("w.scales", ws, _SCALE, device, down, _blocks(k))
        weights = (w.data_ptr(), ldw, ws.data_ptr(), ldws)
    b = 0 if bias is None else _vector("bias", bias, torch.float32, device, count * wide)
    return device, rows, k, n, count, (x.data_ptr(), ldx, xs.data_ptr(), ldxs), weights, b


def _outputs(out, out_dtype, rows, n, device):
    """(result, y, ldy, y_scale, ldys): new tensors, or the caller's, checked."""
    if out_dtype not in _OUT:
        raise ValueError("out_dtype must be one of %s, got %r" % (", ".join(map(str, _OUT)), out_dtype))
    if out_dtype == FP8:
        if out is None:
            out = Quantized(*_new(rows, n, device))
        y, ys = _quantized("out", out)
        return out, y, _matrix("out", y, _CODE, device, rows, n), ys.data_ptr(), _matrix("out.scales", ys, _SCALE, device, rows, _blocks(n))
    if out is None:
        out = torch.empty(rows, n, dtype=out_dtype, device=device)
        return out, out, max(n, 1), 0, 0
    return out, out, _matrix("out", out, (out_dtype,), device, rows, n), 0, 0


def _done(out, given):
    if given:
        for t in out if isinstance(out, tuple) else (out,):
            _written(t)
    return out


def linear(x: Quantized, w: Quantized, bias=None, *, residual=None, act="none", gated=False, out=None,
           out_dtype=torch.bfloat16):
    """``act(x w^T + bias) + residual``: one affine layer with 8-bit operands, rounded once from an FP32 sum.

    The products of 16-bit outputs are the matrix unit's own, cut 8 at a time to 2^-13 of the largest: in the root mean
    square off by 2^-16 to 2^-14 of the outputs' own, which an output whose products cancel may exceed by far.  Of float32
    and float8_e4m3fn outputs no product is cut, at half the rate; ``include/mlp_ops_fp8.h`` states the bound.

    ``x`` has a scale for each row and 128 columns, ``w`` [out, in] one for each 128 x 128; ``bias`` float32 [out];
    ``act`` one of ``ops.ACTIVATIONS``.  ``gated``: w and bias have 2 * out rows, the gates first, with blocks of their
    own (``quantize(gated=True)``).  ``out_dtype`` float16, bfloat16, float32 (a residual's too, which may be ``out``
    itself), or float8_e4m3fn, which gives ``Quantized`` rows and takes no residual."""
    if out is None and forward_ad._current_level < 0:
        r = _usual.linear(x, w, bias, residual, ACTIVATIONS.get(act), gated, _OUT.get(out_dtype))
        if r is not None:
            return Quantized(*r) if out_dtype is FP8 else r
    device, rows, k, n, _, operand, weights, b = _layer(x, w, bias, gated, False)
    given = out is not None
    out, y, ldy, ys, ldys = _outputs(out, out_dtype, rows, n, device)
    ldr = _matrix("residual", residual, (out_dtype,), device, rows, n) if residual is not None else 0
    a = (rows, k, n, _OUT[out_dtype], _choice("act", act, ACTIVATIONS), 1 if gated else 0, *operand, *weights, b,
         0 if residual is None else residual.data_ptr(), ldr, y.data_ptr(), ldy, ys, ldys)
    packed = _linear_args(*a, 0, 0)
    ws = _workspace("mlp_fp8_linear_workspace", packed, device) if ys else None
    _call("mlp_fp8_linear", packed if ws is None else _linear_args(*a, ws.data_ptr(), ws.numel()), device)
    return _done(out, given)


def expert_linear(x: Quantized, w: Quantized, plan: Dispatch, bias=None, *, k, act="none", gated=False, rows="tokens",
                  combine=False, weight=None, residual=None, out=None, out_dtype=torch.bfloat16):
    """Each routed row through its own expert's layer with 8-bit operands, as ``ops.expert_linear``, with the products of
    ``linear`` here; ``combine`` sums FP32 rows, whose products are cut where ``out_dtype`` has 16 bits.

    ``w`` [experts, out or 2 * out, in] with scales [experts, blocks of 128 rows (of each half), blocks], ``bias``
    float32 [experts, out or 2 * out], ``plan`` from ``ops.dispatch``.  Rows by slot may be float8_e4m3fn: ``Quantized``
    rows for the next layer."""
    if rows not in ("tokens", "slots"):
        raise ValueError("rows must be tokens or slots, got %r" % (rows,))
    if out is None and forward_ad._current_level < 0 and isinstance(plan, Dispatch):
        r = _usual.expert_linear(x, w, *plan, bias, k, ACTIVATIONS.get(act), gated, rows == "slots", combine, weight, residual,
                                 _OUT.get(out_dtype))
        if r is not None:
            return Quantized(*r) if out_dtype is FP8 else r
    k = _count("k", k)
    device, x_rows, k_in, n, experts, operand, weights, b = _layer(x, w, bias, gated, True)
    if not isinstance(plan.places, torch.Tensor) or k < 1 or plan.places.numel() % k:
        raise ValueError("plan.places must hold k = %d places for each token" % k)
    total = plan.places.numel()
    tokens = total // k
    if x_rows != (total if rows == "slots" else tokens):
        raise ValueError("x has %d rows, the plan has %d tokens and %d slots" % (x_rows, tokens, total))
    y_rows = tokens if combine else total
    given = out is not None
    out, y, ldy, ys, ldys = _outputs(out, out_dtype, y_rows, n, device)
    ldr = _matrix("residual", residual, (out_dtype,), device, y_rows, n) if residual is not None else 0
    a = (tokens, k, experts, k_in, n, _OUT[out_dtype], _choice("act", act, ACTIVATIONS), 1 if gated else 0,
         1 if rows == "slots" else 0, 1 if combine else 0, *operand, *weights, b,
         _vector("plan.offsets", plan.offsets, torch.int32, device, experts + 1),
         _vector("plan.slots", plan.slots, torch.int32, device, total),
         _vector("plan.places", plan.places, torch.int32, device, total),
         0 if weight is None else _vector("weight", weight, torch.float32, device, total),
         0 if residual is None else residual.data_ptr(), ldr, y.data_ptr(), ldy, ys, ldys)
    packed = _expert_linear_args(*a, 0, 0)
    ws = _workspace("mlp_fp8_expert_linear_workspace", packed, device) if ys or combine else None
    _call("mlp_fp8_expert_linear", packed if ws is None else _expert_linear_args(*a, ws.data_ptr(), ws.numel()), device)
    return _done(out, given)
