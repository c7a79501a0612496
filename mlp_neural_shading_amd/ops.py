"""Torch form of the single operators in ``include/mlp_ops.h``: one affine layer with its epilogue
(``linear``), the router's choice of experts (``route``), the order of rows by expert (``dispatch``) and
the experts' layers on routed rows (``expert_linear``), beside ``binding.infer`` for whole networks.

Each checks its tensors, takes outputs and scratch memory from torch's allocator on the current stream and
enqueues the HIP kernels there; nothing here computes, and nothing waits.  Inference only: inputs that
require gradients are refused while autograd records, and so are forward-mode duals.  A run of them together, a layer of experts::

    index, weight = ops.route(ops.linear(x, w_router, out_dtype=torch.float32), k)
    plan = ops.dispatch(index, experts)
    h = ops.expert_linear(x, w1, plan, k=k, act="silu", gated=True)
    y = ops.expert_linear(h, w2, plan, k=k, rows="slots", combine=True, weight=weight, residual=x)
"""
from __future__ import annotations

import ctypes
import operator
import struct
from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad
from torch.autograd.graph import increment_version

from . import binding as B

MLP_DTYPE_FP16, MLP_DTYPE_BF16, MLP_DTYPE_FP32 = 0, 1, 2
DTYPES = {torch.float16: MLP_DTYPE_FP16, torch.bfloat16: MLP_DTYPE_BF16, torch.float32: MLP_DTYPE_FP32}
ACTIVATIONS = {"none": 0, "leaky_relu": 1, "relu": 2, "gelu": 3, "silu": 4}
SCORES = {"softmax": 0, "sigmoid": 1}
MLP_OPS_MAX_WIDTH = 1 << 20
MLP_OPS_MAX_EXPERTS = 1024
MLP_OPS_MAX_TOPK = 32

EXPORTED = ("mlp_linear", "mlp_route", "mlp_dispatch_workspace", "mlp_dispatch", "mlp_expert_linear_workspace",
            "mlp_expert_linear")
EXPORTED_FP8 = ("mlp_rms_norm", "mlp_quantize", "mlp_fp8_linear_workspace", "mlp_fp8_linear",
                "mlp_fp8_expert_linear_workspace", "mlp_fp8_expert_linear")  # include/mlp_ops_fp8.h, for ops_fp8

_p, _i32, _i64, _u64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_float


class LinearArgs(ctypes.Structure):
    _fields_ = [("rows", _i64), ("in_width", _i32), ("out_width", _i32), ("dtype", _i32), ("out_dtype", _i32),
                ("act", _i32), ("gated", _i32), ("x", _p), ("ldx", _i64), ("w", _p), ("ldw", _i64), ("bias", _p),
                ("residual", _p), ("ldr", _i64), ("y", _p), ("ldy", _i64)]


class RouteArgs(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("experts", _i32), ("k", _i32), ("dtype", _i32), ("score", _i32), ("groups", _i32),
                ("topk_groups", _i32), ("group_top", _i32), ("renormalise", _i32), ("scale", _f32),
                ("logits", _p), ("ld", _i64), ("bias", _p), ("index", _p), ("weight", _p)]


class DispatchArgs(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("k", _i32), ("experts", _i32), ("index", _p), ("offsets", _p), ("slots", _p),
                ("places", _p), ("workspace", _p), ("workspace_bytes", _u64)]


class ExpertLinearArgs(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("k", _i32), ("experts", _i32), ("in_width", _i32), ("out_width", _i32),
                ("dtype", _i32), ("out_dtype", _i32), ("act", _i32), ("gated", _i32), ("x_slots", _i32),
                ("combine", _i32), ("x", _p), ("ldx", _i64), ("w", _p), ("ldw", _i64), ("w_stride", _i64),
                ("bias", _p), ("offsets", _p), ("slots", _p), ("places", _p), ("weight", _p), ("residual", _p),
                ("ldr", _i64), ("y", _p), ("ldy", _i64), ("workspace", _p), ("workspace_bytes", _u64)]


_FORMAT = {_p: "P", _i32: "i", _i64: "q", _u64: "Q", _f32: "f"}


def _packer(cls):
    """The bytes of a ``cls`` of these fields: a third of the time that ctypes takes to fill one, and a number that
    does not fit its field is refused instead of cut."""
    packed = struct.Struct("@" + "".join(_FORMAT[t] for _, t in cls._fields_))
    assert packed.size == ctypes.sizeof(cls)

    def pack(*fields):
        try:
            return packed.pack(*fields)
        except struct.error as e:
            raise ValueError("%s: %s" % (cls.__name__, e)) from None
    return pack


_linear_args, _route_args, _dispatch_args, _expert_linear_args = map(
    _packer, (LinearArgs, RouteArgs, DispatchArgs, ExpertLinearArgs))


class Routing(NamedTuple):
    """``index`` int32 [tokens, k], -1 where no expert was left; ``weight`` float32 [tokens, k]."""
    index: torch.Tensor
    weight: torch.Tensor


class Dispatch(NamedTuple):
    """int32: ``offsets`` [experts + 1], ``slots`` [tokens * k] (the assignment token * k + j in each slot, -1
    behind the last), ``places`` [tokens * k] (the slot of each assignment, -1 if dropped)."""
    offsets: torch.Tensor
    slots: torch.Tensor
    places: torch.Tensor


_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        L = B.lib()
        for name in EXPORTED + EXPORTED_FP8:
            f = getattr(L, name)
            f.argtypes = [_p, _p]
            f.restype = ctypes.c_int
        _lib = L
    return _lib


def _call(name: str, args: bytes, device) -> None:
    """Enqueue on the current stream of the tensors' device."""
    f = getattr(_lib or lib(), name)
    at = device.index
    stream = torch._C._cuda_getCurrentRawStream(at)  # torch.cuda.current_stream takes longer than the launch
    if torch._C._cuda_getDevice() == at:
        rc = f(args, stream)
    else:
        with torch.cuda.device(device):
            rc = f(args, stream)
    if rc != B.MLP_OK:
        raise B.MlpError(rc, name, B.mlp_last_error())


def _workspace(name: str, args: bytes, device):
    """Scratch memory for the call, from the current stream's allocator; None where it needs none."""
    need = _u64()
    rc = getattr(_lib or lib(), name)(args, ctypes.addressof(need))
    if rc != B.MLP_OK:
        raise B.MlpError(rc, name, B.mlp_last_error())
    return torch.empty(need.value, dtype=torch.uint8, device=device) if need.value else None


def _tensor(name, t, dims, dtypes, device=None):
    if not isinstance(t, torch.Tensor):
        raise ValueError("%s must be a tensor" % name)
    if t.dim() != dims or t.dtype not in dtypes:
        raise ValueError("%s must be %d-D of type %s, got %d-D %s" % (name, dims, " or ".join(str(d) for d in dtypes),
                                                                    t.dim(), t.dtype))
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError("%s requires a gradient: these operators are for inference (torch.no_grad())" % name)
    if forward_ad._current_level >= 0 and forward_ad.unpack_dual(t).tangent is not None:
        raise ValueError("%s carries a tangent: these operators are for inference (forward_ad.unpack_dual)" % name)
    if not t.is_cuda:
        raise ValueError("%s must be on the GPU" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, not on %s" % (name, t.device, device))
    return t


def _matrix(name, t, dtypes, device=None, rows=None, cols=None):
    """The row stride of a 2-D tensor with contiguous rows, after checking it."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.dtype not in dtypes or not t.is_cuda or (
            device is not None and t.device != device) or t.requires_grad or forward_ad._current_level >= 0:
        _tensor(name, t, 2, dtypes, device)
    r, c = t.shape
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        raise ValueError("%s must be %s x %s, got %d x %d" % (name, "?" if rows is None else rows,
                                                             "?" if cols is None else cols, r, c))
    ld, step = t.stride()
    if step != 1 and c > 1:
        raise ValueError("the rows of %s must be contiguous" % name)
    return ld if r > 1 else c  # a single row has none to the next


def _written(out):
    """Tells autograd that a caller's tensor has new contents: a graph that kept the old ones refuses to use these."""
    if not out.is_inference():
        increment_version(out)


def _vector(name, t, dtype, device, numel):
    _tensor(name, t, t.dim() if isinstance(t, torch.Tensor) else 1, (dtype,), device)
    if t.numel() != numel or not t.is_contiguous():
        raise ValueError("%s must be contiguous with %d elements" % (name, numel))
    return t.data_ptr()


def _choice(name, value, choices):
    try:
        return choices[value]
    except KeyError:
        raise ValueError("%s must be one of %s, got %r" % (name, ", ".join(choices), value)) from None


def _count(name, value):
    try:
        return operator.index(value)
    except TypeError:
        raise ValueError("%s must be a whole number, got %r" % (name, value)) from None


def _out_dtype(dtype, out_dtype):
    if out_dtype is None:
        return dtype
    if out_dtype != dtype and out_dtype != torch.float32:
        raise ValueError("out_dtype must be %s or torch.float32" % dtype)
    return out_dtype


_HALF = (torch.float16, torch.bfloat16)
_FLOATS = tuple(DTYPES)


def linear(x, w, bias=None, *, residual=None, act="none", gated=False, out=None, out_dtype=None):
    """``act(x w^T + bias) + residual``, computed in FP32 and rounded once: one affine layer.

    ``x`` [rows, in] and ``w`` [out, in] are float16 or bfloat16, their rows contiguous (any row stride);
    ``bias`` [out]; ``act`` one of ``ACTIVATIONS``.  ``gated``: w and bias have 2 * out rows, the gates first,
    and the layer is ``act(gate) * up``.  ``out_dtype``: x's type or float32.  ``residual`` [rows, out] has that
    type and may be ``out`` itself."""
    ldx = _matrix("x", x, _HALF)
    rows, k = x.shape
    device, dtype = x.device, x.dtype
    ldw = _matrix("w", w, (dtype,), device, cols=k)
    wide = w.shape[0]
    if gated and wide % 2:
        raise ValueError("a gated layer's w has an even number of rows, got %d" % wide)
    n = wide // 2 if gated else wide
    out_dtype = _out_dtype(dtype, out_dtype)
    given = out is not None
    if not given:
        out = torch.empty(rows, n, dtype=out_dtype, device=device)
        ldy = max(n, 1)
    else:
        ldy = _matrix("out", out, (out_dtype,), device, rows, n)
    ldr = _matrix("residual", residual, (out_dtype,), device, rows, n) if residual is not None else 0
    a = _linear_args(rows, k, n, DTYPES[dtype], DTYPES[out_dtype], _choice("act", act, ACTIVATIONS), 1 if gated else 0,
                     x.data_ptr(), ldx, w.data_ptr(), ldw,
                     0 if bias is None else _vector("bias", bias, dtype, device, wide),
                     0 if residual is None else residual.data_ptr(), ldr, out.data_ptr(), ldy)
    _call("mlp_linear", a, device)
    if given:
        _written(out)
    return out


def route(logits, k, *, score="softmax", bias=None, groups=1, topk_groups=None, group_top=1, renormalise=False,
          scale=1.0) -> Routing:
    """Each token's ``k`` experts by score + bias, largest first, and their weights (scores, without the bias).

    ``logits`` [tokens, experts] float32, float16 or bfloat16 with contiguous rows; ``bias`` float32 [experts]
    enters the choice only; ``groups`` of consecutive experts, of which the ``topk_groups`` with the largest sum
    of their ``group_top`` (1 or 2) best are chosen from.  -inf and NaN logits are never chosen.  Without a bias and
    without ``group_top`` 2 the logits themselves are compared, else the choices to about 50 bits; a token's row does
    not depend on the others."""
    k = _count("k", k)
    ld = _matrix("logits", logits, _FLOATS)
    tokens, experts = logits.shape
    device = logits.device
    room = k if 0 < k <= MLP_OPS_MAX_TOPK else 0  # others are refused below
    index = torch.empty(tokens, room, dtype=torch.int32, device=device)
    weight = torch.empty(tokens, room, dtype=torch.float32, device=device)
    a = _route_args(tokens, experts, k, DTYPES[logits.dtype], _choice("score", score, SCORES),
                  groups, groups if topk_groups is None else topk_groups, group_top,
                  1 if renormalise else 0, scale,
                  logits.data_ptr(), ld, 0 if bias is None else _vector("bias", bias, torch.float32, device, experts),
                  index.data_ptr(), weight.data_ptr())
    _call("mlp_route", a, device)
    return Routing(index, weight)


def dispatch(index, experts) -> Dispatch:
    """The order of the assignments in ``index`` (int32 [tokens, k], contiguous) by expert: a stable sort.
    Indices outside 0 .. experts - 1 take no slot."""
    experts = _count("experts", experts)
    _tensor("index", index, 2, (torch.int32,))
    if not index.is_contiguous():
        raise ValueError("index must be contiguous")
    tokens, k = index.shape
    device, n = index.device, index.numel()
    offsets = torch.empty(experts + 1 if 0 < experts <= MLP_OPS_MAX_EXPERTS else 0, dtype=torch.int32, device=device)
    slots = torch.empty(n, dtype=torch.int32, device=device)
    places = torch.empty_like(slots)
    a = (tokens, k, experts, index.data_ptr(), offsets.data_ptr(), slots.data_ptr(), places.data_ptr())
    packed = _dispatch_args(*a, 0, 0)
    ws = _workspace("mlp_dispatch_workspace", packed, device)
    _call("mlp_dispatch", packed if ws is None else _dispatch_args(*a, ws.data_ptr(), ws.numel()), device)
    return Dispatch(offsets, slots, places)


def expert_linear(x, w, plan: Dispatch, bias=None, *, k, act="none", gated=False, rows="tokens", combine=False,
                  weight=None, residual=None, out=None, out_dtype=None):
    """Each routed row through its own expert's layer, ``act(x w[e]^T + bias[e])`` (or gated, as ``linear``).

    ``w`` [experts, out or 2 * out, in], ``bias`` [experts, out or 2 * out], ``plan`` from ``dispatch`` of a
    [tokens, k] index.  ``rows``: x has a row for each token ("tokens") or each slot ("slots").  Returns a row
    for each slot (those behind the last slot in use are not written), or with ``combine`` a row for each token:
    the sum of its experts' outputs by ``weight`` (float32 [tokens, k], or 1), plus ``residual``."""
    if rows not in ("tokens", "slots"):
        raise ValueError("rows must be tokens or slots, got %r" % (rows,))
    k = _count("k", k)
    ldx = _matrix("x", x, _HALF)
    device, dtype, k_in = x.device, x.dtype, x.shape[1]
    _tensor("w", w, 3, (dtype,), device)
    experts, wide = w.shape[0], w.shape[1]
    if w.shape[2] != k_in or (w.stride(2) != 1 and k_in > 1):
        raise ValueError("w must be [experts, out, %d] with contiguous rows" % k_in)
    if gated and wide % 2:
        raise ValueError("a gated layer's w has an even number of rows, got %d" % wide)
    n = wide // 2 if gated else wide
    if not isinstance(plan.places, torch.Tensor) or k < 1 or plan.places.numel() % k:
        raise ValueError("plan.places must hold k = %d places for each token" % k)
    total = plan.places.numel()
    tokens = total // k
    if x.shape[0] != (total if rows == "slots" else tokens):
        raise ValueError("x has %d rows, the plan has %d tokens and %d slots" % (x.shape[0], tokens, total))
    out_dtype = _out_dtype(dtype, out_dtype)
    y_rows = tokens if combine else total
    given = out is not None
    if not given:
        out = torch.empty(y_rows, n, dtype=out_dtype, device=device)
        ldy = max(n, 1)
    else:
        ldy = _matrix("out", out, (out_dtype,), device, y_rows, n)
    ldr = _matrix("residual", residual, (out_dtype,), device, y_rows, n) if residual is not None else 0
    a = (
        tokens, k, experts, k_in, n, DTYPES[dtype], DTYPES[out_dtype], _choice("act", act, ACTIVATIONS),
        1 if gated else 0, 1 if rows == "slots" else 0, 1 if combine else 0, x.data_ptr(), ldx, w.data_ptr(),
        w.stride(1) if wide > 1 else k_in, w.stride(0) if experts > 1 else 0,
        0 if bias is None else _vector("bias", bias, dtype, device, experts * wide),
        _vector("plan.offsets", plan.offsets, torch.int32, device, experts + 1),
        _vector("plan.slots", plan.slots, torch.int32, device, total),
        _vector("plan.places", plan.places, torch.int32, device, total),
        0 if weight is None else _vector("weight", weight, torch.float32, device, total),
        0 if residual is None else residual.data_ptr(), ldr, out.data_ptr(), ldy)
    packed = _expert_linear_args(*a, 0, 0)
    ws = _workspace("mlp_expert_linear_workspace", packed, device) if combine else None
    _call("mlp_expert_linear", packed if ws is None else _expert_linear_args(*a, ws.data_ptr(), ws.numel()), device)
    if given:
        _written(out)
    return out
