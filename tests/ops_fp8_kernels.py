"""Which kernel a call of the 8-bit operators takes (the library's test hooks), and sizes for each."""
from __future__ import annotations

import ctypes

from mlp_neural_shading_amd import binding as B
from mlp_neural_shading_amd import ops_fp8 as E

FAR = 1 << 40  # stands for device pointers a terabyte apart: never read


def _name(function, args):
    buf = ctypes.create_string_buffer(64)
    rc = getattr(B.lib(), function)(ctypes.addressof(args), buf, 64)
    if rc != B.MLP_OK:
        raise B.MlpError(rc, function, B.mlp_last_error())
    return buf.value.decode()


def _blocks(n):
    return -(-n // 128)


def linear_kernel(rows, k, n, gated=False, out_dtype=0, ldx=None, ldw=None, x=FAR, w=2 * FAR):
    return _name("mlp_testing_fp8_linear_kernel", E.Fp8LinearArgs(
        rows=rows, in_width=k, out_width=n, out_dtype=out_dtype, act=0, gated=int(gated), x=x, ldx=ldx or k, x_scale=4 * FAR,
        ldxs=_blocks(k), w=w, ldw=ldw or k, w_scale=5 * FAR, ldws=_blocks(k), bias=None, residual=None, ldr=0, y=3 * FAR, ldy=n,
        y_scale=6 * FAR if out_dtype == 3 else None, ldys=_blocks(n), workspace=7 * FAR, workspace_bytes=FAR - 1))


def expert_kernel(tokens, k, experts, k_in, n, gated=False, out_dtype=0, ldx=None, ldw=None, w_stride=None, x=FAR, w=2 * FAR):
    ldw = ldw or k_in
    halves = 2 if gated else 1
    return _name("mlp_testing_fp8_expert_linear_kernel", E.Fp8ExpertLinearArgs(
        tokens=tokens, k=k, experts=experts, in_width=k_in, out_width=n, out_dtype=out_dtype, act=0, gated=int(gated), x_slots=0,
        combine=0, x=x, ldx=ldx or k_in, x_scale=4 * FAR, ldxs=_blocks(k_in), w=w, ldw=ldw,
        w_stride=ldw * n * halves if w_stride is None else w_stride, w_scale=5 * FAR, ldws=_blocks(k_in),
        ws_stride=_blocks(n) * halves * _blocks(k_in), bias=None, offsets=8 * FAR, slots=9 * FAR, places=10 * FAR, weight=None,
        residual=None, ldr=0, y=3 * FAR, ldy=n, y_scale=6 * FAR if out_dtype == 3 else None, ldys=_blocks(n), workspace=7 * FAR,
        workspace_bytes=FAR - 1))


def norm_kernel(rows, width, dtype=1):
    return _name("mlp_testing_norm_kernel", E.RmsNormArgs(
        rows=rows, width=width, dtype=dtype, out_dtype=dtype, eps=1e-6, x=FAR, ldx=width, residual=None, ldr=0, weight=None,
        total=None, ldt=0, y=2 * FAR, ldy=width, values=None, ldv=0, scales=None, lds=0))


# The kernel that writes 16 bits, by size; FP32 and 8-bit outputs take others of them.
LINEAR = {"few": (70, 100, 60, False), "few wide": (100, 72, 700, False), "thin": (300, 3000, 1001, False), "small": (601, 136, 699, False),
          "mid": (2601, 200, 2501, False), "big": (5001, 200, 1801, False), "tile": (9001, 72, 63, False)}
GATED = {"few wide": (100, 72, 40, True), "small": (600, 136, 351, True), "mid": (2601, 200, 1251, True),
         "big": (2601, 264, 1700, True), "tile": (8200, 72, 32, True)}
EXPERTS = {"few": (37, 3, 5, 200, 130, False), "small": (900, 2, 5, 136, 700, False), "mid": (3000, 2, 4, 72, 1201, False),
           "big": (4000, 2, 4, 72, 1200, False), "tile": (700, 2, 6, 33, 300, False), "few wide": (300, 2, 3, 72, 300, False)}
EXPERTS_GATED = {"few wide": (200, 2, 6, 64, 200, True), "small": (900, 2, 5, 136, 351, True), "mid": (2600, 2, 4, 136, 611, True),
                 "big": (3000, 2, 4, 72, 1200, True), "tile": (1500, 2, 6, 33, 150, True)}
NORMS = [(1, 1, "16x1"), (1 << 20, 128, "16x1"), (1, 129, "256x1"), (1023, 2048, "256x1"), (1024, 129, "64x1"), (1024, 512, "64x1"),
         (1024, 513, "64x2"), (1024, 1024, "64x2"), (1024, 1025, "256x1"), (1, 2049, "256x2"), (9999, 4096, "256x2"),
         (2, 4097, "512x2"), (2, 8192, "512x2"), (2, 8193, "512x2 twice"), (2, 32768, "512x2 twice"), (2, 32769, "1024x4 twice")]
