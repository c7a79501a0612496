"""Host-side checks of the 8-bit operators (no GPU needed): exports and struct layouts as include/mlp_ops_fp8.h declares
them, every refusal before any HIP call, the workspace queries, and the choice of kernel."""
import ctypes
import re
import subprocess
from pathlib import Path

import pytest
import torch
import torch.autograd.forward_ad as fa

import ops_fp8_kernels as K
from mlp_neural_shading_amd import binding as B
from mlp_neural_shading_amd import ops
from mlp_neural_shading_amd import ops_fp8 as E

ROOT = Path(__file__).resolve().parents[1]
HEADER = ROOT / "include" / "mlp_ops_fp8.h"
P = 0x100000  # stands for a device pointer: never read, the calls below are refused before any HIP call

STRUCTS = {"mlp_rms_norm_args": E.RmsNormArgs, "mlp_quantize_args": E.QuantizeArgs, "mlp_fp8_linear_args": E.Fp8LinearArgs,
           "mlp_fp8_expert_linear_args": E.Fp8ExpertLinearArgs}


def test_library_exports_every_declared_function():
    decls = set(re.findall(r"^\s*int\s*(mlp_\w+)\s*\(", HEADER.read_text(), re.M))
    assert decls == set(ops.EXPORTED_FP8)
    for name in decls:
        assert hasattr(ops.lib(), name), name


def test_structs_match_the_header(tmp_path):
    """Sizes and offsets as a C compiler lays the header's structs out."""
    lines = []
    for name, cls in STRUCTS.items():
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (name, name))
        lines += ['printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (name, f, name, f) for f, _ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "mlp_ops_fp8.h"\nint main(void) {\n%s\nreturn 0;\n}\n' % "\n".join(lines))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-Wall", "-Werror", "-I", str(ROOT / "include"), str(src), "-o", str(exe)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines())
    for name, cls in STRUCTS.items():
        assert int(got[name]) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(got["%s.%s" % (name, f)]) == getattr(cls, f).offset, (name, f)


def norm_args(**over):
    a = dict(rows=4, width=130, dtype=0, out_dtype=0, eps=1e-6, x=P, ldx=130, residual=None, ldr=130, weight=None, total=None,
             ldt=130, y=2 * P, ldy=130, values=3 * P, ldv=130, scales=4 * P, lds=2)
    a.update(over)
    return E.RmsNormArgs(**a)


def quantize_args(**over):
    a = dict(rows=4, count=1, width=130, dtype=0, block_rows=1, x=P, ldx=130, x_stride=0, values=2 * P, ldv=130, v_stride=0,
             scales=3 * P, lds=2, s_stride=0)
    a.update(over)
    return E.QuantizeArgs(**a)


def linear_args(**over):
    a = dict(rows=4, in_width=130, out_width=8, out_dtype=0, act=0, gated=0, x=P, ldx=130, x_scale=2 * P, ldxs=2, w=3 * P,
             ldw=130, w_scale=4 * P, ldws=2, bias=None, residual=None, ldr=0, y=5 * P, ldy=8, y_scale=None, ldys=0,
             workspace=None, workspace_bytes=0)
    a.update(over)
    return E.Fp8LinearArgs(**a)


def expert_args(**over):
    a = dict(tokens=4, k=2, experts=8, in_width=130, out_width=8, out_dtype=0, act=0, gated=0, x_slots=0, combine=0, x=P,
             ldx=130, x_scale=2 * P, ldxs=2, w=3 * P, ldw=130, w_stride=1040, w_scale=4 * P, ldws=2, ws_stride=2, bias=None,
             offsets=6 * P, slots=7 * P, places=8 * P, weight=None, residual=None, ldr=0, y=5 * P, ldy=8, y_scale=None, ldys=0,
             workspace=None, workspace_bytes=0)
    a.update(over)
    return E.Fp8ExpertLinearArgs(**a)


MAKE = {"mlp_rms_norm": norm_args, "mlp_quantize": quantize_args, "mlp_fp8_linear": linear_args,
        "mlp_fp8_expert_linear": expert_args}

FP8 = dict(out_dtype=3, y_scale=9 * P, ldys=1, workspace=10 * P, workspace_bytes=256)
REFUSED = [
    ("mlp_rms_norm", dict(rows=-1), "rows"), ("mlp_rms_norm", dict(rows=1 << 31), "rows"), ("mlp_rms_norm", dict(width=0), "width"),
    ("mlp_rms_norm", dict(width=(1 << 20) + 1), "width"), ("mlp_rms_norm", dict(dtype=3), "dtype"),
    ("mlp_rms_norm", dict(out_dtype=1), "out_dtype"), ("mlp_rms_norm", dict(out_dtype=3), "out_dtype"),
    ("mlp_rms_norm", dict(eps=0.0), "eps"), ("mlp_rms_norm", dict(eps=1e-40), "eps"), ("mlp_rms_norm", dict(eps=-1.0), "eps"),
    ("mlp_rms_norm", dict(eps=float("nan")), "eps"), ("mlp_rms_norm", dict(eps=float("inf")), "eps"),
    ("mlp_rms_norm", dict(x=None), "x is NULL"), ("mlp_rms_norm", dict(x=P + 1), "aligned"), ("mlp_rms_norm", dict(ldx=129), "stride"),
    ("mlp_rms_norm", dict(residual=5 * P, ldr=129), "stride"), ("mlp_rms_norm", dict(weight=5 * P + 1), "aligned"),
    ("mlp_rms_norm", dict(total=5 * P), "residual"), ("mlp_rms_norm", dict(residual=5 * P, total=6 * P, ldt=1), "stride"),
    ("mlp_rms_norm", dict(y=None, values=None), "NULL"), ("mlp_rms_norm", dict(scales=None), "scales is NULL"),
    ("mlp_rms_norm", dict(lds=1), "stride"), ("mlp_rms_norm", dict(ldv=129), "stride"), ("mlp_rms_norm", dict(ldy=129), "stride"),
    ("mlp_rms_norm", dict(y=P), "overlaps"), ("mlp_rms_norm", dict(values=P + 8), "overlaps"), ("mlp_rms_norm", dict(values=2 * P), "overlaps"),
    ("mlp_rms_norm", dict(scales=3 * P), "overlaps"), ("mlp_rms_norm", dict(residual=5 * P, total=P + 2), "total overlaps"),
    ("mlp_rms_norm", dict(residual=5 * P, total=5 * P, ldt=132), "total overlaps"),
    ("mlp_rms_norm", dict(residual=5 * P, total=6 * P, weight=6 * P), "total overlaps"),
    ("mlp_rms_norm", dict(residual=5 * P, total=6 * P, y=6 * P + 4), "overlaps"), ("mlp_rms_norm", dict(weight=2 * P), "overlaps"),
    ("mlp_rms_norm", dict(residual=2 * P, total=6 * P), "overlaps"),
    ("mlp_quantize", dict(rows=-1), "rows"), ("mlp_quantize", dict(count=-1), "count"), ("mlp_quantize", dict(count=65536), "count"),
    ("mlp_quantize", dict(width=0), "width"), ("mlp_quantize", dict(dtype=3), "dtype"), ("mlp_quantize", dict(block_rows=2), "block_rows"),
    ("mlp_quantize", dict(x=None), "NULL"), ("mlp_quantize", dict(values=None), "NULL"), ("mlp_quantize", dict(scales=None), "NULL"),
    ("mlp_quantize", dict(ldx=1), "stride"), ("mlp_quantize", dict(ldv=1), "stride"), ("mlp_quantize", dict(lds=1), "stride"),
    ("mlp_quantize", dict(count=2, x_stride=519, v_stride=520, s_stride=8), "x_stride"),
    ("mlp_quantize", dict(count=2, x_stride=520, v_stride=519, s_stride=8), "v_stride"),
    ("mlp_quantize", dict(count=2, x_stride=520, v_stride=520, s_stride=7), "s_stride"),
    ("mlp_quantize", dict(count=2, block_rows=128, x_stride=520, v_stride=520, s_stride=1), "s_stride"),
    ("mlp_quantize", dict(values=P + 100), "overlaps"), ("mlp_quantize", dict(scales=2 * P), "overlaps"), ("mlp_quantize", dict(scales=P), "overlaps"),
    ("mlp_quantize", dict(count=3, x_stride=520, v_stride=520, s_stride=8, scales=2 * P + 1500), "overlaps"),
    ("mlp_fp8_linear", dict(rows=-1), "rows"), ("mlp_fp8_linear", dict(in_width=0), "in_width"),
    ("mlp_fp8_linear", dict(out_width=0), "out_width"), ("mlp_fp8_linear", dict(out_width=(1 << 20) + 1), "out_width"),
    ("mlp_fp8_linear", dict(out_dtype=4), "out_dtype"), ("mlp_fp8_linear", dict(act=5), "act"), ("mlp_fp8_linear", dict(gated=2), "gated"),
    ("mlp_fp8_linear", dict(x=None), "x is NULL"), ("mlp_fp8_linear", dict(w=None), "w is NULL"),
    ("mlp_fp8_linear", dict(x_scale=None), "x_scale is NULL"), ("mlp_fp8_linear", dict(w_scale=None), "w_scale is NULL"),
    ("mlp_fp8_linear", dict(x_scale=2 * P + 2), "aligned"), ("mlp_fp8_linear", dict(w_scale=4 * P + 1), "aligned"),
    ("mlp_fp8_linear", dict(ldxs=1), "stride"), ("mlp_fp8_linear", dict(ldws=1), "stride"), ("mlp_fp8_linear", dict(ldx=129), "stride"),
    ("mlp_fp8_linear", dict(ldw=129), "stride"), ("mlp_fp8_linear", dict(y=None), "y is NULL"), ("mlp_fp8_linear", dict(ldy=7), "stride"),
    ("mlp_fp8_linear", dict(ldy=(1 << 24) + 1), "larger"), ("mlp_fp8_linear", dict(bias=6 * P + 2), "aligned"),
    ("mlp_fp8_linear", dict(y=P), "overlaps"), ("mlp_fp8_linear", dict(y=2 * P), "overlaps"), ("mlp_fp8_linear", dict(y=4 * P), "overlaps"),
    ("mlp_fp8_linear", dict(bias=5 * P + 16), "overlaps"), ("mlp_fp8_linear", dict(y_scale=6 * P, ldys=1), "y_scale"),
    ("mlp_fp8_linear", dict(residual=5 * P + 16, ldr=8), "residual"), ("mlp_fp8_linear", dict(residual=6 * P, ldr=7), "stride"),
    ("mlp_fp8_linear", dict(FP8, y_scale=None), "y_scale is NULL"), ("mlp_fp8_linear", dict(FP8, ldys=0), "stride"),
    ("mlp_fp8_linear", dict(FP8, residual=6 * P, ldr=8), "residual"), ("mlp_fp8_linear", dict(FP8, y_scale=5 * P + 4), "overlaps"),
    ("mlp_fp8_linear", dict(FP8, y_scale=P), "overlaps"), ("mlp_fp8_linear", dict(FP8, workspace=None), "workspace is NULL"),
    ("mlp_fp8_linear", dict(FP8, workspace_bytes=127), "workspace holds"), ("mlp_fp8_linear", dict(FP8, workspace=10 * P + 8), "16-byte"),
    ("mlp_fp8_linear", dict(FP8, workspace=9 * P), "workspace overlaps"), ("mlp_fp8_linear", dict(FP8, workspace=3 * P), "workspace overlaps"),
    ("mlp_fp8_expert_linear", dict(tokens=-1), "tokens"), ("mlp_fp8_expert_linear", dict(experts=1025), "experts"),
    ("mlp_fp8_expert_linear", dict(k=0), "k must"), ("mlp_fp8_expert_linear", dict(tokens=1 << 30), "tokens * k"),
    ("mlp_fp8_expert_linear", dict(x_slots=2), "x_slots"), ("mlp_fp8_expert_linear", dict(combine=2), "combine"),
    ("mlp_fp8_expert_linear", dict(FP8, combine=1), "combine"), ("mlp_fp8_expert_linear", dict(weight=9 * P), "combine"),
    ("mlp_fp8_expert_linear", dict(residual=9 * P, ldr=8), "combine"), ("mlp_fp8_expert_linear", dict(w_stride=1039), "w_stride"),
    ("mlp_fp8_expert_linear", dict(ws_stride=1), "ws_stride"), ("mlp_fp8_expert_linear", dict(gated=1, w_stride=2080, ws_stride=3), "ws_stride"),
    ("mlp_fp8_expert_linear", dict(offsets=None), "offsets"), ("mlp_fp8_expert_linear", dict(slots=None), "slots"),
    ("mlp_fp8_expert_linear", dict(combine=1, places=None), "places"), ("mlp_fp8_expert_linear", dict(combine=1), "workspace is NULL"),
    ("mlp_fp8_expert_linear", dict(combine=1, workspace=11 * P, workspace_bytes=255), "workspace holds"),
    ("mlp_fp8_expert_linear", dict(y=6 * P), "overlaps"), ("mlp_fp8_expert_linear", dict(y=3 * P + 8000), "overlaps"),
    ("mlp_fp8_expert_linear", dict(y=4 * P + 60), "overlaps"),
    ("mlp_fp8_expert_linear", dict(combine=1, workspace=7 * P, workspace_bytes=256), "workspace overlaps"),
]


@pytest.mark.parametrize("name,over,says", REFUSED, ids=["%s-%d" % (r[0][4:], i) for i, r in enumerate(REFUSED)])
def test_refusals(name, over, says):
    a = MAKE[name](**over)
    assert getattr(ops.lib(), name)(ctypes.addressof(a), None) == B.MLP_ERR_INVALID_ARGUMENT
    assert says in B.mlp_last_error()


def test_null_struct():
    n = ctypes.c_uint64()
    for name in ops.EXPORTED_FP8:
        if name.endswith("_workspace"):
            assert getattr(ops.lib(), name)(None, ctypes.addressof(n)) == B.MLP_ERR_INVALID_ARGUMENT
            assert getattr(ops.lib(), name)(ctypes.addressof(MAKE[name[:-10]]()), None) == B.MLP_ERR_INVALID_ARGUMENT
        else:
            assert getattr(ops.lib(), name)(None, None) == B.MLP_ERR_INVALID_ARGUMENT


def test_nothing_to_do():
    """No rows: answered without a HIP call, whatever the pointers."""
    for name, over in [("mlp_rms_norm", dict(rows=0, x=None, y=None)), ("mlp_quantize", dict(rows=0, x=None)),
                       ("mlp_quantize", dict(count=0, x=None)), ("mlp_fp8_linear", dict(rows=0, x=None, y=None)),
                       ("mlp_fp8_expert_linear", dict(tokens=0, x=None, y=None))]:
        a = MAKE[name](**over)
        assert getattr(ops.lib(), name)(ctypes.addressof(a), None) == B.MLP_OK


def test_too_many_tiles_is_unsupported():
    a = linear_args(rows=(1 << 31) - 1, out_width=1 << 20, ldy=1 << 20, x=1 << 56, x_scale=1 << 58, w=1 << 40, w_scale=1 << 36, y=1 << 44)
    assert ops.lib().mlp_fp8_linear(ctypes.addressof(a), None) == B.MLP_ERR_UNSUPPORTED


def quantized(*shape, block_rows=1):
    rows, width = shape[-2:]
    return E.Quantized(torch.zeros(shape, dtype=torch.uint8).view(E.FP8),
                       torch.ones(*shape[:-2], -(-rows // block_rows), -(-width // 128)))


def test_torch_refusals():
    x, w = quantized(4, 130), quantized(8, 130, block_rows=128)
    plan = ops.Dispatch(torch.zeros(9, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), torch.zeros(8, dtype=torch.int32))
    f = torch.zeros(4, 130)
    for call in (lambda: E.linear(x, w), lambda: E.quantize(f), lambda: E.quantize(f[None]), lambda: E.rms_norm(f),
                 lambda: E.expert_linear(x, w, plan, k=2)):
        with pytest.raises(ValueError, match="on the GPU"):
            call()
    for call, says in ((lambda: E.linear(f, w), "Quantized"), (lambda: E.linear(E.Quantized(f, f), w), "of type"),
                       (lambda: E.quantize(f.double()), "of type"), (lambda: E.quantize(f[0]), "2-D"), (lambda: E.quantize(None), "tensor"),
                       (lambda: E.quantize(f, block_rows=64), "block_rows"), (lambda: E.quantize(f, block_rows=1.0), "whole"),
                       (lambda: E.rms_norm(f, out="int8"), "out must"), (lambda: E.expert_linear(x, w, plan, k=2, rows="both"), "rows"),
                       (lambda: E.expert_linear(x, w, plan, k=2.0), "whole")):
        with pytest.raises(ValueError, match=says):
            call()
    with pytest.raises(ValueError, match="gradient"):
        E.rms_norm(f.clone().requires_grad_())
    with fa.dual_level(), pytest.raises(ValueError, match="tangent"):
        E.quantize(fa.make_dual(f, f))


# ---- which kernel ----------------------------------------------------------------------------------

def test_kernels_by_size():
    """The sizes take every kernel for 16 bits, for FP32 and for 8-bit outputs (`big` there for gated layers only)."""
    for sizes, kernel in ((K.LINEAR, K.linear_kernel), (K.GATED, K.linear_kernel), (K.EXPERTS, K.expert_kernel),
                          (K.EXPERTS_GATED, K.expert_kernel)):
        for name, size in sizes.items():
            assert kernel(*size) == name, size
        gated = size[-1]
        assert {kernel(*s, out_dtype=2) for s in sizes.values()} == set(sizes) - {"big"}
        assert {kernel(*s, out_dtype=3) for s in sizes.values()} >= set(sizes) - ({"mid"} if gated else {"big"})
    assert K.linear_kernel(0, 8, 8) == "none" and K.expert_kernel(0, 2, 4, 8, 8) == "none"


def test_kernels_for_rows_at_any_byte():
    """Only `tile` and the few-row kernels take rows that are not 4-byte aligned."""
    size = K.LINEAR["big"]
    k = size[1]
    for over in (dict(ldx=k + 1), dict(ldw=k + 2), dict(x=K.FAR + 2), dict(w=2 * K.FAR + 1)):
        assert K.linear_kernel(*size, **over) == "tile", over
    assert K.linear_kernel(*size, ldx=k + 8, ldw=k + 4, x=K.FAR + 4, w=2 * K.FAR + 12) == "big"
    tokens, kk, experts, k_in, n, _ = K.EXPERTS["mid"]
    assert K.expert_kernel(*K.EXPERTS["mid"], w_stride=k_in * n + 1) == "tile"
    for w_stride in (0, 7, -1, 2 ** 40 + 1):  # one expert's means nothing
        assert K.expert_kernel(tokens, kk, 1, k_in, n, w_stride=w_stride) != "tile"


def test_norm_kernels():
    for rows, width, name in K.NORMS:
        assert K.norm_kernel(rows, width) == name, (rows, width)
