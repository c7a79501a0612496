"""Host-side checks of the single operators (no GPU needed): the library exports what include/mlp_ops.h
declares, the binding's structs have the header's layout, every refusal comes back before any HIP call, and
the workspace queries answer."""
import ctypes
import re
import subprocess
from pathlib import Path

import pytest
import torch

from mlp_neural_shading_amd import binding as B
from mlp_neural_shading_amd import ops

ROOT = Path(__file__).resolve().parents[1]
HEADER = ROOT / "include" / "mlp_ops.h"
P = 0x100000  # stands for a device pointer: never read, the calls below are refused before any HIP call

STRUCTS = {"mlp_linear_args": ops.LinearArgs, "mlp_route_args": ops.RouteArgs, "mlp_dispatch_args": ops.DispatchArgs,
           "mlp_expert_linear_args": ops.ExpertLinearArgs}


def test_library_exports_every_declared_function():
    decls = set(re.findall(r"^\s*int\s*(mlp_\w+)\s*\(", HEADER.read_text(), re.M))
    assert decls == set(ops.EXPORTED)
    for name in decls:
        assert hasattr(ops.lib(), name), name


def test_structs_match_the_header(tmp_path):
    """Sizes and offsets as a C compiler lays the header's structs out."""
    lines = []
    for name, cls in STRUCTS.items():
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (name, name))
        lines += ['printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (name, f, name, f) for f, _ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "mlp_ops.h"\nint main(void) {\n%s\nreturn 0;\n}\n' % "\n".join(lines))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-Wall", "-Werror", "-I", str(ROOT / "include"), str(src), "-o", str(exe)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines())
    for name, cls in STRUCTS.items():
        assert int(got[name]) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(got["%s.%s" % (name, f)]) == getattr(cls, f).offset, (name, f)


def linear_args(**over):
    a = dict(rows=4, in_width=8, out_width=8, dtype=0, out_dtype=0, act=0, gated=0, x=P, ldx=8, w=2 * P, ldw=8,
             bias=None, residual=None, ldr=0, y=3 * P, ldy=8)
    a.update(over)
    return ops.LinearArgs(**a)


def route_args(**over):
    a = dict(tokens=4, experts=8, k=2, dtype=2, score=0, groups=1, topk_groups=1, group_top=1, renormalise=0, scale=1.0,
             logits=P, ld=8, bias=None, index=2 * P, weight=3 * P)
    a.update(over)
    return ops.RouteArgs(**a)


def dispatch_args(**over):
    a = dict(tokens=4, k=2, experts=8, index=P, offsets=2 * P, slots=3 * P, places=4 * P, workspace=None,
             workspace_bytes=0)
    a.update(over)
    return ops.DispatchArgs(**a)


def expert_args(**over):
    a = dict(tokens=4, k=2, experts=8, in_width=8, out_width=8, dtype=0, out_dtype=0, act=0, gated=0, x_slots=0, combine=0,
             x=P, ldx=8, w=2 * P, ldw=8, w_stride=64, bias=None, offsets=4 * P, slots=5 * P, places=6 * P, weight=None,
             residual=None, ldr=0, y=3 * P, ldy=8, workspace=None, workspace_bytes=0)
    a.update(over)
    return ops.ExpertLinearArgs(**a)


MAKE = {"mlp_linear": linear_args, "mlp_route": route_args, "mlp_dispatch": dispatch_args, "mlp_expert_linear": expert_args}

REFUSED = [
    ("mlp_linear", dict(rows=-1), "rows"), ("mlp_linear", dict(rows=1 << 31), "rows"),
    ("mlp_linear", dict(in_width=0), "in_width"), ("mlp_linear", dict(in_width=(1 << 20) + 1), "in_width"),
    ("mlp_linear", dict(out_width=0), "out_width"), ("mlp_linear", dict(dtype=2), "dtype"),
    ("mlp_linear", dict(dtype=3), "dtype"), ("mlp_linear", dict(out_dtype=1), "out_dtype"),
    ("mlp_linear", dict(act=5), "act"), ("mlp_linear", dict(act=-1), "act"), ("mlp_linear", dict(gated=2), "gated"),
    ("mlp_linear", dict(x=None), "x is NULL"), ("mlp_linear", dict(w=None), "w is NULL"),
    ("mlp_linear", dict(y=None), "y is NULL"), ("mlp_linear", dict(x=P + 1), "aligned"),
    ("mlp_linear", dict(bias=P + 1), "aligned"), ("mlp_linear", dict(y=P + 2, out_dtype=2), "aligned"),
    ("mlp_linear", dict(ldx=7), "stride"), ("mlp_linear", dict(ldw=7), "stride"), ("mlp_linear", dict(ldy=7), "stride"),
    ("mlp_linear", dict(ldx=-8), "stride"), ("mlp_linear", dict(ldx=1 << 60), "too large"),
    ("mlp_linear", dict(y=P), "overlaps"), ("mlp_linear", dict(y=2 * P + 16), "overlaps"),
    ("mlp_linear", dict(bias=3 * P + 8), "overlaps"), ("mlp_linear", dict(residual=3 * P + 16, ldr=8), "residual"),
    ("mlp_linear", dict(residual=3 * P, ldr=16), "residual"), ("mlp_linear", dict(residual=4 * P, ldr=7), "stride"),
    ("mlp_linear", dict(x=3 * P + 14, ldx=16, ldy=16), "overlaps"),  # one column too many beside y
    ("mlp_linear", dict(ldy=(1 << 24) + 1), "larger"), ("mlp_linear", dict(residual=1 << 40, ldr=(1 << 24) + 1), "larger"),
    ("mlp_expert_linear", dict(ldy=(1 << 24) + 1, y=1 << 40), "larger"),
    ("mlp_route", dict(tokens=-1), "tokens"), ("mlp_route", dict(experts=0), "experts"),
    ("mlp_route", dict(experts=1025), "experts"), ("mlp_route", dict(k=0), "k must"), ("mlp_route", dict(k=9), "k must"),
    ("mlp_route", dict(experts=64, ld=64, k=33), "k must"), ("mlp_route", dict(dtype=3), "dtype"),
    ("mlp_route", dict(score=2), "score"), ("mlp_route", dict(groups=3), "divide"), ("mlp_route", dict(groups=0), "groups"),
    ("mlp_route", dict(groups=2, topk_groups=3), "topk_groups"), ("mlp_route", dict(topk_groups=0), "topk_groups"),
    ("mlp_route", dict(group_top=3), "group_top"), ("mlp_route", dict(renormalise=2), "renormalise"),
    ("mlp_route", dict(scale=float("nan")), "scale"), ("mlp_route", dict(scale=float("inf")), "scale"),
    ("mlp_route", dict(logits=None), "NULL"), ("mlp_route", dict(ld=7), "stride"), ("mlp_route", dict(bias=P + 2), "aligned"),
    ("mlp_route", dict(index=P), "overlaps"), ("mlp_route", dict(index=3 * P), "overlaps"),
    ("mlp_dispatch", dict(tokens=-1), "tokens"), ("mlp_dispatch", dict(k=0), "k must"), ("mlp_dispatch", dict(k=33), "k must"),
    ("mlp_dispatch", dict(experts=0), "experts"), ("mlp_dispatch", dict(tokens=1 << 30, k=2), "tokens * k"),
    ("mlp_dispatch", dict(index=None), "NULL"), ("mlp_dispatch", dict(offsets=None), "NULL"),
    ("mlp_dispatch", dict(places=P + 2), "aligned"), ("mlp_dispatch", dict(slots=P), "overlap"),
    ("mlp_dispatch", dict(tokens=1 << 20, slots=64 * P, places=128 * P, index=256 * P), "workspace is NULL"),
    ("mlp_dispatch", dict(tokens=1 << 20, slots=64 * P, places=128 * P, index=256 * P, workspace=P + 4, workspace_bytes=1 << 30), "16-byte"),
    ("mlp_dispatch", dict(tokens=1 << 20, slots=64 * P, places=128 * P, index=256 * P, workspace=P, workspace_bytes=64), "workspace holds"),
    ("mlp_expert_linear", dict(tokens=-1), "tokens"), ("mlp_expert_linear", dict(experts=1025), "experts"),
    ("mlp_expert_linear", dict(k=0), "k must"), ("mlp_expert_linear", dict(in_width=0), "in_width"),
    ("mlp_expert_linear", dict(x_slots=2), "x_slots"), ("mlp_expert_linear", dict(combine=2), "combine"),
    ("mlp_expert_linear", dict(weight=7 * P), "combine"), ("mlp_expert_linear", dict(residual=7 * P, ldr=8), "combine"),
    ("mlp_expert_linear", dict(slots=None), "slots"), ("mlp_expert_linear", dict(w_stride=63), "w_stride"),
    ("mlp_expert_linear", dict(w_stride=-64), "w_stride"), ("mlp_expert_linear", dict(offsets=None), "offsets"),
    ("mlp_expert_linear", dict(combine=1, workspace=8 * P, workspace_bytes=256, places=None), "places"),
    ("mlp_expert_linear", dict(combine=1), "workspace is NULL"),
    ("mlp_expert_linear", dict(combine=1, workspace=8 * P, workspace_bytes=255), "workspace holds"),
    ("mlp_expert_linear", dict(combine=1, workspace=8 * P + 8, workspace_bytes=256), "16-byte"),
    ("mlp_expert_linear", dict(combine=1, workspace=2 * P + 16, workspace_bytes=256), "workspace overlaps"),
    ("mlp_expert_linear", dict(combine=1, workspace=3 * P - 16, workspace_bytes=256), "workspace overlaps"),
    ("mlp_expert_linear", dict(combine=1, workspace=4 * P + 32, workspace_bytes=256), "workspace overlaps"),
    ("mlp_expert_linear", dict(combine=1, workspace=5 * P, workspace_bytes=256), "workspace overlaps"),
    ("mlp_expert_linear", dict(combine=1, workspace=6 * P + 16, workspace_bytes=256), "workspace overlaps"),
    ("mlp_expert_linear", dict(combine=1, workspace=8 * P, workspace_bytes=256, weight=8 * P + 252), "workspace overlaps"),
    ("mlp_expert_linear", dict(combine=1, workspace=8 * P, workspace_bytes=256, bias=8 * P + 128), "workspace overlaps"),
    ("mlp_dispatch", dict(tokens=1 << 20, slots=64 * P, places=128 * P, index=256 * P, offsets=500 * P, workspace=128 * P + 16, workspace_bytes=1 << 20), "workspace overlaps"),
    ("mlp_expert_linear", dict(y=P), "overlaps"), ("mlp_expert_linear", dict(y=4 * P), "overlaps"),
]


@pytest.mark.parametrize("name,over,says", REFUSED, ids=["%s-%s" % (n[4:], "-".join("%s" % k for k in o)) for n, o, _ in REFUSED])
def test_refusals(name, over, says):
    a = MAKE[name](**over)
    assert getattr(ops.lib(), name)(ctypes.addressof(a), None) == B.MLP_ERR_INVALID_ARGUMENT
    assert says in B.mlp_last_error()


def test_null_struct():
    for name in ops.EXPORTED:
        if name.endswith("_workspace"):
            n = ctypes.c_uint64()
            assert getattr(ops.lib(), name)(None, ctypes.addressof(n)) == B.MLP_ERR_INVALID_ARGUMENT
            assert getattr(ops.lib(), name)(ctypes.addressof(MAKE[name[:-10]]()), None) == B.MLP_ERR_INVALID_ARGUMENT
        else:
            assert getattr(ops.lib(), name)(None, None) == B.MLP_ERR_INVALID_ARGUMENT


def test_nothing_to_do():
    """No rows: answered without a HIP call, whatever the pointers."""
    for name, over in [("mlp_linear", dict(rows=0, x=None, y=None)), ("mlp_route", dict(tokens=0, logits=None, index=None)),
                       ("mlp_expert_linear", dict(tokens=0, x=None, y=None))]:
        a = MAKE[name](**over)
        assert getattr(ops.lib(), name)(ctypes.addressof(a), None) == B.MLP_OK


def test_workspace_queries():
    def need(name, a):
        n = ctypes.c_uint64(1)
        assert getattr(ops.lib(), name + "_workspace")(ctypes.addressof(a), ctypes.addressof(n)) == B.MLP_OK, B.mlp_last_error()
        return n.value

    assert need("mlp_expert_linear", expert_args(x=None, w=None, y=None)) == 0
    # the FP32 rows of every slot, padded to 16 bytes
    assert need("mlp_expert_linear", expert_args(combine=1, out_width=9)) == 4 * 2 * 12 * 4
    assert need("mlp_expert_linear", expert_args(combine=1, tokens=0)) == 0
    assert need("mlp_dispatch", dispatch_args()) == 0
    # a count for each expert and chunk of assignments: far below the assignments themselves
    assert 0 < need("mlp_dispatch", dispatch_args(tokens=1 << 20, k=8, experts=256)) <= 4 * (1 << 20) * 8
    assert need("mlp_dispatch", dispatch_args(tokens=(1 << 31) - 1, k=1, experts=1024)) <= 4 * 1024 * 1025


def test_too_many_tiles_is_unsupported():
    a = linear_args(rows=(1 << 31) - 1, out_width=1 << 20, ldy=1 << 20, x=1 << 56, w=1 << 40, y=1 << 44, in_width=8)
    assert ops.lib().mlp_linear(ctypes.addressof(a), None) == B.MLP_ERR_UNSUPPORTED


def test_torch_refusals():
    x, w = torch.zeros(4, 8, dtype=torch.float16), torch.zeros(8, 8, dtype=torch.float16)
    index = torch.zeros(4, 2, dtype=torch.int32)
    plan = ops.Dispatch(torch.zeros(9, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), torch.zeros(8, dtype=torch.int32))
    for f in (lambda: ops.linear(x, w), lambda: ops.route(x.float(), 2), lambda: ops.dispatch(index, 8),
              lambda: ops.expert_linear(x, w[None], plan, k=2)):
        with pytest.raises(ValueError, match="on the GPU"):
            f()
    for f, says in ((lambda: ops.linear(x.float(), w), "of type"), (lambda: ops.linear(x[0], w), "2-D"),
                    (lambda: ops.linear(None, w), "tensor"), (lambda: ops.dispatch(index.long(), 8), "of type"),
                    (lambda: ops.expert_linear(x, w[None], plan, k=2, rows="both"), "rows")):
        with pytest.raises(ValueError, match=says):
            f()


def test_numbers_that_do_not_fit_their_field_are_refused():
    """The torch form writes the structs' bytes itself: as ctypes does, but a larger number is not cut."""
    fields = dict(tokens=4, experts=8, k=2, dtype=2, score=0, groups=1, topk_groups=1, group_top=1, renormalise=0, scale=2.5,
                  logits=P, ld=8, bias=0, index=2 * P, weight=3 * P)
    assert ops._route_args(*fields.values()) == bytes(ops.RouteArgs(**fields))
    for name, value in (("k", 2 ** 32 + 2), ("groups", 2 ** 31), ("experts", -2 ** 32 + 8), ("tokens", 2 ** 63)):
        with pytest.raises(ValueError, match="RouteArgs"):
            ops._route_args(*{**fields, name: value}.values())
