"""GPU tests of the single operators' kernels one by one, at what each has of its own: its tiles' borders, the
strides and the aliases that its epilogue allows, its activations."""
import math

import pytest
import torch
import torch.autograd.forward_ad as fa

import ops_kernels as K
import ops_reference as R
from gpu_util import device, log
from mlp_neural_shading_amd import ops
from test_ops_kernels_host import EXPERTS, GATED, LINEAR

pytestmark = pytest.mark.gpu

ALL = [(name, size) for sizes in (LINEAR, GATED) for name, size in sizes.items()]
IDS = ["%s%s" % (name, "-gated" if size[3] else "") for name, size in ALL]
BOTH = pytest.mark.parametrize("name,size", ALL, ids=IDS)
HALF = {"fp16": torch.float16, "bf16": torch.bfloat16}


def gen(seed):
    return torch.Generator(device=device()).manual_seed(seed)


def rnd(g, *shape, dtype, scale=1.0):
    return (torch.randn(*shape, generator=g, device=device()) * scale).to(dtype)


def ran(name, x, w, gated):
    """Asserts that the layer of these operands is the kernel's that the test speaks of."""
    rows, k = x.shape
    n = w.shape[0] // (2 if gated else 1)
    assert K.linear_kernel(rows, k, n, gated, x.stride(0) if rows > 1 else k, w.stride(0), x.data_ptr() % 16 + K.FAR,
                           w.data_ptr() % 16 + 2 * K.FAR) == name


def block(t, left, right, fill):
    """t as a column block of a wider matrix, whose other columns hold `fill`."""
    wide = torch.full((t.shape[0], left + t.shape[1] + right), fill, dtype=t.dtype, device=t.device)
    wide[:, left:left + t.shape[1]] = t
    return wide, wide[:, left:left + t.shape[1]]


def layer(name, size, t, seed):
    rows, k, n, gated = size
    g, wide = gen(seed), n * (2 if gated else 1)
    x, w = rnd(g, rows, k, dtype=t), rnd(g, wide, k, dtype=t, scale=k ** -0.5)
    ran(name, x, w, gated)
    return x, w, rnd(g, wide, dtype=t), rnd(g, rows, n, dtype=t)


@BOTH
def test_strides_and_residual_in_place(name, size):
    """y, residual, x and w as column blocks of wider matrices, which hold NaN around the inputs and keep what they
    hold around the outputs; the residual beside y and as y itself.  The bits are those of the plain matrices, whose
    values are checked against 64 bits."""
    rows, k, n, gated = size
    log("strides", name, size)
    for t in HALF.values():
        for out in (t, torch.float32):
            x, w, b, r = layer(name, size, t, 1)
            r = r.to(out)
            want = ops.linear(x, w, b, residual=r, act="leaky_relu", gated=gated, out_dtype=out)
            if out == t:
                some = torch.cat([torch.arange(0, min(rows, 300)), torch.arange(max(0, rows - 300), rows)])
                R.check(want[some.to(device())], *R.linear64(x[some], w, b, r[some], "leaky_relu", gated), t, "plain")
            for left, right in ((8, 8), (2, 4)):
                _, xv = block(x, left, right, math.nan)
                _, wv = block(w, left, right + 2, math.nan)
                ran(name, xv, wv, gated)
                for l2, r2 in ((left, right), (1, 2), (3, 0)):
                    _, rv = block(r, l2, r2, math.nan)
                    whole, y = block(torch.zeros_like(r), l2 + 1, r2, 7.0)
                    ops.linear(xv, wv, b, residual=rv, act="leaky_relu", gated=gated, out=y, out_dtype=out)
                    assert torch.equal(y, want)
                    keep = torch.cat([whole[:, :l2 + 1], whole[:, l2 + 1 + n:]], 1)
                    assert bool((keep == 7).all())
                    whole, y = block(r, l2, r2, 7.0)
                    ops.linear(xv, wv, b, residual=y, act="leaky_relu", gated=gated, out=y, out_dtype=out)
                    assert torch.equal(y, want)
                    keep = torch.cat([whole[:, :l2], whole[:, l2 + n:]], 1)
                    assert bool((keep == 7).all())


@pytest.mark.parametrize("name", ["few", "few wide", "small", "mid", "big", "tile"])
def test_the_largest_strides(name):
    """Rows of y as far apart as they may be, the residual in place, and rows of x beyond 2^31 elements in all; a lane's
    offset within a tile is 32 bits."""
    rows, k, n, gated = {"big": (1100, 200, 8200, False), "tile": (1100, 200, 801, False)}.get(name, LINEAR[name])
    t, ld = torch.float16, 1 << 24
    g = gen(2)
    x, w, r = rnd(g, rows, k, dtype=t), rnd(g, n, k, dtype=t, scale=k ** -0.5), rnd(g, rows, n, dtype=t)
    far = torch.empty(rows * ld, dtype=t, device=device())
    step = ld if name != "tile" else ld - 1
    xv, y = far.as_strided((rows, k), (step, 1), 16384), far.as_strided((rows, n), (step, 1))
    xv.copy_(x)
    y.copy_(r)
    ran(name, xv, w, gated)
    log("largest strides", name, rows, k, n)
    ops.linear(xv, w, residual=y, act="relu", out=y)
    if name == "tile":
        x = block(x, 1, 0, 0)[1]  # odd rows too
    ran(name, x, w, gated)
    assert torch.equal(y, ops.linear(x, w, residual=r, act="relu"))


@BOTH
def test_nan_and_infinity_stay_in_their_rows(name, size):
    rows, k, n, gated = size
    x, w, b, r = layer(name, size, torch.bfloat16, 3)
    log("nan and infinity", name, size)
    clean = ops.linear(x, w, b, residual=r, act="relu", gated=gated)
    assert bool(torch.isfinite(clean).all())
    bad = [1, rows // 2, rows - 1]
    x[bad[0], k // 2], x[bad[1], k - 1], x[bad[2], 0] = math.nan, math.inf, -math.inf
    y = ops.linear(x, w, b, residual=r, act="none", gated=gated)
    assert bool(torch.isnan(y[bad[0]]).all()) and not bool(torch.isfinite(y[bad[1:]]).any())
    y = ops.linear(x, w, b, residual=r, act="relu", gated=gated)
    keep = torch.ones(rows, dtype=torch.bool, device=device())
    keep[bad] = False
    assert torch.equal(y[keep], clean[keep]) and bool(torch.isnan(y[bad[0]]).all())


def values(t):
    """Numbers of a type that an activation sees, to both sides: small, ordinary, large, zeros, subnormals."""
    v = torch.cat([torch.linspace(-6, 6, 20001), torch.linspace(-30, 30, 9001), torch.linspace(-100, 100, 2001),
                   2.0 ** torch.arange(-24, 15), -(2.0 ** torch.arange(-24, 15)), torch.tensor([0.0, -0.0, 1.0, -1.0])])
    return v.to(t)


def through_unit_weights(size, t, gated):
    """A layer whose sums are single inputs, exactly: weight row o takes column o % K, and the row that it gates column
    (o + 7) % K.  (x, w, the sums [rows, n], the factors or None)."""
    rows, k, n, _ = size
    v = values(t)
    x = v[torch.arange(rows * k) % v.numel()].view(rows, k).to(device())
    o = torch.arange(n, device=device())
    wide = n * (2 if gated else 1)
    w = torch.zeros(wide, k, dtype=t, device=device())
    w[o, o % k] = 1
    if gated:
        w[n + o, (o + 7) % k] = 1
    return x, w, x[:, o % k], x[:, (o + 7) % k] if gated else None


def act64(z, act):
    """(value, bound before the rounding): GELU within 3 * 2^-24 of |z|; SiLU's argument of exp2 is rounded
    twice, by 2^-24 of |z| log2(e) and of 32 more, exp2, the sum, the reciprocal and the products by 2^-23 each at
    most; leaky ReLU by half a step."""
    z = z.double()
    y = R.act64(z, act)
    if act == "gelu":
        return y, 3 * 2.0 ** -24 * z.abs()
    if act == "silu":
        return y, y.abs() * 2.0 ** -24 * (2 * z.abs() + 32 + 8)
    return y, y.abs() * 2.0 ** -24


def close(got, want, bound, t, what):
    lim = R.rounded(want, bound, t)
    fine = ((got.double() - want).abs() <= lim) | (want.abs() > torch.finfo(t).max) & torch.isinf(got)
    assert bool(fine.all()), (what, int((~fine).sum()), float(((got.double() - want).abs() / lim)[~fine].max()))


@pytest.mark.parametrize("act", ops.ACTIVATIONS)
@BOTH
def test_activations(name, size, act):
    """Of exact sums, in each kernel, to both 16-bit types."""
    rows, k, n, gated = size
    log("activation", name, size, act)
    for t in HALF.values():
        x, w, z, u = through_unit_weights(size, t, gated)
        ran(name, x, w, gated)
        y = ops.linear(x, w, act=act, gated=gated)
        want, bound = act64(z, act)
        if gated:
            u = u.double()
            want, bound = want * u, bound * u.abs() + 2.0 ** -24 * (want * u).abs()
        close(y, want, bound, t, act)


def test_the_last_slots_of_2_to_the_31():
    """As many slots as there can be, for the kernel with the largest tiles: the last one ends at 2^31 - 1."""
    n, t = 2 ** 31 - 1, torch.float16
    log("2^31 - 1 slots")
    x = torch.empty(n, 1, dtype=t, device=device())
    for i in range(0, n, 1 << 28):
        x[i:i + (1 << 28), 0] = (torch.arange(min(1 << 28, n - i), device=device()) % 61).to(t)
    w = torch.tensor([3.0, 5.0], dtype=t, device=device()).view(2, 1, 1)
    last = 1000
    offsets = torch.tensor([0, n - last, n], dtype=torch.int32, device=device())
    unused = torch.empty(n, dtype=torch.int32, device=device())  # slots and places: x is by slot, nothing is combined
    y = torch.full((n, 1), -1.0, dtype=t, device=device())
    ops.expert_linear(x, w, ops.Dispatch(offsets, unused, unused), k=1, rows="slots", out=y)
    for i in range(0, n, 1 << 28):
        part = slice(i, min(i + (1 << 28), n - last))
        assert torch.equal(y[part], x[part] * 3)
    assert torch.equal(y[-last:], x[-last:] * 5)


@pytest.mark.parametrize("act", ops.ACTIVATIONS)
@BOTH
def test_activations_into_fp32(name, size, act):
    """FP32 outputs, to a few roundings of FP32.  GELU as max(v, 0) - |v| h: h = 2^P is off by the roundings of P (the last
    by half a step of |P|, those before and the fit by as much again, all times ln 2) and by a step of exp2's, the
    result by half a step.  SiLU: exp by two steps, and the argument's second part, the sum, the reciprocal's step of
    Newton's and two products by half a step each, and what lies below FP32's smallest normal number."""
    rows, k, n, gated = size
    log("activation into fp32", name, size, act)
    for t in HALF.values():
        x, w, z, u = through_unit_weights(size, t, gated)
        ran(name, x, w, gated)
        y = ops.linear(x, w, act=act, gated=gated, out_dtype=torch.float32)
        z = z.double()
        want = R.act64(z, act)
        if act == "gelu":
            h = 0.5 * torch.erfc(z.abs() / math.sqrt(2))
            want = z.clamp(min=0) - z.abs() * h  # 1 + erf cancels in 64 bits too
            steps = 2.1 * (-torch.log2(h.clamp(min=2.0 ** -160))).clamp(min=1) + 2
            bound = want.abs() * 2.0 ** -24 + z.abs() * h * torch.where(z.abs() < 5.6, 2.0 ** -24 * steps, 1)  # h < 2^-26
        elif act == "silu":
            bound = want.abs() * 2.0 ** -24 * 10 + z.abs() * 2.0 ** -148
        else:
            bound = want.abs() * 2.0 ** -24
        if gated:
            u = u.double()
            want, bound = want * u, bound * u.abs() + 2.0 ** -24 * (want * u).abs()
        off = (y.double() - want).abs()
        lim = bound + 2.0 ** -149
        assert bool((off <= lim).all()), (int((off > lim).sum()), float((off / lim).max()))


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_activations_of_experts_into_fp32(act):
    """By slot and combined: the layer's own bits for k = 1."""
    x, w, z, _ = through_unit_weights((500, 64, 40, False), torch.bfloat16, False)
    w = torch.stack([w, w])
    plan = ops.dispatch((torch.arange(500, device=device()) % 2).int()[:, None], 2)
    want = ops.linear(x, w[0], act=act, out_dtype=torch.float32)
    by_slot = ops.expert_linear(x, w, plan, k=1, act=act, out_dtype=torch.float32)
    assert torch.equal(by_slot[plan.places.long()], want)
    assert torch.equal(ops.expert_linear(x, w, plan, k=1, act=act, combine=True, out_dtype=torch.float32), want)


@pytest.mark.parametrize("name", EXPERTS)
def test_experts_strides_and_residual_in_place(name):
    """The same of the experts' layers, by slot and combined: the bits of the plain matrices, and nothing written around."""
    tokens, k, experts, k_in, n, gated = EXPERTS[name]
    log("experts", name, EXPERTS[name])
    for t in HALF.values():
        g, wide = gen(5), n * (2 if gated else 1)
        x, w = rnd(g, tokens, k_in, dtype=t), rnd(g, experts, wide, k_in, dtype=t, scale=k_in ** -0.5)
        b, r = rnd(g, experts, wide, dtype=t), rnd(g, tokens, n, dtype=t)
        index = torch.randint(-1, experts, (tokens, k), generator=g, device=device(), dtype=torch.int32)
        plan = ops.dispatch(index, experts)
        used = int(plan.offsets[-1])
        by_slot = ops.expert_linear(x, w, plan, b, k=k, act="relu", gated=gated)
        combined = ops.expert_linear(x, w, plan, b, k=k, act="relu", gated=gated, combine=True, residual=r)
        if tokens < 10000:
            want, bound, _ = R.experts64(x, w, tuple(plan), k, b, "relu", gated)
            R.check(by_slot[:used], want[:used], bound[:used], t, "by slot")
        pad = 2 if k_in % 2 == 0 else 1  # odd rows stay odd
        _, xv = block(x, pad, 2 * pad, math.nan)
        around = torch.full((experts, wide + 3, k_in + 4), math.nan, dtype=t, device=device())
        around[:, 1:wide + 1, 2:2 + k_in] = w
        wv = around[:, 1:wide + 1, 2:2 + k_in]
        assert K.expert_kernel(tokens, k, experts, k_in, n, gated, xv.stride(0), wv.stride(1), wv.stride(0) if name != "tile" else None,
                               xv.data_ptr() % 16 + K.FAR, wv.data_ptr() % 16 + 2 * K.FAR) == name
        whole, y = block(torch.zeros_like(by_slot), 3, 2, 7.0)
        ops.expert_linear(xv, wv, plan, b, k=k, act="relu", gated=gated, out=y)
        assert torch.equal(y[:used], by_slot[:used]) and bool((y[used:] == 0).all())
        assert bool((whole[:, :3] == 7).all()) and bool((whole[:, 3 + n:] == 7).all())
        whole, y = block(r, 1, 4, 7.0)
        ops.expert_linear(xv, wv, plan, b, k=k, act="relu", gated=gated, combine=True, residual=y, out=y)
        assert torch.equal(y, combined)
        assert bool((whole[:, :1] == 7).all()) and bool((whole[:, 1 + n:] == 7).all())


def test_forward_mode_duals_are_refused_anywhere():
    t = torch.bfloat16
    x, w, b = torch.ones(4, 8, dtype=t, device=device()), torch.ones(6, 8, dtype=t, device=device()), torch.ones(6, dtype=t, device=device())
    r = torch.zeros(4, 6, dtype=t, device=device())
    weight = torch.ones(4, 1, device=device())
    plan = ops.dispatch(torch.zeros(4, 1, dtype=torch.int32, device=device()), 1)
    want = ops.linear(x, w, b, residual=r)
    calls = [lambda **d: ops.linear(d.get("x", x), d.get("w", w), d.get("b", b), residual=d.get("r", r)),
             lambda **d: ops.expert_linear(d.get("x", x), d["w"][None] if "w" in d else w[None], plan, d["b"][None] if "b" in d else b[None],
                                           k=1, combine=True, weight=d.get("weight", weight), residual=d.get("r", r))]
    with fa.dual_level():
        for call, names in zip(calls, ("x w b r", "x w b r weight")):
            for name in names.split():
                plain = locals()[name]
                with pytest.raises(ValueError, match="tangent"):
                    call(**{name: fa.make_dual(plain, torch.ones_like(plain))})
            assert torch.equal(call(), want)
            assert torch.equal(call(x=fa.unpack_dual(fa.make_dual(x, torch.ones_like(x))).primal), want)
        logits = torch.zeros(2, 4, device=device())
        with pytest.raises(ValueError, match="tangent"):
            ops.route(fa.make_dual(logits, logits), 2)
        with pytest.raises(ValueError, match="tangent"):
            ops.route(logits, 2, bias=fa.make_dual(logits[0], logits[0]))


def test_autograd_sees_that_out_was_written():
    """A graph that saved the old contents of `out` refuses its backward pass, as after torch's own products."""
    t = torch.float16
    x, w = torch.ones(4, 8, dtype=t, device=device()), torch.ones(6, 8, dtype=t, device=device())
    plan = ops.dispatch(torch.zeros(4, 1, dtype=torch.int32, device=device()), 1)
    for write in (lambda out: ops.linear(x, w, out=out), lambda out: ops.expert_linear(x, w[None], plan, k=1, out=out),
                  lambda out: ops.linear(x, w, residual=out, out=out)):
        leaf = torch.ones(4, 6, dtype=t, device=device(), requires_grad=True)
        saved = leaf.exp()
        write(saved.detach())
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            saved.sum().backward()
        with torch.inference_mode():
            assert float(write(torch.zeros(4, 6, dtype=t, device=device()))[0, 0]) == 8.0


def test_a_single_rows_stride_means_nothing():
    """One row of a matrix whose rows lie farther apart than they may for y: there is no next row to step to."""
    t, far = torch.float16, (1 << 24) + 8
    wide = torch.zeros(2, far, dtype=t, device=device())
    x, w = torch.ones(1, 8, dtype=t, device=device()), torch.ones(6, 8, dtype=t, device=device())
    y = ops.linear(x, w, residual=wide[:1, :6], out=wide[1:, :6])
    assert y.stride(0) == far and bool((y == 8).all())
    plan = ops.dispatch(torch.zeros(1, 1, dtype=torch.int32, device=device()), 1)
    y = ops.expert_linear(x, w[None], plan, k=1, combine=True, residual=wide[1:, :6], out=wide[:1, :6])
    assert bool((y == 16).all())
    narrow = torch.ones(1, 4, device=device()).expand(1, 4)
    assert ops.route(narrow, 2).index.tolist() == [[0, 1]]
    assert bool((ops.linear(torch.ones(3, 8, dtype=t, device=device()), w[:1].as_strided((1, 8), (1 << 30, 1))) == 8).all())
