"""GPU tests of the single operators (include/mlp_ops.h) against their plain forms in 64 bits, at the sizes and
inputs where they can go wrong.  The tolerances are those of ops_reference: an FP32 sum's and one rounding."""
import math

import pytest
import torch

import ops_reference as R
from gpu_util import device, log
from mlp_neural_shading_amd import binding as B
from mlp_neural_shading_amd import ops

pytestmark = pytest.mark.gpu

HALF = {"fp16": torch.float16, "bf16": torch.bfloat16}


def rnd(gen, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(dtype)


def gpu(t):
    return None if t is None else t.to(device())


def gen(seed):
    return torch.Generator().manual_seed(seed)


def padded(t, left, right, fill):
    """The values of t as a column block of a wider matrix, whose other columns hold `fill`."""
    wide = torch.full((t.shape[0], left + t.shape[1] + right), fill, dtype=t.dtype, device=t.device)
    wide[:, left:left + t.shape[1]] = t
    return wide, wide[:, left:left + t.shape[1]]


# ---- linear ----------------------------------------------------------------------------------------

# (rows, in, out): single rows, odd sizes, tile borders and one past them, K below, at and past a stage
SIZES = [(1, 1, 1), (1, 1024, 64), (2, 7, 3), (3, 64, 65), (5, 8, 1000), (16, 100, 48), (17, 129, 33), (31, 200, 130),
         (64, 64, 64), (65, 63, 63), (100, 320, 96), (127, 65, 257), (128, 128, 128), (129, 256, 255), (256, 512, 256),
         (300, 1001, 77), (513, 72, 520)]


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("rows,k,n", SIZES)
def test_linear(rows, k, n, dtype):
    g, t = gen(rows * 7 + k), HALF[dtype]
    x, w = rnd(g, rows, k, dtype=t), rnd(g, n, k, dtype=t, scale=k ** -0.5)
    b, r = rnd(g, n, dtype=t), rnd(g, rows, n, dtype=t)
    log("linear", rows, k, n, dtype)
    R.check(ops.linear(gpu(x), gpu(w)), *R.linear64(x, w), t, "plain")
    y = ops.linear(gpu(x), gpu(w), gpu(b), residual=gpu(r), act="leaky_relu")
    R.check(y, *R.linear64(x, w, b, r, "leaky_relu"), t, "epilogue")
    y = ops.linear(gpu(x), gpu(w), gpu(b), residual=gpu(r.float()), act="gelu", out_dtype=torch.float32)
    R.check(y, *R.linear64(x, w, b, r, "gelu"), torch.float32, "fp32")


# (rows, in, out, gated): sizes that take the larger tiles, whole and with borders in every direction, K below a
# stage, of one, of whole ones and with a rest
LARGE = [(5000, 200, 1800, False), (5000, 40, 1801, False), (4864, 128, 2048, False), (2600, 264, 1700, True),
         (2500, 72, 1500, False), (2048, 64, 2048, False), (1300, 200, 1100, True), (600, 136, 700, False), (640, 192, 640, False),
         (300, 64, 650, True), (9000, 72, 64, False), (9001, 33, 50, False), (4000, 64, 32, True), (700, 101, 903, False),
         (513, 77, 455, True), (150, 1040, 1000, False), (524300, 24, 20, False), (524289, 33, 16, True),
         (20000, 64, 128, False), (5000, 202, 1800, False), (2500, 130, 1500, True), (700, 102, 640, False)]


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("rows,k,n,gated", LARGE)
def test_linear_large(rows, k, n, gated, dtype):
    g, t = gen(rows + k), HALF[dtype]
    wide = 2 * n if gated else n
    x, w = rnd(g, rows, k, dtype=t), rnd(g, wide, k, dtype=t, scale=k ** -0.5)
    b, r = rnd(g, wide, dtype=t), rnd(g, rows, n, dtype=t)
    log("linear large", rows, k, n, gated, dtype)
    y = ops.linear(gpu(x), gpu(w), gpu(b), residual=gpu(r), act="silu", gated=gated)
    R.check(y, *R.linear64(x, w, b, r, "silu", gated), t, "epilogue")
    y = ops.linear(gpu(x), gpu(w), residual=gpu(r.float()), gated=gated, out_dtype=torch.float32)
    R.check(y, *R.linear64(x, w, None, r, "none", gated), torch.float32, "fp32")


@pytest.mark.parametrize("rows,n", [(5000, 1800), (4000, 900), (2500, 640)])
@pytest.mark.parametrize("k", [64, 66, 72, 96, 126, 128, 130, 184, 190, 192, 194, 254, 65, 127, 129, 191, 34])
def test_last_columns_count_once(rows, n, k):
    """Whole numbers, whose sums are exact, for widths that end anywhere in a stage; a row stride beyond the width
    holds NaN, and one row an infinity in the first column of its last 64."""
    t = torch.bfloat16
    ld = k + 6 + k % 2
    x, w = (torch.full((r, ld), math.nan, dtype=t, device=device()) for r in (rows, n))
    x[:, :k] = torch.randint(-3, 4, (rows, k), generator=gen(k)).to(device())
    w[:, :k] = torch.randint(1, 4, (n, k), generator=gen(k + 1)).to(device())
    want = x[:, :k].float().cpu() @ w[:, :k].float().cpu().T
    got = ops.linear(x[:, :k], w[:, :k], out_dtype=torch.float32)
    assert torch.equal(got.cpu(), want)
    x[rows - 2, max(k - 64, 0)] = math.inf
    want[rows - 2] = math.inf
    assert torch.equal(ops.linear(x[:, :k], w[:, :k], out_dtype=torch.float32).cpu(), want)
    index = (torch.arange(rows, device=device()) * 7 // rows % 3).int()[:, None]
    plan = ops.dispatch(index, 3)
    each = torch.stack([w, 2 * w, -w])[:, :, :k]
    x[rows - 2, max(k - 64, 0)] = 1
    want = x[:, :k].float().cpu() @ w[:, :k].float().cpu().T * torch.tensor([1., 2., -1.])[index.cpu().long()]
    got = ops.expert_linear(x[:, :k], each, plan, k=1, combine=True, out_dtype=torch.float32)
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("act", ops.ACTIVATIONS)
@pytest.mark.parametrize("rows,k,n", [(1, 96, 40), (9, 130, 33), (70, 64, 96), (260, 136, 200)])
def test_linear_activations_and_gates(rows, k, n, act):
    g, t = gen(rows + n), torch.bfloat16
    x = rnd(g, rows, k, dtype=t, scale=3.0)
    w, b = rnd(g, 2 * n, k, dtype=t, scale=k ** -0.5), rnd(g, 2 * n, dtype=t)
    r = rnd(g, rows, n, dtype=t)
    log("activation", act, rows, k, n)
    R.check(ops.linear(gpu(x), gpu(w), gpu(b), act=act), *R.linear64(x, w, b, None, act), t, "plain")
    y = ops.linear(gpu(x), gpu(w), gpu(b), residual=gpu(r), act=act, gated=True)
    R.check(y, *R.linear64(x, w, b, r, act, True), t, "gated")
    y = ops.linear(gpu(x), gpu(w), act=act, gated=True, out_dtype=torch.float32)
    R.check(y, *R.linear64(x, w, None, None, act, True), torch.float32, "gated fp32")


@pytest.mark.parametrize("left,right", [(8, 8), (1, 2), (3, 0), (16, 5)])
@pytest.mark.parametrize("rows,k,n", [(1, 72, 24), (12, 64, 40), (90, 136, 72), (300, 264, 280)])
def test_linear_strides(rows, k, n, left, right):
    """Column blocks of wider matrices, aligned or not; the columns around them hold NaN on the way in and
    their own values afterwards."""
    g, t = gen(rows + left), torch.float16
    x, w = rnd(g, rows, k, dtype=t), rnd(g, n, k, dtype=t, scale=k ** -0.5)
    r = rnd(g, rows, n, dtype=t)
    _, xv = padded(gpu(x), left, right, math.nan)
    _, wv = padded(gpu(w), left, right, math.nan)
    _, rv = padded(gpu(r), left, right, math.nan)
    whole, out = padded(torch.zeros_like(gpu(r)), left, right, 7.0)
    log("strides", rows, k, n, left, right)
    assert ops.linear(xv, wv, residual=rv, act="silu", out=out) is out
    R.check(out, *R.linear64(x, w, None, r, "silu"), t)
    assert bool((whole[:, :left] == 7).all()) and bool((whole[:, left + n:] == 7).all())


def test_linear_residual_in_place_and_beside():
    """The residual may be the output itself; and x, y as column blocks of one matrix."""
    g, t = gen(3), torch.bfloat16
    for rows, k, n in ((1, 64, 64), (7, 64, 64), (200, 64, 64), (333, 200, 96)):
        x, w, r = rnd(g, rows, k, dtype=t), rnd(g, n, k, dtype=t, scale=k ** -0.5), rnd(g, rows, n, dtype=t)
        y = gpu(r)
        ops.linear(gpu(x), gpu(w), residual=y, out=y)
        R.check(y, *R.linear64(x, w, None, r), t, "in place")
        both = torch.full((rows, k + n), 3.0, dtype=t, device=device())
        both[:, :k] = gpu(x)
        ops.linear(both[:, :k], gpu(w), out=both[:, k:])
        R.check(both[:, k:], *R.linear64(x, w), t, "beside")
        assert torch.equal(both[:, :k].cpu(), x)


def test_linear_nan_and_infinity_stay_in_their_rows():
    g, t = gen(5), torch.float16
    for rows, k, n in ((4, 72, 40), (100, 72, 40), (300, 200, 300)):
        x, w = rnd(g, rows, k, dtype=t), rnd(g, n, k, dtype=t, scale=k ** -0.5)
        clean = ops.linear(gpu(x), gpu(w), act="relu")
        x[1, 5], x[3, k - 1] = math.nan, math.inf
        y = ops.linear(gpu(x), gpu(w), act="relu")
        assert torch.isnan(y[1]).all() and not torch.isfinite(ops.linear(gpu(x), gpu(w))[3]).any()
        keep = [i for i in range(rows) if i not in (1, 3)]
        assert torch.equal(y[keep], clean[keep])


def test_linear_no_rows():
    x, w = torch.empty(0, 8, dtype=torch.float16, device=device()), torch.ones(4, 8, dtype=torch.float16, device=device())
    assert ops.linear(x, w).shape == (0, 4)


def test_linear_far_offsets():
    """x and y with rows so far apart that byte offsets pass 32 bits."""
    g, t = gen(11), torch.float16
    rows, k, n, ld = 300, 64, 64, 8_000_000
    x, w = rnd(g, rows, k, dtype=t), rnd(g, n, k, dtype=t, scale=k ** -0.5)
    big = torch.empty(rows * ld, dtype=t, device=device())
    xv, yv = big.as_strided((rows, k), (ld, 1)), big.as_strided((rows, n), (ld, 1), 4096)
    xv.copy_(gpu(x))
    ops.linear(xv, gpu(w), out=yv)
    R.check(yv.contiguous(), *R.linear64(x, w), t)


def test_gradients_are_refused():
    x = torch.ones(2, 8, dtype=torch.float16, device=device(), requires_grad=True)
    w = torch.ones(4, 8, dtype=torch.float16, device=device())
    with pytest.raises(ValueError, match="gradient"):
        ops.linear(x, w)
    with torch.no_grad():
        assert float(ops.linear(x, w).sum()) == 64.0


# ---- route -----------------------------------------------------------------------------------------

def check_route(logits, k, **kw):
    want_i, want_w = R.route64(logits, k, **kw)
    bias = kw.pop("bias", None)
    got = ops.route(gpu(logits), k, bias=gpu(bias), **kw)
    assert torch.equal(got.index.cpu(), want_i)
    # computed in 64 bits and rounded once, or to a few steps of FP32: 8 half-steps
    lim = 8 * 2.0 ** -24 * want_w.abs() + 2.0 ** -149
    assert bool(((got.weight.cpu().double() - want_w).abs() <= lim).all())
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens,experts,k", [(1, 1, 1), (3, 2, 2), (5, 7, 3), (33, 64, 4), (40, 65, 8), (17, 128, 2),
                                              (70, 200, 6), (9, 256, 8), (4, 300, 32), (5, 600, 5), (3, 1024, 32)])
def test_route(tokens, experts, k, dtype):
    g = gen(tokens + experts)
    logits, bias = rnd(g, tokens, experts, scale=1.5).to(dtype), rnd(g, experts, scale=0.1)
    log("route", tokens, experts, k, dtype)
    for score in ops.SCORES:
        check_route(logits, k, score=score)
        check_route(logits, k, score=score, bias=bias, renormalise=True, scale=2.5)


@pytest.mark.parametrize("experts,groups,topk_groups", [(8, 2, 1), (64, 8, 4), (256, 8, 3), (160, 5, 2), (96, 96, 7), (512, 4, 4),
                                                        (1024, 128, 9), (12, 6, 2), (264, 2, 1), (10, 2, 1), (63, 3, 2),
                                                        (160, 8, 3), (330, 6, 2), (500, 10, 4), (640, 8, 4)])
@pytest.mark.parametrize("group_top", [1, 2])
def test_route_groups(experts, groups, topk_groups, group_top):
    g = gen(experts + groups)
    logits, bias = rnd(g, 37, experts), rnd(g, experts, scale=0.2)
    k = min(6, topk_groups * (experts // groups))
    for score in ops.SCORES:
        check_route(logits, k, score=score, bias=bias, groups=groups, topk_groups=topk_groups, group_top=group_top,
                    renormalise=True)
        check_route(logits, k, score=score, groups=groups, topk_groups=topk_groups, group_top=group_top)


def test_route_ties_go_to_the_lower_index():
    g = gen(1)
    logits = torch.randint(-2, 3, (64, 200), generator=g).float()
    for score in ops.SCORES:
        check_route(logits, 7, score=score)
        check_route(logits, 7, score=score, bias=torch.zeros(200), renormalise=True)
        check_route(logits, 7, score=score, groups=10, topk_groups=3, group_top=2)
        check_route(torch.zeros(3, 64), 8, score=score, groups=8, topk_groups=3)


def test_route_choices_closer_than_fp32_tells_apart():
    """Sigmoid scores near 1 whose differences FP32 would round away, and biases a step apart."""
    base = torch.linspace(14.0, 18.0, 96)[torch.randperm(96, generator=gen(2))]
    logits = base.expand(5, 96).contiguous()
    check_route(logits, 8, score="sigmoid", bias=torch.full((96,), 0.25))
    check_route(logits, 8, score="sigmoid", bias=torch.full((96,), 0.25), groups=8, topk_groups=2, group_top=2)
    bias = 1.0 + torch.arange(96) % 5 * 2.0 ** -23
    check_route(logits, 8, score="sigmoid", bias=bias)
    check_route(-logits * 2, 8, score="softmax", bias=bias)


@pytest.mark.parametrize("experts,groups", [(64, 8), (128, 4), (256, 8), (500, 1), (512, 16), (900, 1)])
def test_route_near_choices(experts, groups):
    """The same for every layout of experts over lanes, and rows of which only some are near."""
    g = gen(experts)
    base = torch.linspace(14.0, 18.0, experts)[torch.randperm(experts, generator=g)]
    logits = torch.where(torch.arange(37)[:, None] % 3 == 1, base, rnd(g, 37, experts, scale=2.0))
    bias = torch.full((experts,), 0.25)
    for k in (1, 8, 20):
        check_route(logits, k, score="sigmoid", bias=bias, renormalise=True)
        check_route(logits * 3, k, score="softmax", bias=bias)
    if groups > 1:
        check_route(logits, 6, score="sigmoid", bias=bias, groups=groups, topk_groups=groups // 2, group_top=2)


def test_route_masks():
    """Experts masked by -inf or NaN are never chosen; rows with fewer left than k, or none, end in -1; the
    lowest finite value is a logit like any other."""
    g = gen(4)
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        logits = rnd(g, 12, 70).to(dtype)
        logits[0] = -math.inf
        logits[1, 3:] = -math.inf
        logits[2] = math.nan
        logits[3, ::2] = math.nan
        logits[4] = torch.finfo(dtype).min
        logits[5, 1:] = torch.finfo(dtype).min
        logits[6, 9] = math.inf
        logits[7, 9] = logits[7, 60] = math.inf
        logits[8, :68] = -math.inf
        for score in ops.SCORES:
            for kw in (dict(), dict(renormalise=True), dict(groups=10, topk_groups=2, group_top=2, renormalise=True)):
                got = check_route(logits, 5, score=score, **kw)
                assert got.index[0].tolist() == [-1] * 5 and got.weight[0].tolist() == [0.0] * 5
                assert got.index[2].tolist() == [-1] * 5
        bias = rnd(g, 70, scale=0.1)
        bias[7], bias[20], bias[21] = -math.inf, math.nan, math.inf
        for score in ops.SCORES:
            got = check_route(logits, 5, score=score, bias=bias)
            assert not bool(((got.index == 7) | (got.index == 20)).any())


def test_route_strides_and_no_tokens():
    g = gen(6)
    wide = rnd(g, 20, 100)
    want_i, _ = R.route64(wide[:, 11:81], 4)
    assert torch.equal(ops.route(gpu(wide)[:, 11:81], 4).index.cpu(), want_i)
    assert ops.route(torch.empty(0, 8, device=device()), 2).index.shape == (0, 2)


# ---- dispatch --------------------------------------------------------------------------------------

@pytest.mark.parametrize("tokens,k,experts", [(0, 1, 4), (1, 1, 1), (3, 2, 5), (48, 4, 64), (64, 1, 2), (1000, 3, 7), (4096, 1, 16),
                                              (4097, 1, 1024), (3000, 8, 256), (5, 32, 1000), (40000, 2, 33)])
def test_dispatch(tokens, k, experts):
    index = torch.randint(-1, experts + 1, (tokens, k), generator=gen(tokens + experts), dtype=torch.int32)  # with dropped ones
    log("dispatch", tokens, k, experts)
    plan = ops.dispatch(gpu(index), experts)
    for got, want, name in zip(plan, R.dispatch64(index, experts), plan._fields):
        assert torch.equal(got.cpu(), want), name


def test_dispatch_corner_rows():
    for index, experts in ((torch.full((5000, 1), 3), 8), (torch.full((5000, 2), -1), 8), (torch.full((70, 4), 2 ** 31 - 1), 3),
                           (torch.full((6, 2), -2 ** 31), 3), (torch.arange(9000).view(-1, 1) % 2, 2)):
        index = index.to(torch.int32)
        for got, want in zip(ops.dispatch(gpu(index), experts), R.dispatch64(index, experts)):
            assert torch.equal(got.cpu(), want)


def test_dispatch_large():
    """Many chunks, against torch's stable sort."""
    index = torch.randint(0, 300, (1 << 21, 3), generator=gen(9), dtype=torch.int32).to(device())
    offsets, slots, places = ops.dispatch(index, 300)
    flat = index.view(-1).long()
    order = torch.sort(flat, stable=True).indices
    assert torch.equal(slots.long(), order)
    assert torch.equal(places.long()[order], torch.arange(flat.numel(), device=device()))
    assert torch.equal(offsets.long()[1:], torch.bincount(flat, minlength=300).cumsum(0)) and int(offsets[0]) == 0


# ---- the experts' layers -----------------------------------------------------------------------------

EXPERT_SIZES = [(1, 1, 1, 8, 8), (1, 2, 3, 40, 24), (3, 4, 9, 33, 17), (8, 4, 32, 128, 96), (64, 2, 4, 64, 64), (37, 3, 5, 200, 130),
                (300, 1, 16, 64, 64), (500, 2, 3, 96, 264), (260, 6, 70, 72, 40), (20, 2, 200, 16, 16), (3000, 2, 4, 72, 1200),
                (900, 2, 5, 136, 700), (4000, 1, 16, 64, 64), (1000, 3, 20, 40, 264), (700, 2, 6, 33, 300), (530000, 1, 5, 40, 12)]


def routed(g, tokens, k, experts, drop=True):
    index = torch.randint(-1 if drop else 0, experts, (tokens, k), generator=g, dtype=torch.int32)
    return index, tuple(t for t in R.dispatch64(index, experts))


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("tokens,k,experts,k_in,n", EXPERT_SIZES)
def test_expert_linear(tokens, k, experts, k_in, n, dtype):
    g, t = gen(tokens + experts), HALF[dtype]
    _, plan = routed(g, tokens, k, experts)
    on_gpu = ops.Dispatch(*map(gpu, plan))
    w, b = rnd(g, experts, 2 * n, k_in, dtype=t, scale=k_in ** -0.5), rnd(g, experts, 2 * n, dtype=t)
    weight, r = torch.rand(tokens, k, generator=g), rnd(g, tokens, n, dtype=t)
    for rows in ("tokens", "slots"):
        x = rnd(g, tokens if rows == "tokens" else tokens * k, k_in, dtype=t)
        for gated in (False, True):
            wg, bg = (w, b) if gated else (w[:, :n].contiguous(), b[:, :n].contiguous())
            kw = dict(act="silu", gated=gated, rows=rows)
            log("experts", tokens, k, experts, k_in, n, dtype, rows, gated)
            out = torch.full((tokens * k, n), 5.0, dtype=t, device=device())
            ops.expert_linear(gpu(x), gpu(wg), on_gpu, gpu(bg), k=k, out=out, **kw)
            want, bound, used = R.experts64(x, wg, plan, k, bg, **kw)
            R.check(out[:used], want[:used], bound[:used], t, "by slot")
            assert bool((out[used:] == 5).all())  # rows behind the last slot in use
            y = ops.expert_linear(gpu(x), gpu(wg), on_gpu, gpu(bg), k=k, combine=True, weight=gpu(weight), residual=gpu(r), **kw)
            want, bound, _ = R.experts64(x, wg, plan, k, bg, combine=True, weight=weight, residual=r, **kw)
            R.check(y, want, bound, t, "combined")
    y = ops.expert_linear(gpu(x), gpu(wg), on_gpu, k=k, rows="slots", gated=True, combine=True, out_dtype=torch.float32)
    want, bound, _ = R.experts64(x, wg, plan, k, gated=True, rows="slots", combine=True)
    R.check(y, want, bound, torch.float32, "combined fp32, no weights")


def test_expert_linear_strides_and_in_place_residual():
    g, t = gen(21), torch.bfloat16
    tokens, k, experts, k_in, n = 150, 2, 6, 72, 56
    _, plan = routed(g, tokens, k, experts)
    on_gpu = ops.Dispatch(*map(gpu, plan))
    x, w = rnd(g, tokens, k_in, dtype=t), rnd(g, experts, n, k_in, dtype=t, scale=k_in ** -0.5)
    r = rnd(g, tokens, n, dtype=t)
    for left, right in ((8, 8), (1, 2)):
        _, xv = padded(gpu(x), left, right, math.nan)
        wide = torch.full((experts, n + 3, k_in + left + right), math.nan, dtype=t, device=device())
        wide[:, 1:n + 1, left:left + k_in] = gpu(w)
        wv = wide[:, 1:n + 1, left:left + k_in]
        whole, out = padded(gpu(r), left, right, 7.0)
        ops.expert_linear(xv, wv, on_gpu, k=k, combine=True, residual=out, out=out)
        want, bound, _ = R.experts64(x, w, plan, k, combine=True, residual=r)
        R.check(out, want, bound, t)
        assert bool((whole[:, :left] == 7).all()) and bool((whole[:, left + n:] == 7).all())


def test_expert_linear_all_rows_to_one_expert_or_none():
    g, t = gen(22), torch.float16
    x, w = rnd(g, 700, 64, dtype=t), rnd(g, 9, 40, 64, dtype=t, scale=0.125)
    for value in (0, 4, 8, -1):
        index = torch.full((700, 1), value, dtype=torch.int32)
        plan = R.dispatch64(index, 9)
        y = ops.expert_linear(gpu(x), gpu(w), ops.Dispatch(*map(gpu, plan)), k=1, combine=True)
        R.check(y, *R.experts64(x, w, plan, 1, combine=True)[:2], t, value)


@pytest.mark.parametrize("k", [1, 2, 5, 9])
def test_combine_every_assignment_count(k):
    """Odd output widths and counts of experts per token, some tokens without any, the same expert twice, and NaN in
    the outputs of no consequence: the rows behind the last slot."""
    g, t = gen(k), torch.float16
    tokens, experts, k_in, n = 90, 4, 40, 37
    index = torch.randint(-1, experts, (tokens, k), generator=g, dtype=torch.int32)
    index[5] = -1
    index[6] = 2
    plan = R.dispatch64(index, experts)
    x, w = rnd(g, tokens, k_in, dtype=t), rnd(g, experts, n, k_in, dtype=t, scale=k_in ** -0.5)
    weight = torch.randn(tokens, k, generator=g)
    for residual in (None, rnd(g, tokens, n)):
        y = ops.expert_linear(gpu(x), gpu(w), ops.Dispatch(*map(gpu, plan)), k=k, combine=True, weight=gpu(weight),
                              residual=gpu(residual), out_dtype=torch.float32)
        want, bound, _ = R.experts64(x, w, plan, k, combine=True, weight=weight, residual=residual)
        R.check(y, want, bound, torch.float32)
        assert torch.equal(y[5].cpu(), torch.zeros(n) if residual is None else residual[5])


def test_expert_linear_bad_plans_stay_in_bounds():
    """Offsets, slots and places that no dispatch gives: clamped, the rows that are right stay right.  (Shown by
    reading first: every index is clamped to its buffer before use.)"""
    g, t = gen(77), torch.float16
    x, w = rnd(g, 40, 64, dtype=t), rnd(g, 3, 32, 64, dtype=t, scale=0.125)
    index = torch.randint(0, 3, (40, 2), generator=g, dtype=torch.int32)
    offsets, slots, places = R.dispatch64(index, 3)
    y = ops.expert_linear(gpu(x), gpu(w), ops.Dispatch(gpu(offsets), gpu(slots), gpu(places)), k=2)
    far = slots.clone()
    far[-3:] = torch.tensor([-7, 80, 2 ** 31 - 1], dtype=torch.int32)
    bad = ops.expert_linear(gpu(x), gpu(w), ops.Dispatch(gpu(offsets), gpu(far), gpu(places)), k=2)
    assert torch.equal(bad[:-3], y[:-3])
    wide = offsets.clone()
    wide[0], wide[3] = -5, 2 ** 31 - 1
    assert torch.equal(ops.expert_linear(gpu(x), gpu(w), ops.Dispatch(gpu(wide), gpu(slots), gpu(places)), k=2), y)
    out = places.clone()
    out[10], out[11] = -9, 80  # token 5: both dropped
    z = ops.expert_linear(gpu(x), gpu(w), ops.Dispatch(gpu(offsets), gpu(slots), gpu(out)), k=2, combine=True)
    assert bool((z[5] == 0).all())


# ---- together ----------------------------------------------------------------------------------------

def layer_of_experts(x, w_router, w1, w2, k):
    index, weight = ops.route(ops.linear(x, w_router, out_dtype=torch.float32), k, renormalise=True)
    plan = ops.dispatch(index, w1.shape[0])
    h = ops.expert_linear(x, w1, plan, k=k, act="silu", gated=True)
    return ops.expert_linear(h, w2, plan, k=k, rows="slots", combine=True, weight=weight, residual=x), index


def expert_weights(seed, experts, d, hidden, t):
    g = gen(seed)
    return (rnd(g, experts, d, dtype=t, scale=d ** -0.5), rnd(g, experts, 2 * hidden, d, dtype=t, scale=d ** -0.5),
            rnd(g, experts, d, hidden, dtype=t, scale=hidden ** -0.5))


@pytest.mark.parametrize("tokens", [1, 5, 130, 1000])
def test_a_layer_of_experts(tokens):
    """Router, dispatch and both layers of the experts in a row, against the same in 64 bits along the choices made."""
    t, d, hidden, experts, k = torch.bfloat16, 96, 80, 12, 3
    w_router, w1, w2 = expert_weights(31, experts, d, hidden, t)
    x = rnd(gen(tokens), tokens, d, dtype=t)
    log("layer of experts", tokens)
    y, index = layer_of_experts(gpu(x), gpu(w_router), gpu(w1), gpu(w2), k)
    logits = ops.linear(gpu(x), gpu(w_router), out_dtype=torch.float32)
    R.check(logits, *R.linear64(x, w_router), torch.float32, "logits")
    want_i, weight = R.route64(logits, k, renormalise=True)
    assert torch.equal(index.cpu(), want_i)
    plan = R.dispatch64(want_i, experts)
    h, eh, _ = R.experts64(x, w1, plan, k, act="silu", gated=True)
    want, e, _ = R.experts64(h.to(t), w2, plan, k, rows="slots", combine=True, weight=weight, residual=x)
    # h is rounded to bfloat16 on both sides, to neighbours where FP32 and 64 bits fall either side of a border:
    # one step of h, through |w2| and the weights
    step = (h.abs() * torch.finfo(t).eps + eh)
    far, _, _ = R.experts64(step, w2.abs(), plan, k, rows="slots", combine=True, weight=weight)
    # the FP32 weights: 8 half-steps of each term
    near, _, _ = R.experts64(h.abs(), w2.abs(), plan, k, rows="slots", combine=True, weight=weight)
    R.check(y, want, e + far + near * 2.0 ** -21, t)


def test_two_streams_at_once():
    """Two runs on two streams, each with its own workspace, give what each gives alone."""
    t = torch.float16
    weights = [gpu(w) for w in expert_weights(41, 16, 128, 64, t)]
    xs = [gpu(rnd(gen(s), 600, 128, dtype=t)) for s in (1, 2)]
    alone = [layer_of_experts(x, *weights, 4)[0] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for s, x in zip(streams, xs):
        with torch.cuda.stream(s):
            got.append([layer_of_experts(x, *weights, 4)[0] for _ in range(5)])
    torch.cuda.synchronize()
    for a, many in zip(alone, got):
        assert all(torch.equal(a, y) for y in many)


@pytest.mark.parametrize("tokens", [2, 900])
def test_captured_and_replayed(tokens):
    """The run recorded into a graph and replayed on new inputs, with eager work between: each replay is the
    eager result, bit for bit, and so is a second graph's of the same operators."""
    t = torch.bfloat16
    weights = [gpu(w) for w in expert_weights(51, 8, 64, 48, t)]
    x = gpu(rnd(gen(1), tokens, 64, dtype=t))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer_of_experts(x, *weights, 2)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            y, _ = layer_of_experts(x, *weights, 2)
        graphs.append((g, y))
    for i in range(4):
        x.copy_(gpu(rnd(gen(100 + i), tokens, 64, dtype=t)))
        eager, _ = layer_of_experts(x, *weights, 2)
        torch.cuda.synchronize()
        for g, y in graphs:
            y.fill_(math.nan)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, eager), i


def test_same_call_same_bits():
    t = torch.float16
    weights = [gpu(w) for w in expert_weights(61, 8, 200, 136, t)]
    x = gpu(rnd(gen(1), 777, 200, dtype=t))
    first = layer_of_experts(x, *weights, 3)[0]
    assert all(torch.equal(first, layer_of_experts(x, *weights, 3)[0]) for _ in range(5))


def test_sizes_past_32_bits_are_refused():
    logits = torch.zeros(2, 8, device=device())
    for kw in (dict(groups=2 ** 32 + 1), dict(groups=2, topk_groups=2 ** 32 + 1), dict(group_top=2 ** 32 + 1), dict(groups=1 - 2 ** 32)):
        with pytest.raises((ValueError, B.MlpError)):
            ops.route(logits, 2, **kw)
    for k in (2 ** 32 + 2, 2 - 2 ** 32):
        with pytest.raises((ValueError, B.MlpError)):
            ops.route(logits, k)
    index = torch.zeros(2, 2, dtype=torch.int32, device=device())
    for experts in (2 ** 32 + 2, 2 - 2 ** 32, 0, 1025):
        with pytest.raises((ValueError, B.MlpError)):
            ops.dispatch(index, experts)


def test_experts_and_logits_far_apart():
    """Experts' matrices, rows of x and rows of logits whose offsets pass 2^31 elements."""
    far = (1 << 30) + 17
    base = torch.zeros(3 * far, dtype=torch.bfloat16, device=device())
    w = base.as_strided((3, 24, 40), (far, 40, 1))
    w.copy_(torch.randn(3, 24, 40, generator=gen(70)))
    x = base.as_strided((3, 40), (far, 1), 4096)
    x.copy_(torch.randn(3, 40, generator=gen(71)))
    logits = base.as_strided((3, 7), (far, 1), 8192)
    logits.copy_(torch.randn(3, 7, generator=gen(72)))
    near_x, near_w, near_logits = x.contiguous(), w.contiguous(), logits.contiguous()
    index = torch.tensor([[2, 0], [1, 2], [0, 1]], dtype=torch.int32, device=device())
    plan = ops.dispatch(index, 3)
    for combine in (False, True):
        assert torch.equal(ops.expert_linear(x, w, plan, k=2, combine=combine), ops.expert_linear(near_x, near_w, plan, k=2, combine=combine))
    got, want = ops.route(logits, 3), ops.route(near_logits, 3)
    assert torch.equal(got.index, want.index) and torch.equal(got.weight, want.weight)
