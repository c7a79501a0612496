"""GPU tests of the router's choices where they are hard: keys that lie close together, equal ones at the last place,
saturated scores, values of groups whose parts cancel or overflow, rows beside others.  The plain form is
ops_reference.route64; where the logits alone give the order (no bias, and no group valued by two experts) it is
given their ranks, since 64-bit scores of different logits can be equal (sigmoid(40) and sigmoid(50)).

Sizes by layout of the experts over a wave: up to 64, 128 and 256 experts with k < 16 share it among four tokens,
up to 512 take a wave, and more than that another kernel; 8, 300 and 500 fill theirs in part."""
import math

import pytest
import torch

import ops_reference as R
from gpu_util import device, log
from mlp_neural_shading_amd import ops

pytestmark = pytest.mark.gpu

LAYOUTS = [8, 64, 128, 256, 300, 500, 512, 900]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def want(logits, k, score="softmax", bias=None, groups=1, topk_groups=None, group_top=1, renormalise=False):
    kw = dict(score=score, groups=groups, topk_groups=topk_groups, group_top=group_top)
    if bias is not None or (group_top == 2 and (topk_groups or groups) < groups):
        return R.route64(logits, k, bias=bias, renormalise=renormalise, **kw)
    x = logits.double()
    ranks = x.clone()
    for t in range(len(x)):
        if score == "softmax" and bool((x[t] == math.inf).any()):
            continue  # the others' scores are exactly 0
        seen = x[t] > -math.inf
        ranks[t, seen] = torch.unique(x[t, seen], return_inverse=True)[1].double() / 64 - 8
    index, _ = R.route64(ranks, k, **kw)
    weight = torch.zeros(len(x), k, dtype=torch.float64)
    for t in range(len(x)):
        seen = x[t] > -math.inf
        on = index[t] >= 0
        if not bool(on.any()):
            continue
        top = x[t, seen].max()
        if score == "softmax":
            s = torch.where(x[t] == top, torch.ones_like(x[t]), torch.exp(x[t] - top))
            s = torch.where(seen, s, torch.zeros_like(s))
            s = s / s.sum()
        else:
            s = torch.sigmoid(x[t])
        w = s[index[t, on].long()]
        if renormalise:
            w = w / w.sum() if float(w.sum()) > 0 else torch.zeros_like(w)
        weight[t, on] = w
    return index, weight


def check(logits, k, **kw):
    index, weight = want(logits, k, **kw)
    bias = kw.pop("bias", None)
    got = ops.route(logits.to(device()), k, bias=None if bias is None else bias.to(device()), **kw)
    bad = (got.index.cpu() != index).any(1).nonzero().flatten().tolist()
    assert not bad, (logits.shape, k, kw, bad[:3], got.index[bad[0]].tolist(), index[bad[0]].tolist())
    # 8 half-steps of FP32, as everywhere for the weights
    assert bool(((got.weight.cpu().double() - weight).abs() <= 8 * 2.0 ** -24 * weight.abs() + 2.0 ** -149).all())


def counts(experts):
    return [k for k in ((1, 2, 4, 8, 15, 20, 32) if experts < 500 else (1, 8, 32)) if k <= experts]


@pytest.mark.parametrize("experts", LAYOUTS)
def test_equals_at_the_last_place(experts):
    """The k-th and the next are equal, and behind them stands one that FP32 keys, or their places, do not tell from them,
    and that is the better one."""
    log("equals at the last place", experts)
    zero = torch.zeros(experts)
    for k in counts(experts):
        run = min(k + 1, experts - 2)
        for better in (1, 2):
            up = torch.zeros(3, experts)
            up[:, :run] = 17.0
            up[0, run:run + better], up[1, experts - better:], up[2, 0] = 17.125, 17.125, 17.25
            check(up, k, score="sigmoid", bias=zero)
            check(up, k, score="sigmoid", bias=zero + 0.25, renormalise=True)
            near = torch.full((2, experts), -60.0)
            near[:, :run] = 1.0
            near[0, run:run + better], near[1, experts - better:] = 1 + 2.0 ** -22, 1 + 2.0 ** -22
            for score in ops.SCORES:
                check(near, k, score=score)
            check(near, k, score="softmax", bias=zero)
            check(near, k, score="softmax", bias=zero + 16.0)


@pytest.mark.parametrize("experts", [8, 64, 256, 300, 900])
def test_a_row_is_the_same_beside_any_others(experts):
    """Alone, in any place and beside rows that need a closer look: the same bits.  Among them logits whose 64-bit scores
    are equal, though they are not."""
    g = gen(experts)
    log("beside others", experts)
    rows = torch.randn(14, experts, generator=g)
    rows[0, :2] = torch.tensor([40., 50.])
    rows[1] = 36 + torch.arange(experts) % 7
    rows[2] = -600 - 10.0 * (torch.arange(experts) % 9)
    rows[2, 3] = 0
    rows[3, :3] = torch.tensor([17., 17., 17.125])
    rows[4] = 14 + 4 * torch.rand(experts, generator=g)
    rows[5] = torch.randint(-2, 3, (experts,), generator=g).float()
    rows[6, 4] = math.inf
    rows[7] = 1.0
    rows[7, 5] = 1 + 2.0 ** -23
    rows[8] = -math.inf
    rows[9, 1:] = math.nan
    groups = 4 if experts % 4 == 0 else 1
    for k in (1, 4, 8) if experts < 500 else (4,):
        for kw in (dict(), dict(renormalise=True), dict(bias=torch.zeros(experts)), dict(bias=torch.full((experts,), 0.25)),
                   dict(groups=groups, topk_groups=max(1, groups // 2)), dict(groups=groups, topk_groups=max(1, groups // 2), group_top=2)):
            for score in ops.SCORES:
                if kw.get("topk_groups", 1) * experts // kw.get("groups", 1) < k:
                    continue
                check(rows, k, score=score, **kw)
                on_gpu = {**kw, "bias": kw["bias"].to(device())} if "bias" in kw else kw
                x = rows.to(device())
                whole = ops.route(x, k, score=score, **on_gpu)
                order = torch.randperm(14, generator=g).to(device())
                mixed = ops.route(x[order], k, score=score, **on_gpu)
                assert torch.equal(mixed.index, whole.index[order]) and torch.equal(mixed.weight, whole.weight[order])
                for t in range(12):
                    alone = ops.route(x[t:t + 1], k, score=score, **on_gpu)
                    assert torch.equal(alone.index[0], whole.index[t]) and torch.equal(alone.weight[0], whole.weight[t])


@pytest.mark.parametrize("experts", LAYOUTS)
def test_keys_that_hardly_differ(experts):
    """A token whose keys span less than 1e-32, but are not all equal."""
    g = gen(experts)
    log("tiny spans", experts)
    one = torch.zeros(6, experts)
    for t, v in enumerate((1e-33, 1e-35, 1e-38, 1e-42, -1e-35, 1.5e-45)):
        one[t, 2 + t % 2] = v
    few = torch.randint(-3, 4, (6, experts), generator=g).float() * 2.0 ** -140
    low = -75 - 4.5 * torch.rand(6, experts, generator=g)
    low[0], low[1] = torch.linspace(-78, -79.5, experts), torch.linspace(-79.5, -78, experts)
    low[2, :8] = torch.tensor([-75., -80., -76., -82., -85., -79., -81., -78.])
    for k in counts(experts):
        for score in ops.SCORES:
            check(one, k, score=score)
            check(few, k, score=score)
        check(low, k, score="sigmoid", bias=torch.zeros(experts))
        check(low, k, score="sigmoid")
        check(low * 3, k, score="softmax", bias=torch.full((experts,), 2.0 ** -120), renormalise=True)


@pytest.mark.parametrize("experts,groups", [(16, 8), (64, 8), (128, 4), (256, 8), (320, 8), (512, 16), (640, 8)])
def test_values_of_groups_past_fp32(experts, groups):
    """Biases of FP32's lowest value: the sum of two is no FP32 number, and their groups are still there."""
    log("groups past fp32", experts, groups)
    per, lowest = experts // groups, torch.finfo(torch.float32).min
    logits = torch.randn(9, experts, generator=gen(experts))
    bias = torch.full((experts,), lowest)
    bias[2 * per:3 * per] = 0.1
    for k in (2, min(per + 2, 12)):
        for score in ops.SCORES:
            check(logits, k, score=score, bias=bias, groups=groups, topk_groups=3, group_top=2)
            check(logits, k, score=score, bias=-bias, groups=groups, topk_groups=3, group_top=2)
            check(logits, k, score=score, bias=bias, groups=groups, topk_groups=groups - 1, group_top=2)


@pytest.mark.parametrize("experts,groups", [(16, 8), (32, 16), (512, 4), (8, 4)])
def test_values_of_groups_whose_parts_cancel(experts, groups):
    """A large and a large negative bias in each group: the keys are rounded by steps of theirs, the values are small."""
    log("groups that cancel", experts, groups)
    per = experts // groups
    for size in (30.0, 1000.0, 20000.0):
        g = gen(int(size))
        bias = torch.full((experts,), -2 * size)
        bias[::per], bias[1::per] = size, -size
        logits = torch.randn(1000 if per == 2 else 40, experts, generator=g)
        for score in ops.SCORES:
            for topk_groups in (1, groups // 2):
                check(logits, 2, score=score, bias=bias, groups=groups, topk_groups=topk_groups, group_top=2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("experts", LAYOUTS)
def test_drawn_from_few_values(experts, dtype):
    """Rows of few different logits, equal and one step apart, around -80, 0, 17 and 40."""
    g = gen(experts + 1)
    log("few values", experts, dtype)
    near = torch.tensor([0, 1, 2, 3]) * torch.finfo(dtype).eps
    rows = []
    for middle in (-80.0, 0.5, 17.0, 40.0):
        for spread in (1.0, 2000.0):
            values = torch.cat([middle * (1 + near), middle + spread * torch.finfo(dtype).eps * torch.tensor([0., 1., 2., 16.])])
            rows.append(values[torch.randint(0, 8, (2, experts), generator=g)])
            rows[-1][1, : experts // 2] = 0.0
    logits = torch.cat(rows).to(dtype)
    for k in counts(experts):
        for score in ops.SCORES:
            check(logits, k, score=score)
            check(logits, k, score=score, renormalise=True)
            check(logits, k, score=score, bias=torch.zeros(experts))
        check(logits, k, score="sigmoid", bias=torch.full((experts,), 0.25))
        check(logits, k, score="sigmoid", bias=(torch.arange(experts) % 3) * 0.5, renormalise=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("experts", [8, 64, 128, 256, 300, 512, 900])
def test_softmax_weights_are_rounded_once(experts, dtype):
    """Weights of the softmax over all experts: exponentials and their sum to 2^-30 of themselves, their quotient in 64
    bits, and one rounding to FP32 of at most 2^-24 of the value."""
    g = gen(experts + 2)
    logits = (torch.randn(500, experts, generator=g) * 2).to(dtype)
    logits[0], logits[1, 3] = 0.125, 60.0
    x = logits.double()
    score = torch.exp(x - x.max(1, keepdim=True).values)
    score = score / score.sum(1, keepdim=True)
    for bias in (None, torch.randn(experts, generator=g).to(device()) * 0.1):
        got = ops.route(logits.to(device()), min(experts, 10), bias=bias, scale=1.0)
        w = torch.gather(score, 1, got.index.cpu().long())
        off = ((got.weight.cpu().double() - w).abs() / w).max()
        assert float(off) <= 2.0 ** -24 + 2.0 ** -28, float(off) * 2 ** 24
