"""Plain forms of the single operators in 64 bits, on the CPU, and the tolerances of their tests."""
from __future__ import annotations

import math

import torch

SLOPE = float(torch.tensor(0.01, dtype=torch.float16))


def act64(v, name):
    return {"none": lambda: v, "leaky_relu": lambda: torch.where(v < 0, v * SLOPE, v),
            "relu": lambda: torch.where(v < 0, torch.zeros_like(v), v),
            "gelu": lambda: v * 0.5 * (1 + torch.erf(v / math.sqrt(2))),
            "silu": lambda: v / (1 + torch.exp(-v))}[name]()


def layer64(x, w, bias, act, gated):
    """(f(x), bound): the layer in 64 bits and how far an FP32 evaluation of it may be off, before the rounding.

    The FP32 sum of k products and a bias, in any order, is off by at most (k + 1) * 2^-24 * S with
    S = sum |x w| + |b| (each of its k additions rounds a partial sum of at most S; a product of two 11- or
    8-bit significands is exact).  A factor 2 covers the matrix unit's own partial sums.  The activations have a
    slope of at most 1.13 (GELU), and their own FP32 evaluation is off by at most 16 steps of 2^-24 of
    |value| (exp, erf, a division and products); GELU's 1 + erf can cancel, which leaves 2^-22 of |v|."""
    x, w = x.double(), w.double()
    z = x @ w.t()
    s = x.abs() @ w.abs().t()
    if bias is not None:
        z, s = z + bias.double(), s + bias.double().abs()
    err = 2 * (x.shape[1] + 1) * 2.0 ** -24 * s

    def through(v, e):
        y = act64(v, act)
        return y, 1.13 * e + 2.0 ** -20 * y.abs() + (2.0 ** -22 * v.abs() if act == "gelu" else 0)

    if not gated:
        return through(z, err)
    n = z.shape[1] // 2
    y, e = through(z[:, :n], err[:, :n])
    u, eu = z[:, n:], err[:, n:]
    return y * u, e * u.abs() + y.abs() * eu + e * eu + 2.0 ** -24 * (y * u).abs()


def rounded(y, bound, dtype):
    """The bound after rounding to dtype: half a step of the value, or of the smallest subnormal."""
    info = torch.finfo(dtype)
    return bound + (y.abs() + bound) * (info.eps / 2) + info.smallest_normal * info.eps / 2


def check(got, want, bound, dtype, what=""):
    """got (of dtype) within the bound of want (64 bits) everywhere; both finite."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), "%s: non-finite output" % what
    lim = rounded(want, bound, dtype)
    bad = (got - want).abs() > lim
    assert not bad.any(), "%s: %d values off, worst %.3g times the bound" % (
        what, int(bad.sum()), float(((got - want).abs() / lim).max()))


def linear64(x, w, bias=None, residual=None, act="none", gated=False):
    y, e = layer64(x.cpu(), w.cpu(), None if bias is None else bias.cpu(), act, gated)
    if residual is not None:
        r = residual.cpu().double()
        y, e = y + r, e + 2.0 ** -24 * (y.abs() + r.abs())
    return y, e


def route64(logits, k, score="softmax", bias=None, groups=1, topk_groups=None, group_top=1, renormalise=False,
            scale=1.0):
    """(index, weight) by a loop over tokens; ties to the lower index."""
    tokens, experts = logits.shape
    topk_groups = groups if topk_groups is None else topk_groups
    index = torch.full((tokens, k), -1, dtype=torch.int32)
    weight = torch.zeros(tokens, k, dtype=torch.float64)
    x = logits.detach().cpu().double()
    b = [0.0] * experts if bias is None else bias.cpu().double().tolist()
    for t in range(tokens):
        row = x[t].tolist()
        seen = [e for e in range(experts) if row[e] > -math.inf]  # neither NaN nor -inf
        if score == "softmax":
            top = max((row[e] for e in seen), default=0.0)
            ex = {e: 1.0 if row[e] == top else (0.0 if top == math.inf else math.exp(row[e] - top)) for e in seen}
            s = {e: v / math.fsum(ex.values()) for e, v in ex.items()}
        else:
            s = {e: 1 / (1 + math.exp(-row[e])) if row[e] > -700 else 0.0 for e in seen}
        choice = {e: s[e] + b[e] for e in seen if s[e] + b[e] > -math.inf}
        if topk_groups < groups:
            per, value = experts // groups, {}
            for g in range(groups):
                best = sorted((choice[e] for e in range(g * per, (g + 1) * per) if e in choice), reverse=True)
                if best:
                    value[g] = sum(best[:group_top])
            kept = sorted(value, key=lambda g: (-value[g], g))[:topk_groups]
            choice = {e: c for e, c in choice.items() if e // per in kept}
        picks = sorted(choice, key=lambda e: (-choice[e], e))[:k]
        total = math.fsum(s[e] for e in picks)
        for j, e in enumerate(picks):
            w = s[e]
            if renormalise:
                w = w / total if total > 0 else 0.0
            index[t, j], weight[t, j] = e, w * scale
    return index, weight


def dispatch64(index, experts):
    flat = index.cpu().reshape(-1).tolist()
    by = [[] for _ in range(experts)]
    for a, e in enumerate(flat):
        if 0 <= e < experts:
            by[e].append(a)
    offsets, slots, places = [0], [], [-1] * len(flat)
    for rows in by:
        for a in rows:
            places[a] = len(slots)
            slots.append(a)
        offsets.append(len(slots))
    slots += [-1] * (len(flat) - len(slots))
    t = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return t(offsets), t(slots), t(places)


def experts64(x, w, plan, k, bias=None, act="none", gated=False, rows="tokens", combine=False, weight=None,
              residual=None):
    """(y, bound, written): by slot (rows not written are 0 there) or by token."""
    offsets, slots, places = (p.cpu() for p in plan)
    x, w = x.cpu(), w.cpu()
    total, experts = slots.numel(), w.shape[0]
    n = w.shape[1] // 2 if gated else w.shape[1]
    y = torch.zeros(total, n, dtype=torch.float64)
    e = torch.zeros_like(y)
    for ex in range(experts):
        lo, hi = int(offsets[ex]), int(offsets[ex + 1])
        if lo < hi:
            at = slots[lo:hi].long() // k if rows == "tokens" else slice(lo, hi)
            y[lo:hi], e[lo:hi] = layer64(x[at], w[ex], None if bias is None else bias[ex].cpu(), act, gated)
    if not combine:
        return y, e, int(offsets[-1])
    tokens = total // k
    out, err, size = (torch.zeros(tokens, n, dtype=torch.float64) for _ in range(3))
    for j in range(k):
        p = places.view(tokens, k)[:, j].long()
        on = (p >= 0).double()[:, None]
        f = torch.ones(tokens, 1, dtype=torch.float64) if weight is None else weight.cpu()[:, j:j + 1].double()
        part, pe = y[p.clamp(min=0)] * f * on, e[p.clamp(min=0)] * f.abs() * on
        out, err, size = out + part, err + pe, size + part.abs()
    if residual is not None:
        r = residual.cpu().double()
        out, size = out + r, size + r.abs()
    return out, err + (k + 2) * 2.0 ** -24 * size, tokens
