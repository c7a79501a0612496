"""Plain forms of the 8-bit operators in 64 bits, on the CPU, and the tolerances of their tests.

u = 2^-24 is half a step of FP32 relative to a value."""
from __future__ import annotations

import torch

import ops_reference as R

FP8 = torch.float8_e4m3fn
BLOCK = 128
U = 2.0 ** -24


def blocks(n):
    return -(-n // BLOCK)


def spread(scales, rows, width, block_rows=1):
    """Each element's scale."""
    s = scales.repeat_interleave(BLOCK, -1)[..., :width]
    return s.repeat_interleave(block_rows, -2)[..., :rows, :] if block_rows > 1 else s


def by_block(x, block_rows=1):
    """The largest magnitude of each block of a matrix, over its finite elements."""
    rows, width = x.shape
    a = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
    out = a.new_zeros(-(-rows // block_rows), blocks(width))
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            out[i, j] = a[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK].max()
    return out


def quantize(x, block_rows=1):
    """(values, scales) of a matrix as the header defines them, in FP32 operations: every bit is determined."""
    x = x.float()
    scales = torch.maximum(by_block(x, block_rows) / 448, torch.tensor(2.0 ** -126))
    v = x * (1 / spread(scales, *x.shape, block_rows))
    v = torch.where(torch.isfinite(x), v, torch.full_like(v, float("nan")))
    return v.to(FP8), scales


def quantize_weights(w, gated=False):
    """The same for the weights of a layer, or of each expert: blocks of 128 rows, of each half if gated."""
    if w.dim() == 3:
        parts = [quantize_weights(e, gated) for e in w]
        return torch.stack([p[0].view(torch.uint8) for p in parts]).view(FP8), torch.stack([p[1] for p in parts])
    halves = [quantize(h, BLOCK) for h in w.chunk(2 if gated else 1)]
    return torch.cat([h[0].view(torch.uint8) for h in halves]).view(FP8), torch.cat([h[1] for h in halves])


def dequantize(values, scales, block_rows=1):
    return values.cpu().double() * spread(scales.cpu().double(), *values.shape[-2:], block_rows)


def check_quantized(got, y, e, what=""):
    """8-bit rows of values that lie within e of y (64 bits).  The scale is the largest magnitude, which is off by at
    most the block's largest e, by 448 with one rounding.  A value is y / scale, off by e / scale and by two roundings
    (the reciprocal and the product), rounded once to E4M3: half a step, of 2^-3 in a binade and of 2^-9 below 2^-6."""
    values, scales = (t.cpu().double() for t in got)
    assert values.shape == y.shape and scales.shape == (y.shape[0], blocks(y.shape[1])), what
    assert torch.isfinite(values).all() and torch.isfinite(scales).all(), what
    e = torch.as_tensor(e, dtype=torch.float64).expand_as(y)
    want = torch.clamp(by_block(y) / 448, min=2.0 ** -126)
    bad = (scales - want).abs() > by_block(e) / 448 + 2 * U * want
    assert not bad.any(), "%s: %d scales off" % (what, int(bad.sum()))
    s = spread(scales, *y.shape)
    v = y / s
    off = e / s + 4 * U * v.abs()
    step = torch.exp2(torch.floor(torch.log2((v.abs() + off).clamp(min=2.0 ** -6))) - 3)
    bad = (values - v).abs() > step / 2 + off
    assert not bad.any(), "%s: %d values off, worst by %.3g steps" % (what, int(bad.sum()), float(((values - v).abs() / step).max()))


def norm64(x, weight=None, residual=None, eps=1e-6):
    """(y, bound, total): three FP32 roundings (the row's factor, and two products), and the factor's own in 64 bits."""
    total = x.cpu()
    if residual is not None:
        total = (total.float() + residual.cpu().float()).to(x.dtype)
    t = total.double()
    y = t / torch.sqrt((t * t).mean(1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.cpu().double()
    return y, 4 * U * y.abs(), total


def cut(x, w, k):
    """How far the matrix unit's sums of E4M3 products are off (rows of x against rows of w, dequantized): it adds 8 products
    of neighbouring columns after cutting each to a multiple of 2^-13 times 2^e, e the largest sum of two exponents among the
    8.  The largest product is at least 2^e and is not cut (products are multiples of 2^-6 of their 2^e), so the other 7 lose
    less than 7 * 2^-13 of the product of the groups' largest elements.  A last block of less than 128 columns may be grouped in
    any way, into at most 17: each by the largest elements of the whole of it."""
    full = k // BLOCK * BLOCK
    groups = [t[:, :full].abs().unflatten(1, (-1, 8)).amax(2) if full else t[:, :0] for t in (x, w)]
    bound = groups[0] @ groups[1].t()
    if k > full:
        bound = bound + 17 * x[:, full:].abs().amax(1)[:, None] * w[:, full:].abs().amax(1)[None]
    return 7 * 2.0 ** -13 * bound


def layer64(x, xs, w, ws, bias, act, gated, full):
    """(f(x), bound) of a layer with 8-bit operands, before its rounding; full: the sums that FP32 and 8-bit outputs get.

    Products of two 4-bit significands are exact.  The FP32 sum of a block of up to 128, in any order, is off by at most
    128 u of the sum of magnitudes; the product of the two scales, the multiply-add of each block and the bias each round
    once more: (128 + blocks + 3) u of S = sum |x w| xs ws + |b|, and a factor 2 covers the matrix unit's own partial
    sums.  Not full: what `cut` says besides.  The activations as in ops_reference."""
    k, n = x.shape[1], w.shape[0] // (2 if gated else 1)
    xd = dequantize(x, xs)
    halves = [dequantize(w[h * n:(h + 1) * n], ws[h * blocks(n):(h + 1) * blocks(n)], BLOCK) for h in range(2 if gated else 1)]
    wd = torch.cat(halves)
    z, s = xd @ wd.t(), xd.abs() @ wd.abs().t()
    if bias is not None:
        z, s = z + bias.cpu().double(), s + bias.cpu().double().abs()
    err = 2 * (min(k, BLOCK) + blocks(k) + 3) * U * s + (0 if full else cut(xd, wd, k))

    def through(v, e):
        y = R.act64(v, act)
        return y, 1.13 * e + 2.0 ** -20 * y.abs() + (2.0 ** -22 * v.abs() if act == "gelu" else 0)

    if not gated:
        return through(z, err)
    y, e = through(z[:, :n], err[:, :n])
    u, eu = z[:, n:], err[:, n:]
    return y * u, e * u.abs() + y.abs() * eu + e * eu + U * (y * u).abs()


def linear64(x, w, bias=None, residual=None, act="none", gated=False, full=False):
    y, e = layer64(x[0].cpu(), x[1].cpu(), w[0].cpu(), w[1].cpu(), bias, act, gated, full)
    if residual is not None:
        r = residual.cpu().double()
        y, e = y + r, e + U * (y.abs() + r.abs())
    return y, e


def experts64(x, w, plan, k, bias=None, act="none", gated=False, rows="tokens", combine=False, weight=None, residual=None,
              full=False):
    """(y, bound, written): by slot (rows not written are 0 there) or by token, as ops_reference.experts64."""
    offsets, slots, places = (p.cpu() for p in plan)
    xv, xs, wv, ws = (t.cpu() for t in (*x, *w))
    total, experts = slots.numel(), wv.shape[0]
    n = wv.shape[1] // 2 if gated else wv.shape[1]
    y = torch.zeros(total, n, dtype=torch.float64)
    e = torch.zeros_like(y)
    for ex in range(experts):
        lo, hi = int(offsets[ex]), int(offsets[ex + 1])
        if lo < hi:
            at = slots[lo:hi].long() // k if rows == "tokens" else torch.arange(lo, hi)
            rows_x = xv.view(torch.uint8)[at].view(FP8)
            y[lo:hi], e[lo:hi] = layer64(rows_x, xs[at], wv[ex], ws[ex], None if bias is None else bias[ex].cpu(), act, gated, full)
    if not combine:
        return y, e, int(offsets[-1])
    tokens = total // k
    # terms on their way to a 16-bit sum: half a step of 1 / 32,766 of the largest of 32 neighbours (off by e itself), and
    # the roundings of the scale, its reciprocal and two products (4 u of up to 32,766 steps: 2^-7 of a step)
    high = torch.nn.functional.pad(y.abs() + e, (0, -n % 32)).unflatten(1, (-1, 32)).amax(2)
    term = 0 if full else 0.51 * 2.0 ** -15 * high.repeat_interleave(32, 1)[:, :n]
    out, err, size = (torch.zeros(tokens, n, dtype=torch.float64) for _ in range(3))
    for j in range(k):
        p = places.view(tokens, k)[:, j].long()
        on = (p >= 0).double()[:, None]
        f = torch.ones(tokens, 1, dtype=torch.float64) if weight is None else weight.cpu()[:, j:j + 1].double()
        part, pe = y[p.clamp(min=0)] * f * on, (e + term)[p.clamp(min=0)] * f.abs() * on
        out, err, size = out + part, err + pe, size + part.abs()
    if residual is not None:
        r = residual.cpu().double()
        out, size = out + r, size + r.abs()
    return out, err + (k + 2) * U * size, tokens
