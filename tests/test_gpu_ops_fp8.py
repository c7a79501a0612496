"""GPU tests of the 8-bit operators (include/mlp_ops_fp8.h) against their plain forms in 64 bits, at the sizes and
inputs where they can go wrong.  The tolerances are those of ops_fp8_reference; the rounding to 8 bits itself is
compared bit for bit."""
import math

import pytest
import torch

import ops_fp8_kernels as K
import ops_fp8_reference as F
import ops_reference as R
from gpu_util import device, log
from mlp_neural_shading_amd import binding as B
from mlp_neural_shading_amd import ops
from mlp_neural_shading_amd import ops_fp8 as E

pytestmark = pytest.mark.gpu

FLOATS = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
FP8 = torch.float8_e4m3fn


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rnd(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def gpu(t):
    return None if t is None else t.to(device())


def put(q):
    return E.Quantized(*map(gpu, q))


def bits(t):
    return t.cpu().contiguous().view(torch.uint8)


def same(got, want):
    """8-bit values and scales, bit for bit; a NaN is a NaN."""
    v, w = got.values.cpu().float(), want[0].cpu().float()
    assert torch.equal(v.isnan(), w.isnan()) and torch.equal(v.nan_to_num(), w.nan_to_num())
    assert torch.equal(got.scales.cpu(), want[1])


def block(t, left, right, fill):
    """t as a column block of a wider matrix, whose other columns hold `fill`."""
    one = t.element_size() == 1
    raw = t.view(torch.uint8) if one else t
    wide = torch.full((*t.shape[:-1], left + t.shape[-1] + right), fill, dtype=raw.dtype, device=t.device)
    wide[..., left:left + t.shape[-1]] = raw
    wide = wide.view(t.dtype) if one else wide
    return wide, wide[..., left:left + t.shape[-1]]


NAN8 = 0x7F


# ---- quantize ------------------------------------------------------------------------------------

SIZES = [(1, 1), (1, 127), (1, 128), (1, 129), (3, 7), (5, 1000), (17, 256), (130, 300), (128, 128), (129, 1001), (300, 2048),
         (1000, 72), (2, 40000)]


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("rows,width", SIZES)
def test_quantize(rows, width, dtype):
    g = gen(rows + width)
    x = (rnd(g, rows, width) * torch.exp(rnd(g, width))).to(FLOATS[dtype])
    log("quantize", rows, width, dtype)
    for block_rows in (1, 128):
        same(E.quantize(gpu(x), block_rows=block_rows), F.quantize(x, block_rows))
        for left, right in ((8, 8), (1, 2)):
            _, xv = block(gpu(x), left, right, math.nan)
            same(E.quantize(xv, block_rows=block_rows), F.quantize(x, block_rows))


@pytest.mark.parametrize("dtype", FLOATS)
def test_quantize_every_size_of_number(dtype):
    """Blocks of zeros, of subnormals, of the largest numbers, of NaN and infinities among others, and of them alone."""
    t = FLOATS[dtype]
    info = torch.finfo(t)
    x = rnd(gen(1), 260, 300).to(t)
    x[0] = 0
    x[1] = -0.0
    x[2] = info.tiny * info.eps  # the smallest
    x[3] = x[3] * info.tiny
    x[4] = info.max
    x[5] = torch.where(x[5] > 0, x[5] * 0 + info.max, x[5] * info.tiny)
    x[6, ::7] = math.nan
    x[7, ::5] = math.inf
    x[8, 3::5] = -math.inf
    x[9] = math.nan
    x[10, 130:] = math.inf
    for block_rows in (1, 128):
        same(E.quantize(gpu(x), block_rows=block_rows), F.quantize(x, block_rows))


def test_quantize_rounds_to_even():
    """Every step's middle, from both sides: 448 makes the scale 1, so the values are the numbers."""
    codes = torch.arange(127, dtype=torch.uint8).view(FP8).float()  # 0 .. 448
    middle = (codes[1:] + codes[:-1]) / 2
    x = torch.cat([codes, middle, torch.nextafter(middle, middle + 1), torch.nextafter(middle, middle - 1)])
    x = torch.cat([x, -x])
    rows = torch.zeros(9, 128)
    rows[:, 0] = 448
    rows[:, 1:].flatten()[:x.numel()] = x  # a copy
    flat = rows[:, 1:].reshape(-1).clone()
    flat[:x.numel()] = x
    rows[:, 1:] = flat.view(9, 127)
    same(E.quantize(gpu(rows)), (rows.to(FP8), torch.ones(9, 1)))


@pytest.mark.parametrize("count,rows,width", [(1, 40, 130), (3, 128, 128), (5, 200, 77), (4, 260, 300)])
def test_quantize_several_matrices(count, rows, width):
    x = rnd(gen(rows), count, rows, width, dtype=torch.bfloat16)
    for gated in (False, True):
        got = E.quantize(gpu(x), block_rows=128, gated=gated)
        same(got, F.quantize_weights(x, gated))
        one = E.quantize(gpu(x[0]), block_rows=128, gated=gated)
        assert torch.equal(bits(one.values), bits(got.values[0])) and torch.equal(one.scales, got.scales[0])
        wide = torch.full((count, rows + 3, width + 5), math.nan, dtype=torch.bfloat16, device=device())
        wide[:, 2:-1, 1:-4] = gpu(x)
        same(E.quantize(wide[:, 2:-1, 1:-4], block_rows=128, gated=gated), F.quantize_weights(x, gated))
    rows1 = E.quantize(gpu(x))
    for i in range(count):
        same(E.Quantized(rows1.values[i], rows1.scales[i]), F.quantize(x[i]))


# ---- rms_norm ------------------------------------------------------------------------------------

NORMS = [(1, 1), (1, 7), (3, 128), (5, 129), (4, 1001), (2, 2048), (3, 2049), (2, 5000), (3, 8192), (2, 20000), (3, 32768),
         (2, 32769), (2, 70001), (1024, 130), (1500, 300), (1100, 1001), (1030, 1025), (1024, 2048), (4000, 72), (4001, 16)]


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("rows,width", NORMS)
def test_rms_norm(rows, width, dtype):
    g, t = gen(rows + width), FLOATS[dtype]
    x, r, w = rnd(g, rows, width, dtype=t), rnd(g, rows, width, dtype=t, scale=2.0), 1 + rnd(g, width, scale=0.3)
    w = w.to(t)
    log("norm", rows, width, dtype)
    for residual in (None, r):
        y, e, total = F.norm64(x, w, residual)
        got = E.rms_norm(gpu(x), gpu(w), residual=gpu(residual), out="both")
        R.check(got.y, y, e, t, "y")
        F.check_quantized(got.quantized, y, e, "quantized")
        assert (got.total is None) if residual is None else torch.equal(got.total.cpu(), total)
        only = E.rms_norm(gpu(x), gpu(w), residual=gpu(residual), out="fp8")
        assert only.y is None and torch.equal(bits(only.quantized.values), bits(got.quantized.values))
        assert torch.equal(only.quantized.scales, got.quantized.scales)
        wide = E.rms_norm(gpu(x), gpu(w), residual=gpu(residual), out_dtype=torch.float32)
        R.check(wide.y, y, e, torch.float32, "fp32")
        assert wide.quantized is None
    y, e, _ = F.norm64(x, None, None, eps=0.5)
    R.check(E.rms_norm(gpu(x), eps=0.5).y, y, e, t, "no weight")


@pytest.mark.parametrize("rows,width", [(3, 100), (5, 1001), (3, 3000), (4, 6000), (3, 9000), (2, 40000), (1100, 600)])
def test_rms_norm_in_place_and_beside(rows, width):
    """The total as x and as the residual; column blocks of wider matrices, aligned or not, NaN around the inputs."""
    g, t = gen(rows), torch.bfloat16
    x, r, w = rnd(g, rows, width, dtype=t), rnd(g, rows, width, dtype=t), rnd(g, width, dtype=t)
    want = E.rms_norm(gpu(x), gpu(w), residual=gpu(r), out="both")
    for left, right in ((0, 0), (8, 8), (1, 2)):
        for place in ("x", "residual", "beside"):
            whole_x, xv = block(gpu(x), left, right, math.nan)
            whole_r, rv = block(gpu(r), left, right, math.nan)
            whole_t, tv = block(torch.zeros_like(gpu(r)), left, right, 7.0)
            at = {"x": xv, "residual": rv, "beside": tv}[place]
            got = E.rms_norm(xv, gpu(w), residual=rv, total=at, out="both")
            assert got.total is at and torch.equal(at, want.total)
            assert torch.equal(got.y, want.y) and torch.equal(bits(got.quantized.values), bits(want.quantized.values))
            assert torch.equal(got.quantized.scales, want.quantized.scales)
            assert bool((whole_t[:, :left] == 7).all()) and bool((whole_t[:, left + width:] == 7).all())
            for whole in (whole_x, whole_r):
                assert bool(whole[:, :left].isnan().all()) and bool(whole[:, left + width:].isnan().all())


def test_rms_norm_rows_by_themselves():
    """A row of zeros, of numbers whose squares pass FP32 either way, and rows with a NaN or an infinity."""
    t = torch.bfloat16
    x = rnd(gen(3), 12, 260, dtype=t)
    x[1] = 0
    x[2] = (x[2].float() * 1e30).to(t)
    x[3] = (x[3].float() * 1e-30).to(t)
    x[4, 5] = math.nan
    x[5, 250] = math.inf
    got = E.rms_norm(gpu(x), out="both", eps=1e-37)
    fine = [i for i in range(12) if i not in (4, 5)]
    y, e, _ = F.norm64(x[fine], eps=1e-37)
    R.check(got.y[fine], y, e, t)
    F.check_quantized((bits(got.quantized.values)[fine].view(FP8), got.quantized.scales[fine]), y, e)
    assert bool(got.y[4].isnan().all()) and bool(got.quantized.values[4].float().isnan().all())
    assert bool(got.y[5, 250].isnan()) and bool((got.y[5, :250] == 0).all())
    assert bool(got.quantized.values[5, 250].float().isnan()) and bool((got.quantized.values[5, :250].float() == 0).all())


# ---- linear --------------------------------------------------------------------------------------

# (rows, in, out): single rows, odd sizes, tile borders and one past them, K below, at and past a block
LINEAR = [(1, 1, 1), (1, 1024, 64), (2, 7, 3), (3, 64, 65), (5, 8, 1000), (16, 100, 48), (17, 129, 33), (31, 200, 130),
          (64, 64, 64), (65, 63, 63), (100, 320, 96), (127, 65, 257), (128, 128, 128), (129, 256, 255), (256, 512, 256),
          (300, 1001, 77), (513, 72, 520), (9, 5000, 40), (40, 4096, 24)]


def operands(g, rows, k, n, gated=False, aligned=True):
    """x and w in 8 bits; aligned: rows at 16 bytes, as quantize lays them out."""
    x = F.quantize(rnd(g, rows, k) * torch.exp(rnd(g, k, scale=0.5)))
    w = F.quantize_weights(rnd(g, 2 * n if gated else n, k, scale=k ** -0.5), gated)
    if aligned:
        x, w = ((block(q[0], 0, -k % 16, NAN8)[1], q[1]) for q in (x, w))
    return x, w


def on_gpu(q):
    """With the strides that it has."""
    v = q[0]
    whole = v.view(torch.uint8) if v.is_contiguous() else v._base if v._base is not None else v
    return E.Quantized(move(v), gpu(q[1]))


def move(v):
    """An 8-bit tensor to the GPU with the strides that it has; what lies between the rows holds NaN."""
    store = torch.full((v.untyped_storage().nbytes(),), NAN8, dtype=torch.uint8)
    raw = store.as_strided(v.shape, v.stride(), v.storage_offset())
    raw.copy_(v.view(torch.uint8))
    return store.to(device()).view(FP8).as_strided(v.shape, v.stride(), v.storage_offset())


@pytest.mark.parametrize("rows,k,n", LINEAR)
def test_linear(rows, k, n):
    g = gen(rows * 7 + k)
    x, w = operands(g, rows, k, n)
    b, r = rnd(g, n), rnd(g, rows, n)
    X, W = on_gpu(x), on_gpu(w)
    log("linear", rows, k, n)
    R.check(E.linear(X, W), *F.linear64(x, w), torch.bfloat16, "plain")
    R.check(E.linear(X, W, out_dtype=torch.float32), *F.linear64(x, w, full=True), torch.float32, "fp32")
    for t in (torch.float16, torch.bfloat16, torch.float32):
        y = E.linear(X, W, gpu(b), residual=gpu(r.to(t)), act="leaky_relu", out_dtype=t)
        R.check(y, *F.linear64(x, w, b, r.to(t), "leaky_relu", full=t == torch.float32), t, "epilogue")
    F.check_quantized(E.linear(X, W, gpu(b), act="silu", out_dtype=FP8), *F.linear64(x, w, b, None, "silu", full=True), "fp8")


# sizes that take the larger tiles, whole and with borders in every direction; K below a block, of one, of whole ones
# and with a rest
LARGE = [(5000, 200, 1800, False), (5000, 40, 1801, False), (4864, 128, 2048, False), (2600, 264, 1700, True),
         (2500, 72, 1500, False), (2048, 640, 2048, False), (1300, 200, 1100, True), (600, 136, 700, False), (640, 384, 640, False),
         (300, 64, 650, True), (9000, 72, 64, False), (9001, 33, 50, False), (4000, 64, 32, True), (700, 101, 903, False),
         (513, 77, 455, True), (150, 1040, 1000, False), (20000, 64, 128, False), (5000, 202, 1800, False), (300, 2049, 1001, False),
         (2500, 130, 1500, True), (700, 102, 640, False), (700, 512, 1000, False), (2600, 513, 1700, True)]


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("rows,k,n,gated", LARGE)
def test_linear_large(rows, k, n, gated, aligned):
    g = gen(rows + k)
    wide = 2 * n if gated else n
    x, w = operands(g, rows, k, n, gated, aligned)
    b, r = rnd(g, wide), rnd(g, rows, n)
    X, W = on_gpu(x), on_gpu(w)
    log("linear large", rows, k, n, gated, aligned)
    t = torch.float16
    y = E.linear(X, W, gpu(b), residual=gpu(r.to(t)), act="silu", gated=gated, out_dtype=t)
    R.check(y, *F.linear64(x, w, b, r.to(t), "silu", gated), t, "epilogue")
    want = F.linear64(x, w, b, None, "none", gated, full=True)
    R.check(E.linear(X, W, gpu(b), gated=gated, out_dtype=torch.float32), *want, torch.float32, "fp32")
    F.check_quantized(E.linear(X, W, gpu(b), gated=gated, out_dtype=FP8), *want, "fp8")


def whole_numbers(g, rows, k, lo, hi, ld):
    """8-bit whole numbers in rows of stride ld, NaN behind them, and scales that are powers of two."""
    v = torch.full((rows, ld), NAN8, dtype=torch.uint8).view(FP8)
    v.view(torch.uint8)[:, :k] = torch.randint(lo, hi, (rows, k), generator=g).float().to(FP8).view(torch.uint8)
    return v[:, :k]


@pytest.mark.parametrize("rows,n", [(5000, 1800), (4000, 900), (2500, 640), (520, 640), (60, 900)])
@pytest.mark.parametrize("k", [64, 66, 68, 96, 126, 128, 130, 132, 188, 192, 254, 256, 260, 380, 384, 388, 65, 127, 129, 383, 34, 3, 15, 16, 17, 23, 24, 25, 31, 111])
def test_last_columns_count_once(rows, n, k):
    """Whole numbers with scales that are powers of two, whose sums are exact, for widths that end anywhere in a block; a
    row stride beyond the width holds NaN, and one row a NaN in the first column of its last 128."""
    g = gen(k)
    ld = (k + 6) // 4 * 4
    x, w = whole_numbers(g, rows, k, -3, 4, ld), whole_numbers(g, n, k, 1, 4, ld)
    xs = torch.exp2(torch.randint(-2, 3, (rows, F.blocks(k)), generator=g).float())
    ws = torch.exp2(torch.randint(-2, 3, (F.blocks(n), F.blocks(k)), generator=g).float())
    want = (F.dequantize(x, xs) @ F.dequantize(w, ws, 128).T).float()
    X, W = E.Quantized(move(x), gpu(xs)), E.Quantized(move(w), gpu(ws))
    assert torch.equal(E.linear(X, W, out_dtype=torch.float32).cpu(), want)
    assert torch.equal(E.linear(X, W, out_dtype=torch.float16).cpu(), want.half())  # no product of 8 is below 2^-13 of another
    X.values[rows - 2, max(k - 128, 0)] = math.nan
    got = E.linear(X, W, out_dtype=torch.float32).cpu()
    assert bool(got[rows - 2].isnan().all())
    want[rows - 2] = got[rows - 2] = 0
    assert torch.equal(got, want)


@pytest.mark.parametrize("act", ops.ACTIVATIONS)
@pytest.mark.parametrize("rows,k,n", [(1, 96, 40), (9, 130, 33), (70, 64, 96), (260, 136, 200), (700, 200, 520)])
def test_linear_activations_and_gates(rows, k, n, act):
    g, t = gen(rows + n), torch.bfloat16
    (x, w), b, r = operands(g, rows, k, n, True), rnd(g, 2 * n), rnd(g, rows, n, dtype=t)
    X, W = on_gpu(x), on_gpu(w)
    log("activation", act, rows, k, n)
    y = E.linear(X, W, gpu(b), residual=gpu(r), act=act, gated=True)
    R.check(y, *F.linear64(x, w, b, r, act, True), t, "gated")
    want = F.linear64(x, w, None, None, act, True, full=True)
    R.check(E.linear(X, W, act=act, gated=True, out_dtype=torch.float32), *want, torch.float32, "gated fp32")
    F.check_quantized(E.linear(X, W, act=act, gated=True, out_dtype=FP8), *want, "gated fp8")


@pytest.mark.parametrize("left,right", [(16, 16), (1, 2), (4, 8), (3, 0)])
@pytest.mark.parametrize("rows,k,n", [(1, 72, 24), (12, 64, 40), (90, 136, 72), (300, 264, 280), (2000, 300, 1030)])
def test_linear_strides(rows, k, n, left, right):
    """Column blocks of wider matrices, aligned or not, scales too; the columns around them hold NaN on the way in and
    their own values afterwards."""
    g, t = gen(rows + left), torch.float16
    (x, w), r = operands(g, rows, k, n, aligned=False), rnd(g, rows, n, dtype=t)
    xv, wv = (block(gpu(q[0]), left, right, NAN8)[1] for q in (x, w))
    xs, ws = (block(gpu(q[1]), left, right, math.nan)[1] for q in (x, w))
    _, rv = block(gpu(r), left, right, math.nan)
    whole, out = block(torch.zeros_like(gpu(r)), left, right, 7.0)
    log("strides", rows, k, n, left, right)
    X, W = E.Quantized(xv, xs), E.Quantized(wv, ws)
    assert E.linear(X, W, residual=rv, act="silu", out=out, out_dtype=t) is out
    R.check(out, *F.linear64(x, w, None, r, "silu"), t)
    assert bool((whole[:, :left] == 7).all()) and bool((whole[:, left + n:] == 7).all())
    whole, v = block(torch.zeros(rows, n, dtype=torch.uint8, device=device()).view(FP8), left, right, 0x11)
    whole_s, s = block(torch.zeros(rows, F.blocks(n), device=device()), left, right, 7.0)
    q = E.Quantized(v, s)
    assert E.linear(X, W, act="silu", out=q, out_dtype=FP8) is q
    F.check_quantized(q, *F.linear64(x, w, None, None, "silu", full=True))
    raw = whole.view(torch.uint8)
    assert bool((raw[:, :left] == 0x11).all()) and bool((raw[:, left + n:] == 0x11).all())
    assert bool((whole_s[:, :left] == 7).all()) and bool((whole_s[:, left + F.blocks(n):] == 7).all())


def test_scales_are_taken_as_they_are():
    """Scales of any sign and size, 0 and infinities among them, each in its own block."""
    g = gen(8)
    rows, k, n = 300, 400, 300
    x, w = operands(g, rows, k, n)
    xs, ws = x[1] * torch.exp(rnd(g, *x[1].shape, scale=4.0)), w[1] * torch.exp(rnd(g, *w[1].shape, scale=4.0))
    xs[::3], ws[:, 1] = -xs[::3], -ws[:, 1]
    xs[5], ws[2, 0] = 0, 0
    x, w = (x[0], xs), (w[0], ws)
    R.check(E.linear(on_gpu(x), on_gpu(w), out_dtype=torch.float32), *F.linear64(x, w, full=True), torch.float32)
    xs[7, 1] = math.nan
    got = E.linear(on_gpu((x[0], xs)), on_gpu(w), out_dtype=torch.float32)
    assert bool(got[7].isnan().all()) and int(got.isnan().sum()) == n


@pytest.mark.parametrize("rows,k,n,gated", [*K.LINEAR.values(), *K.GATED.values()])
def test_linear_by_kernel(rows, k, n, gated):
    """A size of every kernel's, into each type that it writes."""
    g = gen(rows + n)
    wide = 2 * n if gated else n
    x, w = operands(g, rows, k, n, gated, aligned=False)
    X, W, b = on_gpu(x), on_gpu(w), rnd(g, wide)
    for full in (False, True):
        want = F.linear64(x, w, b, None, "silu", gated, full)
        for t in (torch.float32, FP8) if full else (torch.float16, torch.bfloat16):
            log("linear", rows, k, n, gated, t, K.linear_kernel(rows, k, n, gated, E._OUT[t]))
            y = E.linear(X, W, gpu(b), act="silu", gated=gated, out_dtype=t)
            F.check_quantized(y, *want) if t == FP8 else R.check(y, *want, t)


ODD = ((3, math.inf), (40, math.nan), (41, -math.inf))  # outputs and their bias


def without_odd(t, fill=0):
    t = t.clone()
    for o, _ in ODD:
        t[:, o] = fill
    return t


def check_odd(y, sign=True):
    for o, v in ODD:
        assert bool(y[:, o].float().isnan().all() if math.isnan(v) or not sign else (y[:, o] == v).all()), o


@pytest.mark.parametrize("rows,k,n,gated", [s for s in K.LINEAR.values()] + [K.GATED["big"], K.GATED["small"]])
def test_infinities_and_nans_stay_by_themselves(rows, k, n, gated):
    """Outputs that are not finite, from the bias, in blocks with others: NaN in 8 bits, and the others as without them."""
    g = gen(rows + 5)
    x, w = operands(g, rows, k, n, gated, aligned=False)
    X, W = on_gpu(x), on_gpu(w)
    b = without_odd(rnd(g, 1, 2 * n if gated else n))[0]
    want, e = F.linear64(x, w, b, None, "none", gated)
    full, ef = F.linear64(x, w, b, None, "none", gated, True)
    for o, v in ODD:
        b[o] = v
        if gated:
            b[n + o] = 1e9  # positive, so that the product's sign is the gate's
    log("odd", rows, k, n, gated)
    for t in (torch.bfloat16, torch.float32):
        y = E.linear(X, W, gpu(b), gated=gated, out_dtype=t)
        check_odd(y)
        R.check(without_odd(y), without_odd(full if t == torch.float32 else want), without_odd(ef if t == torch.float32 else e), t)
    q = E.linear(X, W, gpu(b), gated=gated, out_dtype=FP8)
    check_odd(q.values, False)
    F.check_quantized((without_odd(bits(q.values)).view(FP8), q.scales), without_odd(full), without_odd(ef))


# ---- the experts' layers ---------------------------------------------------------------------------

EXPERTS = [(1, 1, 1, 8, 8), (1, 2, 3, 40, 24), (3, 4, 9, 33, 17), (8, 4, 32, 128, 96), (64, 2, 4, 64, 64), (37, 3, 5, 200, 130),
           (300, 1, 16, 64, 64), (500, 2, 3, 160, 264), (260, 6, 70, 72, 40), (20, 2, 200, 16, 16), (3000, 2, 4, 72, 1200),
           (900, 2, 5, 136, 700), (4000, 1, 16, 64, 64), (1000, 3, 20, 40, 264), (700, 2, 6, 33, 300), (2000, 2, 4, 300, 700)]


def expert_weights(g, experts, wide, k, gated):
    v, s = F.quantize_weights(rnd(g, experts, wide, k, scale=k ** -0.5), gated)
    return block(v, 0, -k % 16, NAN8)[1], s


@pytest.mark.parametrize("tokens,k,experts,k_in,n", EXPERTS)
def test_expert_linear(tokens, k, experts, k_in, n):
    g, t = gen(tokens + experts), torch.bfloat16
    index = torch.randint(-1, experts, (tokens, k), generator=g, dtype=torch.int32)
    plan = R.dispatch64(index, experts)
    P = ops.Dispatch(*map(gpu, plan))
    weight, r = torch.rand(tokens, k, generator=g), rnd(g, tokens, n, dtype=t)
    for rows in ("tokens", "slots"):
        x = F.quantize(rnd(g, tokens if rows == "tokens" else tokens * k, k_in))
        x = (block(x[0], 0, -k_in % 16, NAN8)[1], x[1])
        X = on_gpu(x)
        for gated in (False, True):
            wide = 2 * n if gated else n
            w, b = expert_weights(g, experts, wide, k_in, gated), rnd(g, experts, wide)
            W = on_gpu(w)
            kw = dict(act="silu", gated=gated, rows=rows)
            log("experts", tokens, k, experts, k_in, n, rows, gated)
            out = torch.full((tokens * k, n), 5.0, dtype=t, device=device())
            E.expert_linear(X, W, P, gpu(b), k=k, out=out, **kw)
            want, bound, used = F.experts64(x, w, plan, k, b, **kw)
            R.check(out[:used], want[:used], bound[:used], t, "by slot")
            assert bool((out[used:] == 5).all())  # rows behind the last slot in use
            q = E.Quantized(torch.full((tokens * k, n), 0x11, dtype=torch.uint8, device=device()).view(FP8),
                            torch.full((tokens * k, F.blocks(n)), 7.0, device=device()))
            E.expert_linear(X, W, P, gpu(b), k=k, out=q, out_dtype=FP8, **kw)
            if used:
                want, bound, _ = F.experts64(x, w, plan, k, b, full=True, **kw)
                F.check_quantized((bits(q.values)[:used].view(FP8), q.scales[:used]), want[:used], bound[:used], "fp8")
            assert bool((q.values.view(torch.uint8)[used:] == 0x11).all()) and bool((q.scales[used:] == 7).all())
            y = E.expert_linear(X, W, P, gpu(b), k=k, combine=True, weight=gpu(weight), residual=gpu(r), **kw)
            want, bound, _ = F.experts64(x, w, plan, k, b, combine=True, weight=weight, residual=r, **kw)
            R.check(y, want, bound, t, "combined")
    y = E.expert_linear(X, W, P, k=k, rows="slots", gated=True, combine=True, out_dtype=torch.float32)
    want, bound, _ = F.experts64(x, w, plan, k, gated=True, rows="slots", combine=True, full=True)
    R.check(y, want, bound, torch.float32, "combined fp32, no weights")


@pytest.mark.parametrize("tokens,k,experts,k_in,n,gated", [*K.EXPERTS.values(), *K.EXPERTS_GATED.values()])
def test_expert_linear_by_kernel(tokens, k, experts, k_in, n, gated):
    """A size of every kernel's, by slot into each type that it writes, and combined; and outputs that are not finite."""
    g = gen(tokens + n)
    index = torch.randint(0, experts, (tokens, k), generator=g, dtype=torch.int32)
    plan = R.dispatch64(index, experts)
    P = ops.Dispatch(*map(gpu, plan))
    wide = 2 * n if gated else n
    x, w, b = F.quantize(rnd(g, tokens, k_in)), F.quantize_weights(rnd(g, experts, wide, k_in, scale=k_in ** -0.5), gated), rnd(g, experts, wide)
    X, W = put(x), put(w)
    weight, r = 0.1 + torch.rand(tokens, k, generator=g), rnd(g, tokens, n, dtype=torch.float16)
    for full in (False, True):
        want, e, _ = F.experts64(x, w, plan, k, b, "silu", gated, full=full)
        for t in (torch.float32, FP8) if full else (torch.float16, torch.bfloat16):
            log("experts", tokens, k, experts, k_in, n, gated, t, K.expert_kernel(tokens, k, experts, k_in, n, gated, E._OUT[t]))
            y = E.expert_linear(X, W, P, gpu(b), k=k, act="silu", gated=gated, out_dtype=t)
            F.check_quantized(y, want, e) if t == FP8 else R.check(y, want, e, t)
    for t in (torch.float16, torch.bfloat16, torch.float32):
        y = E.expert_linear(X, W, P, gpu(b), k=k, gated=gated, combine=True, weight=gpu(weight), residual=gpu(r.to(t)), out_dtype=t)
        want, e, _ = F.experts64(x, w, plan, k, b, "none", gated, combine=True, weight=weight, residual=r.to(t), full=t == torch.float32)
        R.check(y, want, e, t, "combined")
    b = torch.stack([without_odd(v[None])[0] for v in b])
    want, e, _ = F.experts64(x, w, plan, k, b, "none", gated, combine=True, weight=weight)
    for o, v in ODD:
        b[:, o] = v
        if gated:
            b[:, n + o] = 1e9
    y = E.expert_linear(X, W, P, gpu(b), k=k, gated=gated, combine=True, weight=gpu(weight))
    check_odd(y)
    R.check(without_odd(y), without_odd(want), without_odd(e), torch.bfloat16, "odd")
    q = E.expert_linear(X, W, P, gpu(b), k=k, gated=gated, out_dtype=FP8)
    check_odd(q.values, False)
    want, e, _ = F.experts64(x, w, plan, k, torch.stack([without_odd(v[None])[0] for v in b]), "none", gated, full=True)
    F.check_quantized((without_odd(bits(q.values)).view(FP8), q.scales), without_odd(want), without_odd(e), "odd fp8")


def test_expert_linear_same_expert_twice():
    """A token routed twice to one expert has two slots there, and both count."""
    g = gen(5)
    tokens, k, experts = 300, 4, 3
    x, w = F.quantize(rnd(g, tokens, 200)), expert_weights(g, experts, 136, 200, False)
    index = torch.randint(0, experts, (tokens, 1), generator=g, dtype=torch.int32).repeat(1, k)
    plan, weight = R.dispatch64(index, experts), torch.rand(tokens, k, generator=g)
    y = E.expert_linear(put(x), on_gpu(w), ops.dispatch(gpu(index), experts), k=k, combine=True, weight=gpu(weight))
    R.check(y, *F.experts64(x, w, plan, k, combine=True, weight=weight)[:2], torch.bfloat16)


def test_expert_linear_all_rows_to_one_expert_or_none():
    g, t = gen(22), torch.float16
    x, w = F.quantize(rnd(g, 700, 64)), expert_weights(g, 9, 40, 64, False)
    for value in (0, 4, 8, -1):
        plan = R.dispatch64(torch.full((700, 1), value, dtype=torch.int32), 9)
        P = ops.Dispatch(*map(gpu, plan))
        y = E.expert_linear(on_gpu(x), on_gpu(w), P, k=1, combine=True, out_dtype=t)
        R.check(y, *F.experts64(x, w, plan, 1, combine=True)[:2], t, value)


def test_expert_linear_bad_plans_stay_in_bounds():
    """Offsets, slots and places that no dispatch gives: clamped, the rows that are right stay right.  (Shown by
    reading first: every index is clamped to its buffer before use.)"""
    g = gen(77)
    x, w = on_gpu(F.quantize(rnd(g, 40, 64))), on_gpu(expert_weights(g, 3, 32, 64, False))
    index = torch.randint(0, 3, (40, 2), generator=g, dtype=torch.int32)
    offsets, slots, places = R.dispatch64(index, 3)
    y = E.expert_linear(x, w, ops.Dispatch(gpu(offsets), gpu(slots), gpu(places)), k=2)
    q = E.expert_linear(x, w, ops.Dispatch(gpu(offsets), gpu(slots), gpu(places)), k=2, out_dtype=FP8)
    far = slots.clone()
    far[-3:] = torch.tensor([-7, 80, 2 ** 31 - 1], dtype=torch.int32)
    bad = E.expert_linear(x, w, ops.Dispatch(gpu(offsets), gpu(far), gpu(places)), k=2)
    assert torch.equal(bad[:-3], y[:-3])
    wide = offsets.clone()
    wide[0], wide[3] = -5, 2 ** 31 - 1
    P = ops.Dispatch(gpu(wide), gpu(slots), gpu(places))
    assert torch.equal(E.expert_linear(x, w, P, k=2), y)
    again = E.expert_linear(x, w, P, k=2, out_dtype=FP8)
    assert torch.equal(bits(again.values), bits(q.values)) and torch.equal(again.scales, q.scales)
    out = places.clone()
    out[10], out[11] = -9, 80  # token 5: both dropped
    z = E.expert_linear(x, w, ops.Dispatch(gpu(offsets), gpu(slots), gpu(out)), k=2, combine=True)
    assert bool((z[5] == 0).all())


# ---- together ------------------------------------------------------------------------------------

def layer_of_experts(x, stream, g, w_router, w1, w2, k):
    """The norm of the residual stream, the router on its 16 bits, both layers of the experts on its 8."""
    h, q, stream = E.rms_norm(x, g, residual=stream, out="both")
    index, weight = ops.route(ops.linear(h, w_router, out_dtype=torch.float32), k, renormalise=True)
    plan = ops.dispatch(index, w1.values.shape[0])
    a = E.expert_linear(q, w1, plan, k=k, act="silu", gated=True, out_dtype=FP8)
    return E.expert_linear(a, w2, plan, k=k, rows="slots", combine=True, weight=weight), stream, (q, index, weight, a)


def model(seed, experts, d, hidden, t):
    g = gen(seed)
    w1 = E.quantize(gpu(rnd(g, experts, 2 * hidden, d, dtype=t, scale=d ** -0.5)), block_rows=128, gated=True)
    w2 = E.quantize(gpu(rnd(g, experts, d, hidden, dtype=t, scale=hidden ** -0.5)), block_rows=128)
    return (1 + rnd(g, d, scale=0.2)).to(t).to(device()), gpu(rnd(g, experts, d, dtype=t, scale=d ** -0.5)), w1, w2


@pytest.mark.parametrize("tokens", [1, 5, 130, 1000])
def test_a_layer_of_experts(tokens):
    """Norm, router, dispatch and both layers of the experts in a row: each against 64 bits on what the one before gave."""
    t, d, hidden, experts, k = torch.bfloat16, 200, 136, 12, 3
    weights = model(31, experts, d, hidden, t)
    x, r = rnd(gen(tokens), tokens, d, dtype=t), rnd(gen(tokens + 1), tokens, d, dtype=t)
    log("layer of experts", tokens)
    y, stream, (q, index, weight, a) = layer_of_experts(gpu(x), gpu(r), *weights, k)
    want, e, total = F.norm64(x, weights[0], r)
    assert torch.equal(stream.cpu(), total)
    F.check_quantized(q, want, e, "norm")
    plan = R.dispatch64(index, experts)
    used = int(plan[0][-1])
    assert used == tokens * k
    F.check_quantized(a, *F.experts64(q, weights[2], plan, k, act="silu", gated=True, full=True)[:2], "first")
    R.check(y, *F.experts64(a, weights[3], plan, k, rows="slots", combine=True, weight=weight)[:2], t, "second")


def test_two_streams_at_once():
    """Two runs on two streams, each with its own workspace, give what each gives alone."""
    t = torch.float16
    weights = model(41, 16, 256, 128, t)
    xs = [gpu(rnd(gen(s), 600, 256, dtype=t)) for s in (1, 2)]
    alone = [layer_of_experts(x, x, *weights, 4)[0] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for s, x in zip(streams, xs):
        with torch.cuda.stream(s):
            got.append([layer_of_experts(x, x, *weights, 4)[0] for _ in range(5)])
    torch.cuda.synchronize()
    for a, many in zip(alone, got):
        assert all(torch.equal(a, y) for y in many)


@pytest.mark.parametrize("tokens", [2, 900])
def test_captured_and_replayed(tokens):
    """The run recorded into a graph and replayed on new inputs, with eager work between: each replay is the
    eager result, bit for bit, and so is a second graph's of the same operators."""
    t = torch.bfloat16
    weights = model(51, 8, 192, 160, t)
    x, r = gpu(rnd(gen(1), tokens, 192, dtype=t)), gpu(rnd(gen(2), tokens, 192, dtype=t))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer_of_experts(x, r, *weights, 2)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            y, total, _ = layer_of_experts(x, r, *weights, 2)
        graphs.append((g, y, total))
    for i in range(4):
        x.copy_(gpu(rnd(gen(100 + i), tokens, 192, dtype=t)))
        eager, stream, _ = layer_of_experts(x, r, *weights, 2)
        torch.cuda.synchronize()
        for g, y, total in graphs:
            y.fill_(math.nan)
            total.fill_(math.nan)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, eager) and torch.equal(total, stream), i


def test_same_call_same_bits():
    t = torch.float16
    weights = model(61, 8, 200, 136, t)
    x = gpu(rnd(gen(1), 777, 200, dtype=t))
    first = layer_of_experts(x, x, *weights, 3)[0]
    assert all(torch.equal(first, layer_of_experts(x, x, *weights, 3)[0]) for _ in range(5))


class Never:
    """Stands for the extension: leaves every call to the functions in Python."""

    def __getattr__(self, name):
        return lambda *a: None


def flat(r):
    return [t for x in r for t in (flat(x) if isinstance(x, tuple) else [x])] if isinstance(r, tuple) else [r]


@pytest.mark.parametrize("rows,k,n", [(1, 128, 40), (5, 1001, 130), (300, 264, 300)])
def test_both_ways_to_the_library_are_one(rows, k, n, monkeypatch):
    """The usual call through the extension, and the same through the checks in Python: bits, types, shapes and strides."""
    g = gen(k)
    (x, w), (_, wg) = operands(g, rows, k, n), operands(g, rows, k, n, True)
    X, W, WG = on_gpu(x), on_gpu(w), on_gpu(wg)
    f, r, weight = gpu(rnd(g, rows, k)), gpu(rnd(g, rows, k)), gpu(rnd(g, k))
    b, res = gpu(rnd(g, n)), gpu(rnd(g, rows, n))
    index = torch.randint(-1, 3, (rows, 2), generator=g, dtype=torch.int32).to(device())
    plan = ops.dispatch(index, 3)
    w3 = on_gpu(expert_weights(g, 3, n, k, False))
    calls = [lambda: E.rms_norm(f), lambda: E.rms_norm(f.half(), weight.half(), residual=r.half(), out="both", eps=1e-3),
             lambda: E.rms_norm(f.bfloat16(), weight.bfloat16(), out="fp8"), lambda: E.rms_norm(f.half(), out_dtype=torch.float32),
             lambda: E.quantize(f), lambda: E.quantize(f.half(), block_rows=128), lambda: E.linear(X, W),
             lambda: E.quantize(f.view(rows, 1, k).expand(rows, 3, k).contiguous(), block_rows=128), lambda: E.quantize(f.half()[None]),
             lambda: E.linear(X, W, b, residual=res.half(), act="gelu", out_dtype=torch.float16),
             lambda: E.linear(X, WG, act="silu", gated=True, out_dtype=FP8), lambda: E.linear(X, W, out_dtype=torch.float32),
             lambda: E.expert_linear(X, w3, plan, k=2, combine=True, weight=torch.ones(rows, 2, device=device()), residual=res.bfloat16()),
             lambda: E.expert_linear(X, w3, plan, k=2, combine=True, out_dtype=torch.float32)]
    usual = E._usual
    seen = []

    class Spy:
        def __getattr__(self, name):
            def call(*a):
                seen.append(getattr(usual, name)(*a) is not None)
                return getattr(usual, name)(*a)
            return call
    for call in calls:
        monkeypatch.setattr(E, "_usual", Spy())
        a = flat(call())
        monkeypatch.setattr(E, "_usual", Never())
        for p, q in zip(a, flat(call())):
            assert (p is None) == (q is None)
            if p is not None:
                assert p.dtype == q.dtype and p.shape == q.shape and p.stride() == q.stride()
                assert torch.equal(bits(p), bits(q))
    assert len(seen) == len(calls) and all(seen)


def test_unusual_calls_are_left_to_the_checks():
    """Each is refused with Python's own words, whatever the extension sees of it."""
    d = device()
    x, w = E.quantize(torch.ones(4, 130, device=d)), E.quantize(torch.ones(8, 130, device=d), block_rows=128)
    f = torch.ones(4, 130, device=d)
    plan = ops.dispatch(torch.zeros(4, 2, dtype=torch.int32, device=d), 1)
    w3 = E.Quantized(w.values[None], w.scales[None])
    for call, says in ((lambda: E.linear(x, E.Quantized(w.values[:, :129], w.scales)), "w must be"),
                       (lambda: E.linear(x, E.Quantized(w.values, w.scales[:, :1])), "w.scales must be"),
                       (lambda: E.linear(E.Quantized(x.values, x.scales[:3]), w), "x.scales must be"),
                       (lambda: E.linear(x, w, torch.ones(7, device=d)), "bias"), (lambda: E.linear(x, w, torch.ones(8, device=d).half()), "bias"),
                       (lambda: E.linear(x, w, act="tanh"), "act"), (lambda: E.linear(x, w, out_dtype=torch.float64), "out_dtype"),
                       (lambda: E.linear(x, w, residual=torch.ones(4, 8, device=d)), "residual"),
                       (lambda: E.linear(x, E.Quantized(w.values[:7], w.scales), gated=True), "even"),
                       (lambda: E.linear(x, w, residual=f[:, :8].bfloat16().requires_grad_()), "gradient"),
                       (lambda: E.rms_norm(f, f[0, :7]), "weight"), (lambda: E.rms_norm(f, residual=f[:3]), "residual must be"),
                       (lambda: E.rms_norm(f, residual=f.half()), "of type"), (lambda: E.rms_norm(f.t()), "contiguous"),
                       (lambda: E.rms_norm(f.clone().requires_grad_()), "gradient"), (lambda: E.rms_norm(f, out_dtype=torch.float16), "out_dtype"),
                       (lambda: E.rms_norm(f, total=f), "total"), (lambda: E.quantize(f.t()), "contiguous"),
                       (lambda: E.quantize(f, block_rows=2), "block_rows"), (lambda: E.quantize(f[:3], block_rows=128, gated=True), "even"),
                       (lambda: E.expert_linear(x, w3, plan, k=3), "places"), (lambda: E.expert_linear(x, w3, plan, k=1), "rows, the plan"),
                       (lambda: E.expert_linear(x, w, plan, k=2), "3-D"), (lambda: E.expert_linear(x, w3, plan, k=2.0), "whole"),
                       (lambda: E.expert_linear(x, w3, plan._replace(offsets=plan.offsets[:1]), k=2), "offsets"),
                       (lambda: E.expert_linear(x, w3, plan, k=2, combine=True, weight=torch.ones(4, device=d)), "weight")):
        with pytest.raises(ValueError, match=says):
            call()
    for call, says in ((lambda: E.rms_norm(f, eps=0.0), "eps"), (lambda: E.linear(x, w, residual=torch.ones(4, 8, dtype=torch.uint8, device=d).view(FP8), out_dtype=FP8), "residual"),
                       (lambda: E.expert_linear(x, w3, plan, k=2, combine=True, out_dtype=FP8), "combine")):
        with pytest.raises(B.MlpError, match=says):
            call()


def test_no_rows():
    d = device()
    empty = E.Quantized(torch.empty(0, 130, dtype=torch.uint8, device=d).view(FP8), torch.empty(0, 2, device=d))
    w = E.quantize(torch.ones(5, 130, device=d), block_rows=128)
    assert E.linear(empty, w).shape == (0, 5)
    q = E.linear(empty, w, out_dtype=FP8)
    assert q.values.shape == (0, 5) and q.scales.shape == (0, 1)
    n = E.rms_norm(torch.empty(0, 130, device=d), out="both")
    assert n.y.shape == (0, 130) and n.quantized.scales.shape == (0, 2)
    assert E.quantize(torch.empty(0, 130, device=d)).scales.shape == (0, 2)
    plan = ops.dispatch(torch.empty(0, 2, dtype=torch.int32, device=d), 3)
    w3 = E.quantize(torch.ones(3, 5, 130, device=d), block_rows=128)
    assert E.expert_linear(empty, w3, plan, k=2, combine=True).shape == (0, 5)


def test_rows_and_experts_far_apart():
    """Matrices and rows whose offsets pass 2^31 elements."""
    far = (1 << 30) + 16
    base = torch.zeros(3 * far, dtype=torch.uint8, device=device()).view(FP8)
    near_w = E.quantize(gpu(rnd(gen(70), 3, 24, 300)), block_rows=128)
    near_x = E.quantize(gpu(rnd(gen(71), 3, 300)))
    w = base.as_strided((3, 24, 300), (far, 304, 1))
    w.view(torch.uint8).copy_(near_w.values.view(torch.uint8))
    x = base.as_strided((3, 300), (far, 1), 1 << 20)
    x.view(torch.uint8).copy_(near_x.values.view(torch.uint8))
    index = torch.tensor([[2, 0], [1, 2], [0, 1]], dtype=torch.int32, device=device())
    plan = ops.dispatch(index, 3)
    for combine in (False, True):
        got = E.expert_linear(E.Quantized(x, near_x.scales), E.Quantized(w, near_w.scales), plan, k=2, combine=combine)
        assert torch.equal(got, E.expert_linear(near_x, near_w, plan, k=2, combine=combine))
    wide = base.view(torch.uint8).view(torch.float16).as_strided((3, 500), (far // 2, 1), 1 << 19)
    values = rnd(gen(72), 3, 500, dtype=torch.float16)
    wide.copy_(gpu(values))
    same(E.quantize(wide), F.quantize(values))
    assert torch.equal(E.rms_norm(wide).y, E.rms_norm(gpu(values)).y)


def test_more_than_32_bits_of_elements():
    """Outputs, 8-bit rows, terms and normed rows of more than 2^31 elements; the last rows against 64 bits."""
    g = gen(80)
    rows, k, n = (1 << 20) + 300, 16, 2056
    x, w = F.quantize(rnd(g, 1000, k)), F.quantize_weights(rnd(g, n, k, scale=k ** -0.5))
    many = [gpu(t).repeat(-(-rows // 1000), 1)[:rows] for t in (x[0].view(torch.uint8), x[1])]
    X, W = E.Quantized(many[0].view(FP8), many[1]), put(w)
    last = slice(rows - 700, rows)
    tail = (X.values[last].cpu(), X.scales[last].cpu())
    for t in (torch.bfloat16, FP8):
        log("many rows", t)
        y = E.linear(X, W, out_dtype=t)
        if t == FP8:
            F.check_quantized((bits(y.values[last]).view(FP8), y.scales[last]), *F.linear64(tail, w, full=True))
        else:
            R.check(y[last], *F.linear64(tail, w), t)
        if t != FP8:
            log("norm, 8 bits")
            normed = E.rms_norm(y, residual=y, out="both")
            h, e, total = F.norm64(y[last], residual=y[last])
            R.check(normed.y[last], h, e, t)
            assert torch.equal(normed.total[last].cpu(), total)
            same(E.Quantized(normed.quantized.values[last], normed.quantized.scales[last]),
                 tuple(q.cpu() for q in E.rms_norm(y[last], residual=y[last], out="fp8").quantized))
            del normed
            q = E.quantize(y)
            same(E.Quantized(q.values[last], q.scales[last]), F.quantize(y[last].cpu()))
            del q
        del y
    tokens, kk, experts = rows // 4, 4, 3
    we = F.quantize_weights(rnd(g, experts, n, k, scale=k ** -0.5))
    index = torch.randint(0, experts, (tokens, kk), generator=g, dtype=torch.int32)
    weight = torch.rand(tokens, kk, generator=g)
    log("many slots")
    y = E.expert_linear(E.Quantized(X.values[:tokens], X.scales[:tokens]), put(we), ops.dispatch(gpu(index), experts), k=kk,
                        combine=True, weight=gpu(weight))
    at = slice(tokens - 500, tokens)
    want, e, _ = F.experts64((X.values[at].cpu(), X.scales[at].cpu()), we, R.dispatch64(index[at], experts), kk, combine=True, weight=weight[at])
    R.check(y[at], want, e, torch.bfloat16)


@pytest.mark.parametrize("rows,k,n", [(3, 1 << 20, 3), (2, 9, 1 << 20), (70, 17, (1 << 20) - 3), (700, 8200, 701), (700, 8201, 700)])
def test_widest(rows, k, n):
    """The largest widths, and long rows through the kernels that stage them."""
    g = gen(rows + k)
    x, w = operands(g, rows, k, n)
    X, W, b = on_gpu(x), on_gpu(w), rnd(g, n)
    for full in (False, True):
        want = F.linear64(x, w, b, full=full)
        for t in (torch.float32, FP8) if full else (torch.bfloat16,):
            log("widest", rows, k, n, t, K.linear_kernel(rows, k, n, out_dtype=E._OUT[t]))
            y = E.linear(X, W, gpu(b), out_dtype=t)
            F.check_quantized(y, *want) if t == FP8 else R.check(y, *want, t)


def test_widest_rows():
    g, t, width = gen(90), torch.bfloat16, 1 << 20
    x, r, w = rnd(g, 3, width, dtype=t), rnd(g, 3, width, dtype=t), rnd(g, width, dtype=t)
    y, e, total = F.norm64(x, w, r)
    got = E.rms_norm(gpu(x), gpu(w), residual=gpu(r), out="both")
    R.check(got.y, y, e, t)
    assert torch.equal(got.total.cpu(), total)
    same(got.quantized, tuple(q.cpu() for q in E.rms_norm(gpu(x), gpu(w), residual=gpu(r), out="fp8").quantized))
    for block_rows in (1, 128):
        got = E.quantize(gpu(x), block_rows=block_rows)
        one = E.quantize(gpu(x[:, 5 * 128:6 * 128].contiguous()), block_rows=block_rows)
        assert torch.equal(bits(got.values[:, 640:768]), bits(one.values)) and torch.equal(got.scales[:, 5:6], one.scales)
        last = E.quantize(gpu(x[:, -256:].contiguous()), block_rows=block_rows)
        assert torch.equal(bits(got.values[:, -256:]), bits(last.values)) and torch.equal(got.scales[:, -2:], last.scales)
    index = torch.tensor([[0, 1], [1, 1]], dtype=torch.int32)
    plan, x, w = R.dispatch64(index, 2), F.quantize(rnd(g, 2, 40)), F.quantize_weights(rnd(g, 2, width, 40))
    y = E.expert_linear(put(x), put(w), ops.Dispatch(*map(gpu, plan)), k=2, combine=True)
    R.check(y, *F.experts64(x, w, plan, 2, combine=True)[:2], t)
