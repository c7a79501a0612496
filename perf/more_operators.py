"""Cases for the operators of ``include/mlp_ops_fp8.h``: layers whose operands are 8-bit floating point (E4M3) with
an FP32 scale for each block of 128 columns.  The root-mean-square norm with the residual's addition that feeds them
(``rms_norm``), the rounding to 8 bits itself (``quantize``), one affine layer (``linear``) and the experts' layers
on routed rows of ragged counts (``expert_linear``).

``run`` with ``own = False`` is each operator in plain torch operations, in 32 bits; with ``own = True`` it is the
call that a user makes.  ``exact`` is the definition in 64 bits, 8-bit outputs before their rounding.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32, "fp8": torch.float8_e4m3fn}
FP8 = torch.float8_e4m3fn
BLOCK = 128  # columns (and, of weights, rows) that share a scale
LARGEST = 448.0  # of E4M3
SMALLEST = 2.0 ** -126  # of a scale
EPS = 1e-6
SLOPE = 0.01000213623046875  # half(0.01), the slope of the leaky ReLU throughout the library


# ---- the cases -----------------------------------------------------------------------------------

def _norm(rows, width, dtype, out, residual=False, name=None):
    c = {"op": "norm", "rows": rows, "width": width, "dtype": dtype, "out": out, "residual": residual}
    return dict(c, name=name) if name else c


def _quantize(count, rows, width, dtype, block_rows, name=None):
    c = {"op": "quantize", "count": count, "rows": rows, "width": width, "dtype": dtype, "block_rows": block_rows}
    return dict(c, name=name) if name else c


def _linear(rows, k, n, out, act, gated=False, bias=True, residual=False, name=None):
    c = {"op": "linear", "rows": rows, "in": k, "out": n, "out_dtype": out, "act": act, "gated": gated, "bias": bias,
         "residual": residual}
    return dict(c, name=name) if name else c


def _experts(tokens, k, experts, width_in, width_out, out, act, gated=False, bias=False, rows="tokens", combine=False,
             residual=False, name=None):
    c = {"op": "experts", "tokens": tokens, "k": k, "experts": experts, "in": width_in, "out": width_out,
         "out_dtype": out, "act": act, "gated": gated, "bias": bias, "rows": rows, "combine": combine,
         "residual": residual}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token before its layer: latency
        _norm(1, 2048, "bf16", "fp8", residual=True, name="norm 1 token"),
        # a batch and a width that no block divides, 16 bits to 16 bits
        _norm(5003, 1001, "fp16", "same", name="norm odd"),
        # the residual stream of the 1024-wide network over its whole batch, into 8 bits
        _norm(65536, 1024, "bf16", "fp8", residual=True, name="norm 65536 rows"),
        # a small batch's activations rounded before a layer: latency
        _quantize(1, 33, 2048, "fp16", 1, name="quantize 33 rows"),
        # the experts' first layers rounded when a model is loaded, a scale for each 128 x 128
        _quantize(32, 2048, 2048, "bf16", 128, name="quantize experts"),
        # one evaluation of a 1024-wide hidden layer: latency, bound by reading the weights once
        _linear(1, 1024, 1024, "fp16", "leaky_relu", name="linear 1 row"),
        # a handful of concurrent requests through a gated first layer: bound by the weights' bytes
        _linear(7, 2048, 4096, "bf16", "silu", gated=True, bias=False, name="linear 7 rows gated"),
        # widths and a batch that no tile and no block divides, with a skip connection
        _linear(5003, 1001, 777, "fp16", "relu", residual=True, name="linear odd residual"),
        # the hidden layer of the library's 1024-wide network over its whole batch
        _linear(65536, 1024, 1024, "bf16", "gelu", residual=True, name="linear 65536 rows"),
        # eight tokens through their experts' first layers: each chosen expert's weights are read once
        _experts(8, 4, 32, 1024, 1024, "bf16", "silu", gated=True, name="experts 8 tokens gated"),
        # a prompt through the experts' gated first layers, into 8 bits for the second
        _experts(8192, 4, 32, 2048, 1024, "fp8", "silu", gated=True, name="experts 8192 gated"),
        # the same prompt's second layers, summed by the router's weights onto the residual stream
        _experts(8192, 4, 32, 1024, 2048, "bf16", "none", rows="slots", combine=True, residual=True,
                 name="experts 8192 combine"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    w = _log(rng, lo, hi)
    return w if rng.random() < 0.3 else max(8, w // 8 * 8)


def _act(rng, gated):
    return rng.choice(["silu", "gelu", "relu"] if gated else ["none", "leaky_relu", "relu", "gelu", "silu"])


def draw(rng):
    op = rng.choice(["norm", "quantize", "linear", "linear", "experts", "experts"])
    if op == "norm":
        width = _width(rng, 16, 8192)
        return _norm(_log(rng, 1, min(65536, (1 << 26) // width)), width, rng.choice(["fp16", "bf16", "fp32"]),
                     rng.choice(["same", "fp8", "both"]), rng.random() < 0.6)
    if op == "quantize":
        width, dtype = _width(rng, 16, 8192), rng.choice(["fp16", "bf16", "fp32"])
        if rng.random() < 0.5:
            return _quantize(1, _log(rng, 1, min(65536, (1 << 26) // width)), width, dtype, 1)
        count = _log(rng, 1, 32)
        return _quantize(count, _log(rng, 16, max(16, min(8192, (1 << 26) // width // count))), width, dtype, 128)
    gated = rng.random() < 0.3
    act = _act(rng, gated)
    if op == "linear":
        rows, k, n = _log(rng, 1, 65536), _width(rng, 16, 4096), _width(rng, 16, 4096)
        rows = max(1, min(rows, int(1.3e11 / (2 * k * n * (1 + gated)))))
        out = rng.choice(["fp16", "bf16", "fp32", "fp8"])
        return _linear(rows, k, n, out, act, gated, rng.random() < 0.6, out != "fp8" and rng.random() < 0.4)
    experts = _log(rng, 2, 128)
    k = min(_log(rng, 1, 8), experts)
    combine = rng.random() < 0.5
    k_in, n = _width(rng, 16, 2048), _width(rng, 16, 2048)
    while experts * k_in * n * (1 + gated) > 1 << 27:
        experts, k = max(2, experts // 2), min(k, max(2, experts // 2))
    most = min(int(1.3e11 / (2 * k_in * n * (1 + gated))), (1 << 26) // max(k_in, n * (1 + gated)), 262144) // k
    out = rng.choice(["fp16", "bf16", "fp32"] if combine else ["fp16", "bf16", "fp32", "fp8"])
    return _experts(_log(rng, 1, max(1, most)), k, experts, k_in, n, out, act, gated, rng.random() < 0.5,
                    rng.choice(["tokens", "slots"]), combine, combine and rng.random() < 0.5)


# ---- 8 bits --------------------------------------------------------------------------------------

def _blocks(x):
    """The last dimension in blocks of 128, the last one filled with zeros: [..., blocks, 128]."""
    n = -(-x.shape[-1] // BLOCK)
    full = x.new_zeros(*x.shape[:-1], n * BLOCK)
    full[..., :x.shape[-1]] = x
    return full.unflatten(-1, (n, BLOCK))


def _scales(x, block_rows):
    """amax / 448 of each block of `block_rows` x 128 of the last two dimensions of x (32 or 64 bits)."""
    amax = _blocks(x).abs().amax(-1)
    if block_rows > 1:
        n = -(-amax.shape[-2] // block_rows)
        full = amax.new_zeros(*amax.shape[:-2], n * block_rows, amax.shape[-1])
        full[..., :amax.shape[-2], :] = amax
        amax = full.unflatten(-2, (n, block_rows)).amax(-2)
    return (amax / LARGEST).clamp(min=SMALLEST)


def _spread(scales, rows, width, block_rows):
    """Each element's scale."""
    s = scales.repeat_interleave(BLOCK, dim=-1)[..., :width]
    return s.repeat_interleave(block_rows, dim=-2)[..., :rows, :] if block_rows > 1 else s


def _to8(x, block_rows=1):
    """x in 8 bits and its scales."""
    scales = _scales(x, block_rows)
    return (x / _spread(scales, x.shape[-2], x.shape[-1], block_rows)).to(FP8), scales


def _from8(values, scales, block_rows=1):
    return values.to(scales.dtype) * _spread(scales, values.shape[-2], values.shape[-1], block_rows)


# ---- inputs --------------------------------------------------------------------------------------

def _choices(tokens, k, experts, gen):
    """Each token's k distinct experts, some of them more popular than others."""
    popularity = torch.randn(experts, generator=gen, device="cuda") * 0.5
    if k == 1:
        return torch.multinomial(popularity.exp(), tokens, replacement=True, generator=gen).to(torch.int32)[:, None]
    noise = -torch.log(-torch.log(torch.rand(tokens, experts, generator=gen, device="cuda").clamp(1e-9, 1 - 1e-7)))
    return (noise + popularity).topk(k, dim=1).indices.to(torch.int32)


def _aligned(values):
    """The same values in rows of whole 16 bytes, as the framework lays them out."""
    width = values.shape[-1]
    wide = torch.zeros(*values.shape[:-1], -(-width // 16) * 16, dtype=torch.uint8, device=values.device)
    wide[..., :width] = values.view(torch.uint8)
    return wide.view(FP8)[..., :width]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    def activations(rows, width, dtype=torch.float32):
        # some channels are larger than others, as behind a norm's weights
        return (normal(rows, width) * torch.exp(normal(width, scale=0.5))).to(dtype)

    def eight(x, block_rows=1, halves=1):
        parts = [_to8(p, block_rows) for p in x.chunk(halves, dim=-2)]  # a gated layer's blocks start anew at its second half
        return _aligned(torch.cat([p[0].view(torch.uint8) for p in parts], -2).view(FP8)), torch.cat([p[1] for p in parts], -2)

    st = {"case": case}
    if case["op"] == "norm":
        dtype = DTYPES[case["dtype"]]
        st["x"] = activations(case["rows"], case["width"], dtype)
        st["residual"] = normal(case["rows"], case["width"], dtype=dtype, scale=2.0) if case["residual"] else None
        st["weight"] = (1 + normal(case["width"], scale=0.2)).to(dtype)
        return st
    if case["op"] == "quantize":
        dtype = DTYPES[case["dtype"]]
        if case["block_rows"] == 1:
            st["x"] = activations(case["rows"], case["width"], dtype)
        else:
            st["x"] = normal(case["count"], case["rows"], case["width"], dtype=dtype, scale=case["width"] ** -0.5)
        return st
    k_in, n = case["in"], case["out"]
    halves = 2 if case["gated"] else 1
    wide = n * halves
    out = DTYPES[case["out_dtype"]]
    if case["op"] == "linear":
        rows = case["rows"]
        st["x"], st["xs"] = eight(activations(rows, k_in))
        st["w"], st["ws"] = eight(normal(wide, k_in, scale=k_in ** -0.5), BLOCK, halves)
        st["b"] = normal(wide, scale=0.1) if case["bias"] else None
        st["residual"] = normal(rows, n, dtype=out) if case["residual"] else None
        return st
    tokens, k, experts = case["tokens"], case["k"], case["experts"]
    index = _choices(tokens, k, experts, gen)
    flat = index.reshape(-1).long()
    slots = torch.sort(flat, stable=True).indices
    places = torch.empty_like(slots)
    places[slots] = torch.arange(tokens * k, device="cuda")
    counts = torch.bincount(flat, minlength=experts)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    st.update(offsets=offsets.to(torch.int32), slots=slots.to(torch.int32), places=places.to(torch.int32),
              most=int(counts.max()))  # the plan, and the largest expert's rows, which the plain form pads to
    st["x"], st["xs"] = eight(activations(tokens if case["rows"] == "tokens" else tokens * k, k_in))
    st["w"], st["ws"] = eight(normal(experts, wide, k_in, scale=k_in ** -0.5), BLOCK, halves)
    st["b"] = normal(experts, wide, scale=0.1) if case["bias"] else None
    weight = torch.rand(tokens, k, generator=gen, device="cuda") + 0.1
    st["weight"] = weight / weight.sum(1, keepdim=True) if case["combine"] else None
    st["residual"] = normal(tokens, n, dtype=out) if case["residual"] else None
    return st


# ---- one pass ------------------------------------------------------------------------------------

def _activation(v, name):
    if name == "leaky_relu":
        return torch.where(v > 0, v, v * SLOPE)
    if name == "relu":
        return v.clamp(min=0)
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if name == "silu":
        return v / (1 + torch.exp(-v))
    return v


def _epilogue(z, c):
    n = c["out"]
    return _activation(z[..., :n], c["act"]) * z[..., n:] if c["gated"] else _activation(z, c["act"])


def _weights(st):
    """The weights in 32 bits; a gated layer's two halves have blocks of their own."""
    w, ws = st["w"], st["ws"]
    if not st["case"]["gated"]:
        return _from8(w, ws, BLOCK)
    n, b = w.shape[-2] // 2, ws.shape[-2] // 2
    return torch.cat([_from8(w[..., :n, :], ws[..., :b, :], BLOCK), _from8(w[..., n:, :], ws[..., b:, :], BLOCK)], -2)


def _plain_norm(st):
    c, x = st["case"], st["x"]
    total = x if st["residual"] is None else (x.float() + st["residual"].float()).to(x.dtype)
    t = total.float()
    y = t * torch.rsqrt((t * t).mean(1, keepdim=True) + EPS) * st["weight"].float()
    out = (() if c["out"] == "fp8" else (y.to(x.dtype),)) + (() if c["out"] == "same" else _to8(y))
    return out + (() if st["residual"] is None else (total,))


def _plain_linear(st):
    c = st["case"]
    z = _from8(st["x"], st["xs"]) @ _weights(st).t()
    if st["b"] is not None:
        z = z + st["b"]
    y = _epilogue(z, c)
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return _to8(y) if c["out_dtype"] == "fp8" else y.to(DTYPES[c["out_dtype"]])


def _plain_experts(st):
    c, offsets, slots = st["case"], st["offsets"].long(), st["slots"].long()
    tokens, k, most = c["tokens"], c["k"], st["most"]
    at = torch.arange(tokens * k, device=slots.device)
    expert = torch.searchsorted(offsets, at, right=True) - 1
    row = expert * most + at - offsets[expert]  # the slot's place among its expert's padded rows
    x = _from8(st["x"], st["xs"])
    padded = x.new_zeros(c["experts"] * most, c["in"])
    padded[row] = x[slots // k] if c["rows"] == "tokens" else x
    z = torch.bmm(padded.view(c["experts"], most, c["in"]), _weights(st).transpose(1, 2).contiguous())
    if st["b"] is not None:
        z = z + st["b"][:, None]
    y = _epilogue(z, c).reshape(c["experts"] * most, c["out"])[row]
    if c["combine"]:
        y = (y[st["places"].long()].view(tokens, k, c["out"]) * st["weight"][..., None]).sum(1)
        if st["residual"] is not None:
            y = y + st["residual"].float()
    return _to8(y) if c["out_dtype"] == "fp8" else y.to(DTYPES[c["out_dtype"]])


def run(state):
    c = state["case"]
    if own:
        from mlp_neural_shading_amd import ops, ops_fp8

        if c["op"] == "norm":
            y, quantized, total = ops_fp8.rms_norm(state["x"], state["weight"], residual=state["residual"], eps=EPS, out=c["out"])
            return (() if y is None else (y,)) + (() if quantized is None else tuple(quantized)) + (() if total is None else (total,))
        if c["op"] == "quantize":
            return tuple(ops_fp8.quantize(state["x"], block_rows=c["block_rows"]))
        x, w = ops_fp8.Quantized(state["x"], state["xs"]), ops_fp8.Quantized(state["w"], state["ws"])
        out = DTYPES[c["out_dtype"]]
        if c["op"] == "linear":
            y = ops_fp8.linear(x, w, state["b"], residual=state["residual"], act=c["act"], gated=c["gated"], out_dtype=out)
        else:
            plan = ops.Dispatch(state["offsets"], state["slots"], state["places"])
            y = ops_fp8.expert_linear(x, w, plan, state["b"], k=c["k"], act=c["act"], gated=c["gated"], rows=c["rows"],
                                      combine=c["combine"], weight=state["weight"], residual=state["residual"],
                                      out_dtype=out)
        return tuple(y) if c["out_dtype"] == "fp8" else y
    if c["op"] == "norm":
        return _plain_norm(state)
    if c["op"] == "quantize":
        return _to8(state["x"].float(), c["block_rows"])
    if c["op"] == "linear":
        return _plain_linear(state)
    return _plain_experts(state)


# ---- what a pass cannot do without ---------------------------------------------------------------

SIZES = {"fp32": 4, "fp16": 2, "bf16": 2, "fp8": 1}


def work(case):
    c = case
    up = lambda n: -(-n // BLOCK)  # noqa: E731
    if c["op"] == "norm":
        size, n = SIZES[c["dtype"]], c["rows"] * c["width"]
        eight = n + 4 * c["rows"] * up(c["width"])
        return {"bytes": n * size * (1 + 2 * c["residual"] + (c["out"] != "fp8")) + (c["out"] != "same") * eight + size * c["width"],
                "flops": 5.0 * n}
    if c["op"] == "quantize":
        n = c["count"] * c["rows"] * c["width"]
        return {"bytes": n * (SIZES[c["dtype"]] + 1) + 4 * c["count"] * up(c["width"]) * -(-c["rows"] // c["block_rows"]),
                "flops": 2.0 * n}
    halves = 2 if c["gated"] else 1
    wide, out = c["out"] * halves, SIZES[c["out_dtype"]]
    each = c["out"] * out + (4 * up(c["out"]) if c["out_dtype"] == "fp8" else 0)  # bytes of a row of outputs
    w_bytes = wide * c["in"] + 4 * halves * up(c["out"]) * up(c["in"]) + 4 * wide * c["bias"]
    x_bytes = c["in"] + 4 * up(c["in"])
    if c["op"] == "linear":
        return {"bytes": float(c["rows"] * (x_bytes + each + c["residual"] * c["out"] * out) + w_bytes),
                "flops": 2.0 * c["rows"] * c["in"] * wide}
    slots = c["tokens"] * c["k"]
    hit = c["experts"] * (1 - (1 - c["k"] / c["experts"]) ** c["tokens"])  # experts that some token chose
    rows_in = c["tokens"] if c["rows"] == "tokens" else slots
    rows_out = c["tokens"] if c["combine"] else slots
    return {"bytes": hit * w_bytes + rows_in * x_bytes + rows_out * each + c["tokens"] * c["out"] * out * c["residual"]
            + 4.0 * slots * (2 if c["combine"] else 1),
            "flops": 2.0 * slots * c["in"] * wide}


# ---- the definitions in 64 bits ------------------------------------------------------------------

def _exact_act(v, name):
    if name == "leaky_relu":
        return torch.maximum(v, v * SLOPE)
    if name == "relu":
        return torch.maximum(v, torch.zeros_like(v))
    if name == "gelu":
        return v * torch.special.erfc(-v / math.sqrt(2.0)) / 2
    if name == "silu":
        return v * torch.sigmoid(v)
    return v


def _exact8(y, block_rows=1):
    """What the 8-bit values and the scales stand for, before any rounding."""
    rows, width = y.shape[-2:]
    scales = y.new_zeros(*y.shape[:-2], -(-rows // block_rows), -(-width // BLOCK))
    values = torch.empty_like(y)
    for j in range(scales.shape[-1]):
        part = y[..., j * BLOCK:(j + 1) * BLOCK]
        if block_rows == 1:
            s = part.abs().max(-1).values / LARGEST
            scales[..., j] = s
            values[..., j * BLOCK:(j + 1) * BLOCK] = part / torch.maximum(s, s.new_tensor(SMALLEST))[..., None]
            continue
        for i in range(scales.shape[-2]):
            block = part[..., i * block_rows:(i + 1) * block_rows, :]
            s = block.abs().flatten(-2).max(-1).values / LARGEST
            scales[..., i, j] = s
            values[..., i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK] = \
                block / torch.maximum(s, s.new_tensor(SMALLEST))[..., None, None]
    return values, torch.maximum(scales, scales.new_tensor(SMALLEST))


def _exact_operand(values, scales, block_rows):
    v = values.to(torch.float64)
    for j in range(scales.shape[-1]):
        s = scales[:, j].double()
        s = s.repeat_interleave(block_rows)[:v.shape[0]] if block_rows > 1 else s
        v[:, j * BLOCK:(j + 1) * BLOCK] *= s[:, None]
    return v


def _exact_layer(x, xs, w, ws, b, c):
    x = _exact_operand(x, xs, 1)
    halves = 2 if c["gated"] else 1
    parts = []
    for i in range(halves):
        n, blocks = w.shape[0] // halves, ws.shape[0] // halves
        z = x @ _exact_operand(w[i * n:(i + 1) * n], ws[i * blocks:(i + 1) * blocks], BLOCK).t()
        parts.append(z if b is None else z + b[i * n:(i + 1) * n].double())
    y = _exact_act(parts[0], c["act"])
    return y * parts[1] if c["gated"] else y


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "quantize":
        return _exact8(st["x"].double(), c["block_rows"])
    if c["op"] == "norm":
        total = st["x"].double()
        if st["residual"] is not None:
            total = (total + st["residual"].double()).to(st["x"].dtype).double()  # the stream's one rounding
        y = total / torch.sqrt((total ** 2).sum(1, keepdim=True) / c["width"] + EPS) * st["weight"].double()
        out = [] if c["out"] == "fp8" else [y]
        if c["out"] != "same":
            out += _exact8(y)
        return tuple(out + ([] if st["residual"] is None else [total]))
    if c["op"] == "linear":
        y = _exact_layer(st["x"], st["xs"], st["w"], st["ws"], st["b"], c)
        y = y if st["residual"] is None else y + st["residual"].double()
        return _exact8(y) if c["out_dtype"] == "fp8" else y
    ends, order, k = st["offsets"].tolist(), st["slots"].long(), c["k"]
    y = torch.zeros(c["tokens"] * k, c["out"], dtype=torch.float64, device="cuda")
    for e in range(c["experts"]):
        lo, hi = ends[e], ends[e + 1]
        if lo < hi:
            at = order[lo:hi] // k if c["rows"] == "tokens" else torch.arange(lo, hi, device="cuda")
            y[lo:hi] = _exact_layer(st["x"][at], st["xs"][at], st["w"][e], st["ws"][e],
                                    None if st["b"] is None else st["b"][e], c)
    if c["combine"]:
        out = torch.zeros(c["tokens"], c["out"], dtype=torch.float64, device="cuda")
        if st["residual"] is not None:
            out += st["residual"].double()
        for j in range(k):
            out += y[st["places"].view(-1, k)[:, j].long()] * st["weight"][:, j:j + 1].double()
        return out
    return _exact8(y) if c["out_dtype"] == "fp8" else y
