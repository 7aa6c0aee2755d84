"""The MXFP4 operators with both operands in 4 bits: what they compute, in plain torch operations, on real work.

MXFP4 (OCP Microscaling Formats, version 1.0): a block of 32 values along the contracted axis is held as 32 E2M1 codes
(levels 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign) and one E8M0 byte s that stands for 2^(s - 127); s = 255 marks a block with
a NaN. A block's byte is floor(log2(largest magnitude)) - 2 + 127, at least 0; its values are rounded to the nearest
level times the scale, halves to the even code, and what lies past 6 times the scale becomes 6 times the scale.

Four operators:
  quantize  x -> codes and scales along its rows, along its columns (the transposed operand), or both from one reading
  product   y = A B^T of two MXFP4 operands
  linear    y = Q(x) B^T, x dense: the activations are quantised on the way into the product
  train     y = Q(x) Q(w)^T and, for a gradient g of y, dx = Q(g) Q(w^T)^T and dw = Q(g^T) Q(x^T)^T, every operand
            quantised along the axis that its product contracts

`own` False computes these in plain torch operations, True calls the library.
"""
import math

import torch

own = False

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
BYTES = {"float32": 4, "bfloat16": 2, "float16": 2}


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one token's activations in front of a projection: the smallest call, all latency
        {"name": "quantize token", "op": "quantize", "axes": "rows", "m": 1, "k": 4096, "dtype": "bfloat16"},
        # a prompt's activations in front of the down projection
        {"name": "quantize prompt", "op": "quantize", "axes": "rows", "m": 2048, "k": 9728, "dtype": "bfloat16"},
        # a gradient that two products contract along different axes, with a ragged number of tokens
        {"name": "quantize gradient", "op": "quantize", "axes": "both", "m": 4095, "k": 9728, "dtype": "bfloat16"},
        # master weights at the start of a training step
        {"name": "quantize weights", "op": "quantize", "axes": "both", "m": 9728, "k": 2560, "dtype": "float32"},
        # decode of one token, gate projection of a 4B-class layer
        {"name": "product token", "op": "product", "m": 1, "n": 9728, "k": 2560, "out": "float32"},
        # verifying eight drafted tokens, down projection of the same layer
        {"name": "product verify", "op": "product", "m": 9, "n": 2560, "k": 9728, "out": "float32"},
        # a batch of 64 requests at decode, a wide projection
        {"name": "product batch", "op": "product", "m": 64, "n": 14336, "k": 4096, "out": "bfloat16"},
        # prefill of a long prompt, the largest product
        {"name": "product prompt", "op": "product", "m": 8192, "n": 14336, "k": 4096, "out": "bfloat16"},
        # one token through a square projection, activations still dense
        {"name": "linear token", "op": "linear", "m": 1, "n": 4096, "k": 4096, "dtype": "bfloat16", "out": "float32"},
        # a chunk of a prompt with an odd number of tokens, activations still dense
        {"name": "linear chunk", "op": "linear", "m": 333, "n": 2560, "k": 9728, "dtype": "bfloat16", "out": "bfloat16"},
        # a small training step: key/value projection, ragged tokens, float32 master weights
        {"name": "train small", "op": "train", "m": 257, "n": 1024, "k": 2560, "dtype": "bfloat16", "weight": "float32"},
        # a large training step: gate projection over 8192 tokens
        {"name": "train large", "op": "train", "m": 8192, "n": 9728, "k": 2560, "dtype": "bfloat16", "weight": "bfloat16"},
    ]


def _spread(rng, low, high):
    """A whole number whose logarithm is spread evenly."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("quantize", "product", "product", "linear", "train"))
    if op == "quantize":
        # the rows of the largest listed case and its values are not passed
        m = _spread(rng, 1, 16384)
        k = _spread(rng, 32, max(32, min(16384, 36_000_000 // m)))
        return {"op": op, "axes": rng.choice(("rows", "columns", "both")), "m": m, "k": k,
                "dtype": rng.choice(("float32", "bfloat16", "float16"))}
    if op == "train":
        m = _spread(rng, 32, 8192)
        return {"op": op, "m": m, "n": 8 * _spread(rng, 16, 1216), "k": 8 * _spread(rng, 16, 320), "dtype": "bfloat16",
                "weight": rng.choice(("float32", "bfloat16"))}
    m, n, k = _spread(rng, 1, 4096), _spread(rng, 128, 14336), 32 * _spread(rng, 4, 304)
    case = {"op": op, "m": m, "n": n, "k": k, "out": rng.choice(("float32", "bfloat16"))}
    if op == "linear":
        case["dtype"] = rng.choice(("bfloat16", "float16"))
    return case


def work(case):
    m, k = case["m"], case["k"]
    packed = lambda r, d: r * d / 2 + r * d / 32  # noqa: E731
    if case["op"] == "quantize":
        back = 2 if case["dtype"] == "bfloat16" else 4
        return {"bytes": m * k * (BYTES[case["dtype"]] + back * (2 if case["axes"] == "both" else 1)), "flops": 0}
    n = case["n"]
    if case["op"] == "product":
        return {"bytes": packed(m, k) + packed(n, k) + m * n * BYTES[case["out"]], "flops": 2 * m * n * k}
    if case["op"] == "linear":
        return {"bytes": m * k * BYTES[case["dtype"]] + packed(n, k) + m * n * BYTES[case["out"]], "flops": 2 * m * n * k}
    a, w = BYTES[case["dtype"]], BYTES[case["weight"]]
    return {"bytes": 2 * m * k * a + 2 * n * k * w + 2 * m * n * a, "flops": 6 * m * n * k}


# ----------------------------------------------------------------------------------------------- inputs

def _activations(m, k, dtype, gen):
    """Normal values with a few loud channels, quiet rows, and blocks of zeros, as layers meet them."""
    x = torch.randn(m, k, generator=gen, device="cuda")
    loud = torch.rand(k, generator=gen, device="cuda") < 0.004
    x = x * torch.where(loud, 12.0, 1.0)
    x = x * torch.exp2(torch.randint(-3, 4, (m, 1), generator=gen, device="cuda").float())
    pad = (k + 31) // 32
    keep = (torch.rand(m, pad, generator=gen, device="cuda") >= 0.01).float()
    return (x * keep.repeat_interleave(32, 1)[:, :k]).to(dtype)


def _operand(values):
    """Codes [r][d/2] (element 2j in the low half of byte j) and scales [r][d/32] of dense values, the rows of the
    scales a multiple of 4 bytes apart: what a program holds of an operand that was quantised earlier."""
    r, d = values.shape
    b = values.float().reshape(r, d // 32, 32)
    s = ((b.abs().amax(2).view(torch.int32) >> 23) - 2).clamp_min(0)
    a = (b.abs() * torch.exp2((127 - s).float())[..., None]).reshape(r, d)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=values.device)
    code = torch.bucketize(a, edges) + 8 * (values < 0)
    codes = (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8)
    held = torch.zeros(r, (d // 32 + 3) // 4 * 4, dtype=torch.uint8, device=values.device)
    held[:, : d // 32] = s.to(torch.uint8)
    return codes, held[:, : d // 32]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    m, k, op = case["m"], case["k"], case["op"]
    state = {"case": case}
    if op == "quantize":
        state["x"] = _activations(m, k, DTYPES[case["dtype"]], gen)
        return state
    w = torch.randn(case["n"], k, generator=gen, device="cuda") * 0.02
    if op == "train":
        state["x"] = _activations(m, k, DTYPES[case["dtype"]], gen).requires_grad_()
        state["w"] = w.to(DTYPES[case["weight"]]).requires_grad_()
        g = torch.randn(m, case["n"], generator=gen, device="cuda") * 1e-3
        g = g * torch.exp2(torch.randint(-6, 3, (m, 1), generator=gen, device="cuda").float())
        state["g"] = g.to(DTYPES[case["dtype"]])
        return state
    state["b"] = _operand(w)
    if op == "product":
        state["a"] = _operand(_activations(m, k, torch.float32, gen))
    else:
        state["x"] = _activations(m, k, DTYPES[case["dtype"]], gen)
    return state


# ----------------------------------------------------------------------------------------- plain forms

def _quantized(x):
    """The values that the MXFP4 form of x stands for, blocks along its last axis, in float32."""
    r, d = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -d % 32)).reshape(r, -1, 32)
    big = x.abs().amax(2, keepdim=True)
    field = ((big.view(torch.int32) >> 23) - 2).clamp_min(0)
    inverse = ((254 - field) << 23).view(torch.float32)
    scale = torch.where(field > 0, field << 23, 1 << 22).view(torch.float32)
    a = x.abs() * inverse
    level = ((a > 0.25) * 0.5 + (a >= 0.75) * 0.5 + (a > 1.25) * 0.5 + (a >= 1.75) * 0.5 + (a > 2.5) * 1.0
             + (a >= 3.5) * 1.0 + (a > 5.0) * 2.0)
    y = torch.sign(x) * level * scale
    y = torch.where(torch.isfinite(big), y, math.nan)
    return y.reshape(r, -1)[:, :d]


def _values(operand):
    """The values that codes and scales stand for, in float32."""
    codes, scales = operand
    table = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    v = table[torch.stack((codes & 15, codes >> 4), 2).long()].reshape(codes.shape[0], -1, 32)
    s = scales.int()
    s = torch.where(s > 0, s << 23, 1 << 22).view(torch.float32)
    return (v * s[..., None]).reshape(codes.shape[0], -1)


def _run_plain(state):
    case = state["case"]
    op = case["op"]
    if op == "quantize":
        x, to = state["x"], torch.bfloat16 if case["dtype"] == "bfloat16" else torch.float32
        rows = _quantized(x).to(to) if case["axes"] != "columns" else None
        columns = _quantized(x.T).to(to) if case["axes"] != "rows" else None
        return {"rows": rows, "columns": columns}
    if op == "product":
        return (_values(state["a"]) @ _values(state["b"]).T).to(DTYPES[case["out"]])
    if op == "linear":
        return (_quantized(state["x"]) @ _values(state["b"]).T).to(DTYPES[case["out"]])
    x, w, g = state["x"].detach(), state["w"].detach(), state["g"]
    return {"y": (_quantized(x) @ _quantized(w).T).to(x.dtype),
            "dx": (_quantized(g) @ _quantized(w.T).T).to(x.dtype),
            "dw": (_quantized(g.T) @ _quantized(x.T).T).to(w.dtype)}


# ------------------------------------------------------------------------------------ the library's calls

def _run_own(state):
    import block_scaled_fp4_w4a16_amd as fp4
    case = state["case"]
    op = case["op"]
    if op == "quantize":
        x, to = state["x"], torch.bfloat16 if case["dtype"] == "bfloat16" else torch.float32
        if case["axes"] == "rows":
            return {"rows": fp4.MXTensor.quantize(x).dequant(to), "columns": None}
        if case["axes"] == "columns":
            return {"rows": None, "columns": fp4.MXTensor.quantize_t(x).dequant(to)}
        rows, columns = fp4.MXTensor.quantize_both(x)
        return {"rows": rows.dequant(to), "columns": columns.dequant(to)}
    if op == "train":
        x, w = state["x"], state["w"]
        y = fp4.mx_linear(x, w)
        dx, dw = torch.autograd.grad(y, (x, w), state["g"])
        return {"y": y.detach(), "dx": dx, "dw": dw}
    b = fp4.MXTensor.from_canonical(*state["b"])
    a = fp4.MXTensor.from_canonical(*state["a"]) if op == "product" else state["x"]
    return b.matmul(a, out_dtype=DTYPES[case["out"]])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------------------------- 64 bits

def _exact_blocks(x):
    """Nearest level by distance: of all levels times the block's power of two, the closest to each value, the even
    code where two are as close."""
    r, d = x.shape
    wide = torch.zeros(r, (d + 31) // 32 * 32, dtype=torch.float64, device=x.device)
    wide[:, :d] = x.double()
    wide = wide.reshape(r, -1, 32)
    _, e = torch.frexp(wide.abs().amax(2))          # largest magnitude = f 2^e, f in [1/2, 1)
    power = torch.exp2((e - 3).clamp_min(-127).double())
    power = torch.where(wide.abs().amax(2) > 0, power, torch.full_like(power, 2.0 ** -127))
    q = wide / power[..., None]
    best = torch.zeros_like(q)
    far = q.abs()
    for code, level in enumerate(LEVELS):
        away = (q.abs() - level).abs()
        nearer = (away < far) | ((away == far) & (code % 2 == 0))
        best = torch.where(nearer, torch.full_like(best, level), best)
        far = torch.minimum(far, away)
    return (torch.copysign(best, q) * power[..., None]).reshape(r, -1)[:, :d]


def _exact_operand(operand):
    codes, scales = operand
    r = codes.shape[0]
    v = torch.empty(r, codes.shape[1] * 2, dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        c = (codes.int() >> (4 * half)) & 15
        mantissa, exponent = (c & 1).double(), (c >> 1) & 3
        size = torch.where(exponent > 0, (1 + mantissa / 2) * torch.exp2(exponent.double() - 1), mantissa / 2)
        v[:, half::2] = torch.where(c >= 8, -size, size)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return {"rows": None if case["axes"] == "columns" else _exact_blocks(state["x"]),
                "columns": None if case["axes"] == "rows" else _exact_blocks(state["x"].T)}
    if op == "train":
        x, w, g = state["x"].detach(), state["w"].detach(), state["g"]
        return {"y": torch.mm(_exact_blocks(x), _exact_blocks(w).T), "dx": torch.mm(_exact_blocks(g), _exact_blocks(w.T).T),
                "dw": torch.mm(_exact_blocks(g.T), _exact_blocks(x.T).T)}
    a = _exact_operand(state["a"]) if op == "product" else _exact_blocks(state["x"])
    return torch.mm(a, _exact_operand(state["b"]).T)
