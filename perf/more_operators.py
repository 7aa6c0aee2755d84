"""MXFP4 products with an epilogue and MXFP4 products of experts: what they compute, in plain torch operations, on real work.

MXFP4 (OCP Microscaling Formats, version 1.0): a block of 32 values along the contracted axis is held as 32 E2M1 codes
(levels 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign) and one E8M0 byte s that stands for 2^(s - 127); s = 255 marks a block with
a NaN. A block's byte is floor(log2(largest magnitude)) - 2 + 127, at least 0; its values are rounded to the nearest
level times the scale, halves to the even code, and what lies past 6 times the scale becomes 6 times the scale. Q(.) stands
for the values of that form, blocks along the last axis.

Four operators, with z = Q(x) W^T + bias and an activation f (none, relu, silu, gelu, or gelu by tanh):
  linear         y = f(z) + residual; x dense, or quantised earlier; W quantised earlier
  train          the same with dense w, and for a gradient g of y: dz = g f'(z), dx = Q(D) Q(w^T)^T, dw = Q(D^T) Q(x^T)^T with D
                 dz in g's type, dbias = the sum of dz over the rows, dresidual = g
  experts        rows sorted by expert, expert e's the rows offsets[e] .. offsets[e + 1] - 1, each with W and bias of its own;
                 rows behind the last expert's are padding and take no product: they are the residual, or zero
  experts train  the gradients of that; blocks of Q(D^T) and Q(x^T) begin anew at each expert's first row

D, what the gradients' products take up, has the type that g has, as a gradient between two layers does. Without an activation
it is g. With one its rounding belongs to the definition: where f' is 1 but for its last bits, the values of g that lie
halfway between two levels would else go up or down by those bits.

`own` False computes these in plain torch operations, True calls the library.
"""
import math

import torch

own = False

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
BYTES = {"float32": 4, "bfloat16": 2, "float16": 2}
ACTIVATIONS = ("none", "relu", "silu", "gelu", "gelu_tanh")


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # decode of one token, gate projection of a 4B-class layer with its activation: the smallest call, all latency
        {"name": "linear token", "op": "linear", "m": 1, "n": 9728, "k": 2560, "x": "bfloat16", "out": "bfloat16",
         "activation": "silu", "bias": "", "residual": ""},
        # verifying eight drafted tokens, down projection added to the residual stream
        {"name": "linear verify", "op": "linear", "m": 9, "n": 2560, "k": 9728, "x": "packed", "out": "float32",
         "activation": "none", "bias": "", "residual": "float32"},
        # a chunk of a prompt with an odd number of tokens, down projection with bias onto the residual stream
        {"name": "linear chunk", "op": "linear", "m": 333, "n": 2560, "k": 9728, "x": "bfloat16", "out": "bfloat16",
         "activation": "none", "bias": "bfloat16", "residual": "bfloat16"},
        # prefill of a long prompt, up projection of a layer with biases
        {"name": "linear prompt", "op": "linear", "m": 8192, "n": 14336, "k": 4096, "x": "bfloat16", "out": "bfloat16",
         "activation": "gelu", "bias": "bfloat16", "residual": ""},
        # a small training step with float32 master weights: key/value projection, ragged tokens
        {"name": "train small", "op": "train", "m": 257, "n": 1024, "k": 2560, "weight": "float32", "activation": "none",
         "bias": True, "residual": True},
        # a large training step: up projection over 8192 tokens
        {"name": "train large", "op": "train", "m": 8192, "n": 9728, "k": 2560, "weight": "bfloat16", "activation": "gelu_tanh",
         "bias": True, "residual": False},
        # decode of one token that goes to eight of 64 experts
        {"name": "experts token", "op": "experts", "tokens": 1, "top": 8, "e": 64, "pad": 0, "n": 1024, "k": 2560, "x": "bfloat16",
         "out": "bfloat16", "activation": "silu", "bias": "", "residual": ""},
        # decode of 64 requests, down projections of the same kind of experts, rows quantised earlier
        {"name": "experts batch", "op": "experts", "tokens": 64, "top": 8, "e": 64, "pad": 0, "n": 2560, "k": 1024, "x": "packed",
         "out": "float32", "activation": "none", "bias": "float32", "residual": ""},
        # a prompt's chunk, padded to a whole number of rows
        {"name": "experts chunk", "op": "experts", "tokens": 1000, "top": 4, "e": 32, "pad": 96, "n": 2560, "k": 2560, "x": "bfloat16",
         "out": "bfloat16", "activation": "gelu_tanh", "bias": "bfloat16", "residual": "bfloat16"},
        # prefill through a few large experts: the largest call
        {"name": "experts prompt", "op": "experts", "tokens": 8192, "top": 2, "e": 8, "pad": 0, "n": 14336, "k": 4096, "x": "bfloat16",
         "out": "bfloat16", "activation": "silu", "bias": "", "residual": ""},
        # a small training step of experts with float32 master weights
        {"name": "experts train small", "op": "experts train", "tokens": 100, "top": 2, "e": 8, "pad": 0, "n": 1024, "k": 2560,
         "weight": "float32", "activation": "none", "bias": True, "residual": False},
        # a large one, with the activation
        {"name": "experts train large", "op": "experts train", "tokens": 4096, "top": 2, "e": 16, "pad": 0, "n": 4096, "k": 2560,
         "weight": "bfloat16", "activation": "silu", "bias": True, "residual": False},
    ]


def _spread(rng, low, high):
    """A whole number whose logarithm is spread evenly."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("linear", "linear", "train", "experts", "experts", "experts train"))
    activation = rng.choice(ACTIVATIONS)
    if op == "linear":
        return {"op": op, "m": _spread(rng, 1, 4096), "n": _spread(rng, 128, 14336), "k": 32 * _spread(rng, 4, 304),
                "x": rng.choice(("packed", "bfloat16", "float16")), "out": rng.choice(("float32", "bfloat16")), "activation": activation,
                "bias": rng.choice(("", "bfloat16", "float32")), "residual": rng.choice(("", "bfloat16", "float32"))}
    # float32 weights go without an activation: what is rounded to 4 bits behind a computed number moves by a whole level
    # where that number's last bit does, which a gradient in 32 bits is too exact to be compared over
    weight = rng.choice(("float32", "bfloat16")) if activation == "none" else "bfloat16"
    if op == "train":
        return {"op": op, "m": _spread(rng, 32, 8192), "n": 8 * _spread(rng, 16, 1216), "k": 8 * _spread(rng, 16, 320), "weight": weight,
                "activation": activation, "bias": rng.random() < 0.5, "residual": rng.random() < 0.5}
    train = op == "experts train"
    e = _spread(rng, 2, 128)
    top = rng.randint(1, min(8, e))
    tokens = _spread(rng, 1, 16384 // top)
    n = _spread(rng, 64, 4096)
    # neither the experts' weights nor the products are more than the largest listed case's
    most = min(100_000_000 // (e * n), 400_000_000_000 // (tokens * top * n)) // 32
    k = 32 * _spread(rng, 2, max(2, min(160, most)))
    case = {"op": op, "tokens": tokens, "top": top, "e": e, "pad": rng.choice((0, 0, rng.randint(1, 64))), "n": n, "k": k}
    if train:
        return case | {"weight": weight, "activation": activation, "bias": rng.random() < 0.5, "residual": rng.random() < 0.5}
    return case | {"x": rng.choice(("packed", "bfloat16", "float16")), "out": rng.choice(("float32", "bfloat16")),
                   "activation": activation, "bias": rng.choice(("", "bfloat16", "float32")),
                   "residual": rng.choice(("", "bfloat16", "float32"))}


def _rows(case):
    return case["m"] if "m" in case else case["tokens"] * case["top"]


def work(case):
    m, n, k = _rows(case), case["n"], case["k"]
    packed = lambda r, d: r * d / 2 + r * d / 32  # noqa: E731
    used, experts = 1, 1
    if "e" in case:  # experts that get a row, where every expert is as likely as another
        experts = case["e"]
        used = experts * (1 - (1 - case["top"] / experts) ** case["tokens"])
    if case["op"].endswith("train"):
        # x, w and g read, y, dx and dw written; the weights' gradient has zeros where an expert has no row
        a, w = 2, BYTES[case["weight"]]
        b = 2 * experts * n * w if case["bias"] else 0
        r = 2 * m * n * a if case["residual"] else 0
        return {"bytes": 2 * m * k * a + (used + experts) * n * k * w + 2 * m * n * a + b + r, "flops": 6 * m * n * k}
    x = packed(m, k) if case["x"] == "packed" else m * k * BYTES[case["x"]]
    b = used * n * BYTES[case["bias"]] if case["bias"] else 0
    r = m * n * BYTES[case["residual"]] if case["residual"] else 0
    return {"bytes": x + used * packed(n, k) + m * n * BYTES[case["out"]] + b + r, "flops": 2 * m * n * k}


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


def _routed(case, gen):
    """Each token's experts by the largest of its router's logits, some experts more popular than others: which token each
    row is, rows sorted by expert, and where each expert's rows begin."""
    tokens, e = case["tokens"], case["e"]
    logits = torch.randn(tokens, e, generator=gen, device="cuda") + 0.7 * torch.randn(e, generator=gen, device="cuda")
    chosen = logits.topk(case["top"], 1).indices.reshape(-1)
    order = torch.argsort(chosen, stable=True)
    counts = torch.bincount(chosen, minlength=e)
    offsets = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return order // case["top"], offsets, int(counts.max())


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    n, k = case["n"], case["k"]
    train, experts = case["op"].endswith("train"), "e" in case
    normal = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    state = {"case": case, "bias": None, "residual": None}
    form = torch.bfloat16 if train else torch.float32 if case["x"] == "packed" else DTYPES[case["x"]]
    if experts:
        which, state["offsets"], state["most"] = _routed(case, gen)
        tokens = _activations(case["tokens"], k, form, gen)
        x = torch.cat((tokens[which], _activations(case["pad"], k, form, gen))) if case["pad"] else tokens[which]
    else:
        x = _activations(case["m"], k, form, gen)
    m, e = x.shape[0], case.get("e", 1)
    w = normal(e * n, k) * 0.02
    out = (e, n) if experts else (n,)
    if train:
        state["x"] = x.requires_grad_()
        state["w"] = w.reshape(*out, k).to(DTYPES[case["weight"]]).requires_grad_()
        g = normal(m, n) * 1e-3
        g = g * torch.exp2(torch.randint(-6, 3, (m, 1), generator=gen, device="cuda").float())
        state["g"] = g.to(torch.bfloat16)
        if case["bias"]:
            state["bias"] = (normal(*out) * 0.1).to(DTYPES[case["weight"]]).requires_grad_()
        if case["residual"]:
            state["residual"] = normal(m, n).to(torch.bfloat16).requires_grad_()
        return state
    state["b"] = _operand(w)
    state["x"] = _operand(x) if case["x"] == "packed" else x
    if case["bias"]:
        state["bias"] = (normal(*out) * 0.1).to(DTYPES[case["bias"]])
    if case["residual"]:
        state["residual"] = normal(m, n).to(DTYPES[case["residual"]])
    return state


# ----------------------------------------------------------------------------------------- plain forms

def _quantized(x):
    """The values that the MXFP4 form of x stands for, blocks along its last axis, in float32."""
    shape = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -shape[-1] % 32)).reshape(math.prod(shape[:-1]), -1, 32)
    big = x.abs().amax(2, keepdim=True)
    field = ((big.view(torch.int32) >> 23) - 2).clamp_min(0)
    inverse = ((254 - field) << 23).view(torch.float32)
    scale = torch.where(field > 0, field << 23, 1 << 22).view(torch.float32)
    a = x.abs() * inverse
    level = ((a > 0.25) * 0.5 + (a >= 0.75) * 0.5 + (a > 1.25) * 0.5 + (a >= 1.75) * 0.5 + (a > 2.5) * 1.0
             + (a >= 3.5) * 1.0 + (a > 5.0) * 2.0)
    y = torch.sign(x) * level * scale
    y = torch.where(torch.isfinite(big), y, math.nan)
    return y.reshape(*shape[:-1], -1)[..., : shape[-1]]


def _values(operand):
    """The values that codes and scales stand for, in float32."""
    codes, scales = operand
    table = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    v = table[torch.stack((codes & 15, codes >> 4), 2).long()].reshape(codes.shape[0], -1, 32)
    s = scales.int()
    s = torch.where(s > 0, s << 23, 1 << 22).view(torch.float32)
    return (v * s[..., None]).reshape(codes.shape[0], -1)


def _activate(name, z):
    if name == "relu":
        return z.clamp_min(0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
    return z


def _slope(name, z):
    """The derivative of the activation at z."""
    if name == "relu":
        return (z > 0).float()
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        s = torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
        return s + z * s * (1 - s) * (2 * math.sqrt(2 / math.pi)) * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _dense_plain(state):
    case = state["case"]
    train = case["op"] == "train"
    x = state["x"].detach() if train else state["x"]
    if train:
        z = _quantized(x) @ _quantized(state["w"].detach()).T
    else:
        z = (_values(x) if case["x"] == "packed" else _quantized(x)) @ _values(state["b"]).T
    bias, residual = state["bias"], state["residual"]
    if bias is not None:
        z = z + bias.detach().float()
    y = _activate(case["activation"], z)
    if residual is not None:
        y = y + residual.detach().float()
    if not train:
        return y.to(DTYPES[case["out"]])
    w, g = state["w"].detach(), state["g"]
    dz = g.float() * _slope(case["activation"], z)
    d = dz.to(g.dtype)
    return {"y": y.to(x.dtype), "dx": (_quantized(d) @ _quantized(w.T).T).to(x.dtype), "dw": (_quantized(d.T) @ _quantized(x.T).T).to(w.dtype),
            "dbias": None if bias is None else dz.double().sum(0).to(bias.dtype), "dresidual": None if residual is None else g.to(residual.dtype)}


def _experts_plain(state):
    """Every expert's rows padded to the most that one has, then products of batches of matrices."""
    case, offsets, most = state["case"], state["offsets"].long(), state["most"]
    train = case["op"] == "experts train"
    e, n, k = case["e"], case["n"], case["k"]
    x = state["x"].detach() if train else state["x"]
    rows = _values(x) if not train and case["x"] == "packed" else _quantized(x)
    m = rows.shape[0]
    every = torch.arange(m, device=rows.device)
    expert = torch.searchsorted(offsets, every, right=True) - 1
    inside = expert < e                       # rows behind the last expert's have none
    expert = expert.clamp_max(e - 1)
    place = torch.where(inside, expert * most + every - offsets[expert], e * most)  # one more place for those
    spread = lambda v: v.new_zeros(e * most + 1, v.shape[1]).index_copy_(0, place, v)[:-1].reshape(e, most, -1)  # noqa: E731
    gather = lambda v: torch.cat((v.reshape(e * most, -1), v.new_zeros(1, v.shape[2])))[place]  # noqa: E731
    w = _quantized(state["w"].detach()) if train else _values(state["b"]).reshape(e, n, k)
    z = gather(torch.bmm(spread(rows), w.transpose(1, 2).contiguous()))
    bias, residual = state["bias"], state["residual"]
    if bias is not None:
        z = z + bias.detach().float()[expert]
    y = torch.where(inside[:, None], _activate(case["activation"], z), 0.0)
    if residual is not None:
        y = y + residual.detach().float()
    if not train:
        return y.to(DTYPES[case["out"]])
    g = state["g"]
    dz = torch.where(inside[:, None], g.float() * _slope(case["activation"], z), 0.0)
    wt = _quantized(state["w"].detach().transpose(1, 2)).transpose(1, 2).contiguous()
    columns = lambda v: _quantized(spread(v.float()).transpose(1, 2))  # noqa: E731
    d = dz.to(g.dtype)
    dx = gather(torch.bmm(spread(_quantized(d)), wt))
    dw = torch.bmm(columns(d), columns(x).transpose(1, 2).contiguous())
    dbias = None if bias is None else spread(dz).double().sum(1).to(bias.dtype)
    return {"y": y.to(x.dtype), "dx": dx.to(x.dtype), "dw": dw.to(state["w"].dtype), "dbias": dbias,
            "dresidual": None if residual is None else g.to(residual.dtype)}


def _run_plain(state):
    return _experts_plain(state) if "e" in state["case"] else _dense_plain(state)


# ------------------------------------------------------------------------------------ the library's calls

def _run_own(state):
    import block_scaled_fp4_w4a16_amd as fp4
    case, x = state["case"], state["x"]
    activation = None if case["activation"] == "none" else case["activation"]
    after = {"bias": state["bias"], "activation": activation, "residual": state["residual"]}
    if case["op"].endswith("train"):
        w = state["w"]
        y = fp4.mx_grouped_linear(x, w, state["offsets"], **after) if "e" in case else fp4.mx_linear(x, w, **after)
        leaves = {"dx": x, "dw": w, "dbias": state["bias"], "dresidual": state["residual"]}
        wanted = [name for name, leaf in leaves.items() if leaf is not None]
        gradients = torch.autograd.grad(y, [leaves[name] for name in wanted], state["g"])
        return {"y": y.detach()} | dict.fromkeys(leaves) | dict(zip(wanted, gradients))
    b = fp4.MXTensor.from_canonical(*state["b"])
    a = fp4.MXTensor.from_canonical(*x) if case["x"] == "packed" else x
    if "e" in case:
        return b.grouped_matmul(a, state["offsets"], out_dtype=DTYPES[case["out"]], **after)
    return b.matmul(a, out_dtype=DTYPES[case["out"]], **after)


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


def _exact_activation(name, z):
    """The activation and its derivative at z: by the normal distribution and by tanh."""
    if name == "relu":
        return torch.relu(z), torch.sign(torch.relu(z))
    if name == "silu":
        half = torch.tanh(z / 2)
        return z / 2 + z / 2 * half, 0.5 + half / 2 + z / 4 * (1 - half * half)
    if name == "gelu":
        share = torch.special.ndtr(z)
        return z * share, share + z * torch.exp(-z * z / 2) / math.sqrt(math.tau)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * z + c * 0.044715 * z ** 3)
        return z / 2 * (1 + t), (1 + t) / 2 + z / 2 * (1 - t * t) * c * (1 + 0.134145 * z ** 2)
    return z, torch.ones_like(z)


def exact(case, seed):
    state = prepare(case, seed)
    train = case["op"].endswith("train")
    n, bias, residual = case["n"], state["bias"], state["residual"]
    if train:
        x, g = state["x"].detach(), state["g"].double()
        weights = state["w"].detach().reshape(-1, n, case["k"])
        weight = lambda i: _exact_blocks(weights[i])  # noqa: E731
        a = _exact_blocks(x)
    else:
        codes, scales = state["b"]
        weight = lambda i: _exact_operand((codes[i * n:(i + 1) * n], scales[i * n:(i + 1) * n]))  # noqa: E731
        a = _exact_operand(state["x"]) if case["x"] == "packed" else _exact_blocks(state["x"])
    m = a.shape[0]
    bounds = state["offsets"].tolist() if "e" in case else [0, m]
    y = torch.zeros(m, n, dtype=torch.float64, device=a.device)
    if train:
        dx = torch.zeros_like(a)
        dw = torch.zeros(weights.shape, dtype=torch.float64, device=a.device)
        db = torch.zeros(len(weights), n, dtype=torch.float64, device=a.device)
    for i, (low, high) in enumerate(zip(bounds, bounds[1:])):
        if low == high:
            continue
        z = torch.mm(a[low:high], weight(i).T)
        if bias is not None:
            z = z + bias.detach().double().reshape(-1, n)[i]
        y[low:high], slope = _exact_activation(case["activation"], z)
        if train:
            dz = g[low:high] * slope
            d = dz.to(state["g"].dtype)
            dx[low:high] = torch.mm(_exact_blocks(d), _exact_blocks(weights[i].T).T)
            dw[i] = torch.mm(_exact_blocks(d.T), _exact_blocks(x[low:high].T).T)
            db[i] = dz.sum(0)
    if residual is not None:
        y = y + residual.detach().double()
    if not train:
        return y
    return {"y": y, "dx": dx, "dw": dw.reshape(state["w"].shape), "dbias": None if bias is None else db.reshape(bias.shape),
            "dresidual": None if residual is None else g}
