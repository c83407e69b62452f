"""Cases, plain forms and 64-bit values of the gated feed-forward block, its backward pass and 8-bit products.

Four operators next to the library's 4-bit products:

* ``gated``       ``h = act(g) * u`` with ``g = x . Wg^T`` and ``u = x . Wu^T``: the first half of a dense
  feed-forward block over 4-bit weights, or over 8-bit weights with the tokens quantized to 8 bits in the
  same pass; on request the products ``g | u`` that its backward pass needs come with it.
* ``gated_grad``  the gradients of ``g | u`` from that of ``h``: ``dg = dh * u * act'(g)``, ``du = dh * act(g)``.
* ``grad``        the input gradient of a product with frozen 4-bit weights: ``dx = d . W_hat``.
* ``int8``        ``y = s_t * s_n * sum_k q[t, k] * q[n, k]``: tokens quantized to 8 bits by rows (the scale is
  the fp32 value of ``max|x| / 127``, the code the integer nearest to ``x / scale``, ties to even), times
  8-bit weights with a scale for each channel.

``run`` computes them with elementary torch operations in fp32, or, where ``own`` is true, through
the library.  ``exact`` computes them in fp64 from the definitions.
"""
import math

import torch

own = False

NF4 = (-1.0, -0.6961928009986877, -0.5250729322433472, -0.39491742849349976, -0.2844413220882416,
       -0.18477340042591095, -0.09104997664690018, 0.0, 0.07958031445741653, 0.16093014180660248,
       0.24611225724220276, 0.3379151225090027, 0.4407097399234772, 0.5626168847084045,
       0.722956657409668, 1.0)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
GROUP = {"nf4": 64, "fp4": 64, "int4": 128, "int4a": 128, "mxfp4": 32}
SCALE_BYTES = {"nf4": 4, "fp4": 4, "int4": 2, "int4a": 4, "mxfp4": 1}
FORMATS = tuple(f"{w}_{x}" for w in ("nf4", "int4", "fp4", "int4a", "mxfp4") for x in ("f16", "bf16"))
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
MOST_WEIGHTS = 2 * 11008 * 4096          # of one drawn gated block
MOST_FLOPS = 2 * 4096 * 8192 * 8192      # of any drawn case


def listed():
    return [
        # decode, one sequence: a layer's gate and up products, the weights' bytes count
        {"name": "gated 1 token nf4", "op": "gated", "fmt": "nf4_bf16", "tokens": 1, "hidden": 1536,
         "inter": 8960, "act": "silu", "save": False},
        # a decode batch or drafted tokens, an odd number of them
        {"name": "gated 23 tokens int4", "op": "gated", "fmt": "int4_f16", "tokens": 23, "hidden": 2048,
         "inter": 8192, "act": "silu", "save": False},
        # a training step's forward pass over a ragged batch: g | u kept for the backward pass
        {"name": "gated 1000 tokens mxfp4", "op": "gated", "fmt": "mxfp4_bf16", "tokens": 1000,
         "hidden": 1536, "inter": 8960, "act": "gelu_tanh", "save": True},
        # a long prompt through 8-bit weights: the matrix cores count
        {"name": "gated 2048 tokens int8", "op": "gated", "fmt": "int8_bf16", "tokens": 2048,
         "hidden": 4096, "inter": 11008, "act": "silu", "save": False},
        # a few tokens: latency alone
        {"name": "gated_grad 3x8960", "op": "gated_grad", "dtype": "f16", "tokens": 3, "inter": 8960,
         "act": "silu"},
        # a training batch: five streams through memory
        {"name": "gated_grad 4096x8960", "op": "gated_grad", "dtype": "bf16", "tokens": 4096,
         "inter": 8960, "act": "gelu_tanh"},
        # a short sequence back through a down projection
        {"name": "grad 16 tokens nf4", "op": "grad", "fmt": "nf4_bf16", "tokens": 16, "n": 1536,
         "k": 8960},
        # a micro-batch of odd length back through a projection of odd height
        {"name": "grad 333 tokens fp4", "op": "grad", "fmt": "fp4_bf16", "tokens": 333, "n": 4001,
         "k": 2048},
        # a training batch back through gate and up
        {"name": "grad 2048 tokens int4", "op": "grad", "fmt": "int4_f16", "tokens": 2048, "n": 17920,
         "k": 1536},
        # decode, one token, 8-bit weights
        {"name": "int8 1 token", "op": "int8", "dtype": "f16", "out": "f32", "tokens": 1, "n": 8960,
         "k": 1536},
        # a batch of 77 rows, long rows of weights
        {"name": "int8 77 tokens", "op": "int8", "dtype": "bf16", "out": "bf16", "tokens": 77,
         "n": 1536, "k": 8960},
        # a prompt: as large as products get
        {"name": "int8 4096 tokens", "op": "int8", "dtype": "bf16", "out": "bf16", "tokens": 4096,
         "n": 8192, "k": 8192},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("gated", "gated", "gated_grad", "grad", "grad", "int8", "int8"))
    act = rng.choice(("silu", "gelu_tanh"))
    if op == "gated_grad":
        return {"op": op, "dtype": rng.choice(("f16", "bf16")), "tokens": _log(rng, 1, 4096),
                "inter": _log(rng, 1, 14336), "act": act}
    while True:
        if op == "gated":
            fmt = rng.choice(FORMATS + ("int8_f16", "int8_bf16"))
            step = max(64, GROUP.get(fmt.split("_")[0], 64))
            case = {"op": op, "fmt": fmt, "tokens": _log(rng, 1, 2048), "hidden": step * _log(rng, 1, 8192 // step),
                    "inter": _log(rng, 1, 14336), "act": act, "save": rng.random() < 0.4}
            size = 2 * case["hidden"] * case["inter"]
        elif op == "grad":
            fmt = rng.choice(FORMATS)
            step = max(64, GROUP[fmt.split("_")[0]])
            case = {"op": op, "fmt": fmt, "tokens": _log(rng, 1, 2048), "n": _log(rng, 1, 18000),
                    "k": step * _log(rng, 1, 8960 // step)}
            size = case["n"] * case["k"]
        else:
            case = {"op": op, "dtype": rng.choice(("f16", "bf16")), "out": rng.choice(("f32", "f16", "bf16")),
                    "tokens": _log(rng, 1, 4096), "n": _log(rng, 1, 28672), "k": 64 * _log(rng, 1, 224)}
            size = case["n"] * case["k"]
        if size <= MOST_WEIGHTS and work(case)["flops"] <= MOST_FLOPS:
            return case


def _tables(device):
    return (torch.tensor(NF4, dtype=torch.float32, device=device),
            torch.tensor(E2M1, dtype=torch.float32, device=device))


def _quantize(weight, w):
    """fp32 [rows, K] -> packed nibbles and scales of the encoding, as the quantizers store them."""
    rows, k = w.shape
    g = GROUP[weight]
    b = w.view(rows, k // g, g)
    top = b.abs().amax(2)
    if weight == "nf4":
        nf4 = _tables(w.device)[0]
        scales = top
        q = torch.bucketize(b / top.unsqueeze(2), (nf4[1:] + nf4[:-1]) / 2)
    elif weight == "int4":
        s = (top / 7).bfloat16()
        scales = s.view(torch.int16)
        q = (b / s.float().unsqueeze(2)).round().clamp(-8, 7) + 8
    elif weight == "int4a":
        lo, hi = b.amin(2).clamp(max=0), b.amax(2).clamp(min=0)
        s = ((hi - lo) / 15).bfloat16()
        z = (-lo / s.float()).round().clamp(0, 15)
        scales = (s.view(torch.int16).int() & 0xFFFF) | (z.int() << 16)
        q = (b / s.float().unsqueeze(2) + z.unsqueeze(2)).round().clamp(0, 15)
    else:  # E2M1
        edges = torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), device=w.device)
        if weight == "fp4":
            scales = s = top / 6
        else:
            e = torch.frexp(top)[1] - 3  # floor(log2(top)) - 2
            scales = (e + 127).clamp(0, 254).to(torch.uint8)
            s = torch.ldexp(torch.ones_like(top), e)
        r = b / s.unsqueeze(2)
        q = torch.bucketize(r.abs(), edges) + 8 * (r < 0)
    q = q.to(torch.uint8).view(rows, k // 2, 2)
    return (q[..., 0] << 4) | q[..., 1], scales


def _weights(weight, n, k, gen, device):
    """Normal weights (sigma 0.02) of shape [n, k] in the encoding; int8: codes and channel scales."""
    w = torch.randn(n, k, generator=gen, device=device) * 0.02
    if weight != "int8":
        return _quantize(weight, w)
    scales = w.abs().amax(1) / 127
    return (w / scales.unsqueeze(1)).round().clamp(-127, 127).to(torch.int8), scales


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device).manual_seed(seed)
    t = case["tokens"]
    if case["op"] == "gated_grad":
        dtype = TYPES[case["dtype"]]
        products = torch.randn(t, 2 * case["inter"], generator=gen, device=device) * 0.8
        dh = torch.randn(t, case["inter"], generator=gen, device=device) * 0.1
        return {"case": case, "dh": dh.to(dtype), "products": products.to(dtype)}
    if case["op"] == "int8":
        weight, xtype, n, k = "int8", case["dtype"], case["n"], case["k"]
    elif case["op"] == "grad":
        (weight, xtype), n, k = case["fmt"].split("_"), case["n"], case["k"]
    else:
        (weight, xtype), n, k = case["fmt"].split("_"), 2 * case["inter"], case["hidden"]
    w, scales = _weights(weight, n, k, gen, device)
    if case["op"] == "grad":
        x = torch.randn(t, n, generator=gen, device=device) * 0.1
    else:
        x = torch.randn(t, k, generator=gen, device=device)
    return {"case": case, "x": x.to(TYPES[xtype]), "w": w, "scales": scales}


def _decode(weight, packed, scales):
    """The fp32 weights that packed nibbles and scales stand for."""
    nf4, e2m1 = _tables(packed.device)
    q = torch.stack((packed >> 4, packed & 15), dim=-1).flatten(-2).int()
    if weight == "nf4":
        w, s = nf4[q], scales
    elif weight == "fp4":
        w, s = e2m1[q], scales
    elif weight == "mxfp4":
        w, s = e2m1[q], torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.int() - 127)
    elif weight == "int4":
        w, s = (q - 8).float(), scales.view(torch.bfloat16).float()
    else:
        s = (scales << 16).view(torch.float32)
        w = (q - ((scales >> 16) & 15).repeat_interleave(128, dim=-1)).float()
    return w * s.repeat_interleave(GROUP[weight], dim=-1)


def _int8(x, w, scales):
    """Tokens to 8 bits by rows, then the product.  The scale (a division by a number is a product with its
    reciprocal here, one step off in 32 bits) and the quotients are taken in 64 bits: a quotient next to
    the middle between two codes may round to that middle in 32."""
    s = (x.double().abs().amax(1) / 127).float()
    q = (x.double() / s.double().unsqueeze(1)).round().clamp(-127, 127)
    q = torch.where(s.unsqueeze(1) > 0, q, torch.zeros_like(q)).float()
    return (q @ w.float().t()) * s.unsqueeze(1) * scales


def _act(act, g):
    """act(g) and its derivative."""
    if act == "silu":
        p = 1 / (1 + (-g).exp())
        return g * p, p * (1 + g * (1 - p))
    a, b = math.sqrt(2 / math.pi), 0.044715
    th = torch.tanh(a * (g + b * g * g * g))
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * a * (1 + 3 * b * g * g)


def _run_own(state):
    import bit_weight_only_w4_amd as w4

    case = state["case"]
    if case["op"] == "gated_grad":
        return {"d_products": w4.gated_grad(state["dh"], state["products"], case["act"])}
    x, w, scales = state["x"], state["w"], state["scales"]
    if case["op"] == "grad":
        return {"dx": w4.gemm_grad(x, w, scales, case["fmt"])}
    if case["op"] == "int8":
        codes, s = w4.quantize_int8(x)
        return {"y": w4.gemm_int8(codes, s, w, scales, TYPES[case["out"]])}
    if case["fmt"].startswith("int8"):
        codes, s = w4.quantize_int8(x)
        out = w4.gated_int8(codes, s, w, scales, case["act"], x.dtype, save=case["save"])
    else:
        out = w4.gated(x, w, scales, case["fmt"], case["act"], save=case["save"])
    return {"h": out[0], "products": out[1]} if case["save"] else {"h": out}


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    if case["op"] == "gated_grad":
        g, u = state["products"].float().chunk(2, dim=1)
        dh = state["dh"].float()
        y, dy = _act(case["act"], g)
        return {"d_products": torch.cat((dh * u * dy, dh * y), dim=1).to(state["dh"].dtype)}
    x, w, scales = state["x"], state["w"], state["scales"]
    if case["op"] == "int8":
        return {"y": _int8(x, w, scales).to(TYPES[case["out"]])}
    weight = case["fmt"].split("_")[0]
    if case["op"] == "grad":
        return {"dx": (x.float() @ _decode(weight, w, scales)).to(x.dtype)}
    if weight == "int8":
        both = _int8(x, w, scales)
    else:
        both = x.float() @ _decode(weight, w, scales).t()
    g, u = both.chunk(2, dim=1)
    h = (_act(case["act"], g)[0] * u).to(x.dtype)
    return {"h": h, "products": both.to(x.dtype)} if case["save"] else {"h": h}


def _matrix_bytes(weight, n, k):
    if weight == "int8":
        return n * k + 4 * n
    return n * k // 2 + n * (k // GROUP[weight]) * SCALE_BYTES[weight]


def work(case):
    t = case["tokens"]
    if case["op"] == "gated_grad":
        return {"bytes": 10 * t * case["inter"], "flops": 20 * t * case["inter"]}
    if case["op"] == "int8":
        n, k = case["n"], case["k"]
        return {"bytes": _matrix_bytes("int8", n, k) + 2 * t * k + t * n * (4 if case["out"] == "f32" else 2),
                "flops": 2 * t * n * k}
    weight = case["fmt"].split("_")[0]
    if case["op"] == "grad":
        n, k = case["n"], case["k"]
        return {"bytes": _matrix_bytes(weight, n, k) + 2 * t * (n + k), "flops": 2 * t * n * k}
    h, i = case["hidden"], case["inter"]
    return {"bytes": _matrix_bytes(weight, 2 * i, h) + 2 * t * (h + (3 * i if case["save"] else i)),
            "flops": 4 * t * h * i}


def _exact_matrix(weight, packed, scales):
    """fp64 weights of one matrix [N, K], element 2i in the high nibble of byte i."""
    if weight == "int8":
        return packed.double() * scales.double().unsqueeze(1)
    n, half = packed.shape
    q = torch.empty(n, 2 * half, dtype=torch.int64, device=packed.device)
    q[:, 0::2] = packed.long() // 16
    q[:, 1::2] = packed.long() % 16
    q = q.view(n, -1, GROUP[weight])
    if weight in ("int4", "int4a"):
        bits = scales.int() & 0xFFFF
        sign, exponent, fraction = bits >> 15, (bits >> 7) & 255, bits & 127
        s = (1 - 2 * sign) * (1 + fraction.double() / 128) * torch.pow(2.0, exponent.double() - 127)
        s = torch.where(exponent == 0, torch.zeros_like(s), s)
        zero = 8 if weight == "int4" else ((scales.int() >> 16) & 15).unsqueeze(2)
        w = (q - zero).double()
    else:
        table = torch.tensor(NF4 if weight == "nf4" else E2M1, dtype=torch.float64, device=packed.device)
        w = table[q]
        s = torch.pow(2.0, scales.double() - 127) if weight == "mxfp4" else scales.double()
    return (w * s.unsqueeze(2)).view(n, -1)


def _exact_tokens(x):
    """fp64 values of the tokens' 8-bit codes: q * s, s an fp32 number."""
    x = x.double()
    s = (x.abs().max(dim=1, keepdim=True).values / 127).float().double()
    return torch.where(s > 0, torch.round(x / s).clamp(-127, 127), 0.0) * s


def _exact_act(act, g):
    """act(g) and act'(g) from the logistic function: gelu's tanh form is g * sigmoid(2 v(g))."""
    if act == "silu":
        v, dv = g, torch.ones_like(g)
    else:
        c = 2 * math.sqrt(2 / math.pi)
        v, dv = c * (g + 0.044715 * g.pow(3)), c * (1 + 3 * 0.044715 * g.square())
    p = torch.sigmoid(v)
    return g * p, p + g * dv * p * torch.sigmoid(-v)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gated_grad":
        inter = case["inter"]
        g, u, dh = s["products"][:, :inter].double(), s["products"][:, inter:].double(), s["dh"].double()
        y, dy = _exact_act(case["act"], g)
        out = torch.empty_like(s["products"], dtype=torch.float64)
        out[:, :inter] = dh * u * dy
        out[:, inter:] = dh * y
        return {"d_products": out}
    weight = "int8" if case["op"] == "int8" else case["fmt"].split("_")[0]
    x = _exact_tokens(s["x"]) if weight == "int8" else s["x"].double()
    n, k = s["scales"].shape[0], s["w"].shape[1] * (1 if weight == "int8" else 2)
    if case["op"] == "grad":
        dx = torch.zeros(case["tokens"], k, dtype=torch.float64, device=x.device)
        for r in range(0, n, 8192):
            dx += x[:, r:r + 8192] @ _exact_matrix(weight, s["w"][r:r + 8192], s["scales"][r:r + 8192])
        return {"dx": dx}
    both = torch.empty(case["tokens"], n, dtype=torch.float64, device=x.device)
    for r in range(0, n, 8192):
        both[:, r:r + 8192] = x @ _exact_matrix(weight, s["w"][r:r + 8192], s["scales"][r:r + 8192]).t()
    if case["op"] == "int8":
        return {"y": both}
    inter = case["inter"]
    h = _exact_act(case["act"], both[:, :inter])[0] * both[:, inter:]
    return {"h": h, "products": both} if case["save"] else {"h": h}
