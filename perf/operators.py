"""Cases, plain forms and 64-bit values of the mixture-of-experts and MXFP4 operators.

Three operators next to the library's 4-bit products:

* ``route``  the router's choice: for each token the ``top_k`` largest of its expert logits (ties to
  the lowest expert, a NaN logit never chosen) and their softmax weights.
* ``moe``    the expert layer: ``y[t] = sum_j w[t, j] * Down_e(silu(Gate_e x[t]) * (Up_e x[t]))``
  with ``e = ids[t, j]`` and every expert matrix held in 4 bits.
* ``mx``     ``y = x . W_hat^T`` for MXFP4 weights: E2M1 codes, one power-of-two scale byte for each
  32 weights of a row.

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
FORMATS = tuple(f"{w}_{x}" for w in ("nf4", "int4", "fp4", "int4a", "mxfp4") for x in ("f16", "bf16"))


def listed():
    return [
        # one token's router: the smallest call, latency alone
        {"name": "route 1x64", "op": "route", "tokens": 1, "experts": 64, "top_k": 8, "dtype": "f32",
         "renorm": True},
        # a prompt's worth of tokens over many experts, logits as a 16-bit product leaves them
        {"name": "route 4096x256", "op": "route", "tokens": 4096, "experts": 256, "top_k": 8,
         "dtype": "bf16", "renorm": False},
        # a small model's layer for one token: little to read, launches count
        {"name": "moe 1 token, 8 small experts", "op": "moe", "fmt": "nf4_f16", "tokens": 1,
         "experts": 8, "top_k": 2, "hidden": 512, "inter": 256, "absent": False},
        # decode, one sequence
        {"name": "moe 1 token int4", "op": "moe", "fmt": "int4_bf16", "tokens": 1, "experts": 64,
         "top_k": 8, "hidden": 2048, "inter": 1024, "absent": False},
        # decode or drafted tokens, a few rows, the experts of this rank only (the rest absent)
        {"name": "moe 5 tokens nf4, absent", "op": "moe", "fmt": "nf4_bf16", "tokens": 5,
         "experts": 60, "top_k": 4, "hidden": 1536, "inter": 1408, "absent": True},
        # a decode batch over many experts: nearly every expert is read
        {"name": "moe 32 tokens mxfp4", "op": "moe", "fmt": "mxfp4_bf16", "tokens": 32,
         "experts": 128, "top_k": 8, "hidden": 2048, "inter": 768, "absent": False},
        # a large decode batch over few experts with zero points, odd widths
        {"name": "moe 150 tokens int4a", "op": "moe", "fmt": "int4a_f16", "tokens": 150,
         "experts": 16, "top_k": 2, "hidden": 1920, "inter": 2432, "absent": False},
        # a short prompt: dozens of tokens for each expert
        {"name": "moe 512 tokens fp4", "op": "moe", "fmt": "fp4_f16", "tokens": 512, "experts": 64,
         "top_k": 6, "hidden": 1536, "inter": 1408, "absent": False},
        # one MXFP4 product of a decode step
        {"name": "mx 8960x1536 b1", "op": "mx", "fmt": "mxfp4_f16", "n": 8960, "k": 1536, "batch": 1},
        # the output projection over the vocabulary, one token
        {"name": "mx 151936x1536 b1", "op": "mx", "fmt": "mxfp4_bf16", "n": 151936, "k": 1536,
         "batch": 1},
        # long rows, an odd number of drafted tokens
        {"name": "mx 1536x8960 b5", "op": "mx", "fmt": "mxfp4_bf16", "n": 1536, "k": 8960, "batch": 5},
        # a decode batch on a large matrix
        {"name": "mx 28672x8192 b32", "op": "mx", "fmt": "mxfp4_f16", "n": 28672, "k": 8192,
         "batch": 32},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("route", "moe", "moe", "mx"))
    if op == "route":
        experts = _log(rng, 2, 256)
        return {"op": op, "tokens": _log(rng, 1, 4096), "experts": experts,
                "top_k": rng.randint(1, min(8, experts)),
                "dtype": rng.choice(("f32", "f16", "bf16")), "renorm": rng.random() < 0.5}
    if op == "moe":
        fmt = rng.choice(FORMATS)
        step = max(64, GROUP[fmt.split("_")[0]])
        while True:
            experts = _log(rng, 2, 128)
            case = {"op": op, "fmt": fmt, "tokens": _log(rng, 1, 512), "experts": experts,
                    "top_k": rng.randint(1, min(8, experts)),
                    "hidden": step * _log(rng, 256 // step, 4096 // step),
                    "inter": step * _log(rng, 128 // step, 2560 // step),
                    "absent": rng.random() < 0.3}
            size = experts * case["hidden"] * case["inter"]
            if size <= 64 * 1536 * 1408 and work(case)["flops"] <= 512 * 6 * 6 * 1536 * 1408:
                return case
    while True:
        case = {"op": op, "fmt": rng.choice(("mxfp4_f16", "mxfp4_bf16")), "n": _log(rng, 1, 160000),
                "k": 64 * _log(rng, 1, 448), "batch": _log(rng, 1, 256)}
        size = case["n"] * case["k"]
        if size <= 28672 * 8192 and size * case["batch"] <= 28672 * 8192 * 32:
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


def _weights(weight, shape, gen, device):
    """Normal weights (sigma 0.02) of shape [..., N, K] in the encoding."""
    rows = math.prod(shape[:-1])
    packed, scales = _quantize(weight, torch.randn(rows, shape[-1], generator=gen, device=device) * 0.02)
    return packed.view(*shape[:-1], -1), scales.view(*shape[:-1], -1)


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device).manual_seed(seed)
    if case["op"] == "route":
        dtype = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[case["dtype"]]
        logits = torch.randn(case["tokens"], case["experts"], generator=gen, device=device) * 1.5
        return {"case": case, "logits": logits.to(dtype)}
    weight, xtype = case["fmt"].split("_")
    dtype = torch.float16 if xtype == "f16" else torch.bfloat16
    if case["op"] == "mx":
        packed, scales = _weights(weight, (case["n"], case["k"]), gen, device)
        x = torch.randn(case["batch"], case["k"], generator=gen, device=device).to(dtype)
        return {"case": case, "x": x, "packed": packed, "scales": scales}
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    h, i = case["hidden"], case["inter"]
    gate_up, gate_up_scales = _weights(weight, (e, 2 * i, h), gen, device)
    down, down_scales = _weights(weight, (e, h, i), gen, device)
    x = torch.randn(t, h, generator=gen, device=device).to(dtype)
    top = torch.randn(t, e, generator=gen, device=device).topk(k, dim=1)
    ids, weights = top.indices.int(), top.values.softmax(1)
    if case["absent"]:
        ids = torch.where(torch.rand(t, k, generator=gen, device=device) < 0.25, -1, ids)
    return {"case": case, "x": x, "ids": ids, "weights": weights, "gate_up": gate_up,
            "gate_up_scales": gate_up_scales, "down": down, "down_scales": down_scales}


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


def _route(logits, top_k, renorm):
    """Descending stable order (ties to the lowest expert), softmax over all or over the chosen."""
    v = logits.float()
    ids = v.sort(dim=1, descending=True, stable=True).indices[:, :top_k]
    e = (v - v.amax(1, keepdim=True)).exp()
    chosen = e.gather(1, ids)
    return ids.int(), chosen / (chosen if renorm else e).sum(1, keepdim=True)


def _moe(weight, s):
    """Every expert on every token, then the routed sum: h is scattered to [T, E, I] with its
    routing weight, and one product over (E, I) adds a token's experts."""
    t, hidden = s["x"].shape
    experts, inter = s["gate_up"].shape[0], s["gate_up"].shape[1] // 2
    gate_up = _decode(weight, s["gate_up"], s["gate_up_scales"]).view(-1, hidden)
    both = (s["x"].float() @ gate_up.t()).view(t, experts, 2, inter)
    del gate_up
    gate, up = both[:, :, 0], both[:, :, 1]
    h = gate * (1 / (1 + (-gate).exp())) * up
    ids = s["ids"].long()
    here = (ids >= 0) & (ids < experts)
    share = torch.zeros(t, experts, device=ids.device)
    share.scatter_add_(1, ids.clamp(0, experts - 1), s["weights"] * here)
    down = _decode(weight, s["down"], s["down_scales"])
    return (h * share.unsqueeze(2)).view(t, -1) @ down.transpose(1, 2).reshape(-1, hidden)


def run(state):
    case = state["case"]
    if own:
        import bit_weight_only_w4_amd as w4

        if case["op"] == "route":
            ids, weights = w4.moe_route(state["logits"], case["top_k"], renormalize=case["renorm"])
            return {"ids": ids, "weights": weights}
        if case["op"] == "moe":
            return {"y": w4.moe(state["x"], state["ids"], state["weights"], state["gate_up"],
                                state["gate_up_scales"], state["down"], state["down_scales"],
                                case["fmt"])}
        return {"y": w4.gemm_smallbatch(state["x"], state["packed"], state["scales"], case["fmt"])}
    if case["op"] == "route":
        ids, weights = _route(state["logits"], case["top_k"], case["renorm"])
        return {"ids": ids, "weights": weights}
    weight = case["fmt"].split("_")[0]
    if case["op"] == "moe":
        return {"y": _moe(weight, state)}
    return {"y": state["x"].float() @ _decode(weight, state["packed"], state["scales"]).t()}


def _matrix_bytes(weight, n, k):
    return n * k // 2 + n * (k // GROUP[weight]) * {"nf4": 4, "fp4": 4, "int4": 2, "int4a": 4, "mxfp4": 1}[weight]


def work(case):
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        return {"bytes": t * (e * (4 if case["dtype"] == "f32" else 2) + 8 * k), "flops": 4 * t * e}
    weight = case["fmt"].split("_")[0]
    if case["op"] == "mx":
        n, k, b = case["n"], case["k"], case["batch"]
        return {"bytes": _matrix_bytes(weight, n, k) + 2 * b * k + 4 * b * n, "flops": 2 * b * n * k}
    t, e, k, h, i = (case[v] for v in ("tokens", "experts", "top_k", "hidden", "inter"))
    live = 0.75 if case["absent"] else 1.0
    read = e * (1 - (1 - live * k / e) ** t)  # experts that some token is routed to, on average
    return {"bytes": read * (_matrix_bytes(weight, 2 * i, h) + _matrix_bytes(weight, h, i))
            + t * (6 * h + 8 * k), "flops": live * t * k * 6 * h * i}


def _exact_matrix(weight, packed, scales):
    """fp64 weights of one matrix [N, K], element 2i in the high nibble of byte i."""
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


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        v = s["logits"].double()
        first = torch.arange(case["experts"], device=v.device)
        # rank by (value descending, index ascending)
        before = (v.unsqueeze(1) > v.unsqueeze(2)) | ((v.unsqueeze(1) == v.unsqueeze(2))
                                                      & (first.view(1, 1, -1) < first.view(1, -1, 1)))
        rank = before.sum(2)
        ids = rank.argsort(dim=1)[:, :case["top_k"]]
        value = v.gather(1, ids)
        whole = value if case["renorm"] else v
        return {"ids": ids.int(), "weights": (value - torch.logsumexp(whole, 1, keepdim=True)).exp()}
    weight = case["fmt"].split("_")[0]
    if case["op"] == "mx":
        y = torch.empty(case["batch"], case["n"], dtype=torch.float64, device=s["x"].device)
        for r in range(0, case["n"], 16384):
            y[:, r:r + 16384] = s["x"].double() @ _exact_matrix(
                weight, s["packed"][r:r + 16384], s["scales"][r:r + 16384]).t()
        return {"y": y}
    x = s["x"].double()
    y = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device=x.device)
    for e in range(case["experts"]):
        token, slot = (s["ids"] == e).nonzero(as_tuple=True)
        if token.numel() == 0:
            continue
        both = x[token] @ _exact_matrix(weight, s["gate_up"][e], s["gate_up_scales"][e]).t()
        gate, up = both.chunk(2, dim=1)
        out = (gate * torch.sigmoid(gate) * up) @ _exact_matrix(weight, s["down"][e], s["down_scales"][e]).t()
        y.index_add_(0, token, out * s["weights"][token, slot].double().unsqueeze(1))
    return {"y": y}
