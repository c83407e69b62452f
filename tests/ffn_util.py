"""Seeded inputs, plain fp64 forms and error bounds of the gated block, its gradients and the 8-bit products.

Bounds, each rounding at its largest:

* a product over K: K additions in fp32, 2^-23 of the terms' magnitudes each (the matrix cores may cut where others
  round), and a weight rounded to the fp16 or bf16 operand: 2^-11 or 2^-8 of its terms; operands of a common exponent
  a row lose at most 2^-39 of that row's largest;
* |act'| <= 1.13 for both activations; exp's argument, exp, the reciprocal and the products: (2 |g| + 16) 2^-23 of
  the value;
* p = 1 / (1 + exp(-v)) below 2^-126, the smallest normal number, may come out as 0: the reciprocal of the hardware
  gives no subnormal numbers, and 1 + exp(-v) is then 2^126 or more.  What holds it as a factor is off by at most
  2^-126 times the other factors (a gate of -10.06: p = 2^-127.3, a gradient of 1e-36, reads 0);
* the result is rounded to its type once: half a step, eps / 2 of it, and half the smallest subnormal.
"""
import math

import numpy as np
import torch

import oracle
import synth_inputs

FMTS = [f"{w}_{x}" for w in ("nf4", "int4", "fp4", "int4a", "mxfp4") for x in ("f16", "bf16")]
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
LEAST = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}
LIPSCHITZ = 1.13


def group(fmt):
    return 128 if fmt.startswith("int4") else 64


def device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm GPU"
    return torch.device("cuda:0")


def weights(fmt, n, k, seed, sigma=0.05):
    """Packed weights, scales (as the binding takes them) and fp64 values of an [n, k] matrix, on the CPU."""
    w = fmt.split("_")[0]
    q = {"nf4": oracle.quantize_nf4, "int4": oracle.quantize_int4, "fp4": oracle.quantize_fp4,
         "int4a": oracle.quantize_int4_asym, "mxfp4": oracle.quantize_mxfp4}[w]
    p, s = q(synth_inputs.weights(n, k, sigma=sigma, seed=seed))
    return as_operands(fmt, p, s)


def as_operands(fmt, p, s):
    hat = oracle.dequant(fmt.split("_")[0], p, s)
    s = s.view(np.int16) if s.dtype == np.uint16 else s.view(np.int32) if s.dtype == np.uint32 else s
    return torch.from_numpy(p), torch.from_numpy(np.ascontiguousarray(s)), torch.from_numpy(hat)


def normal(shape, dtype, seed, sigma=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen, dtype=torch.float64) * sigma).to(dtype)


def act(name, g):
    """act(g) and act'(g) in fp64."""
    if name == "silu":
        v, dv = g, torch.ones_like(g)
    else:
        c = 2 * math.sqrt(2 / math.pi)
        v, dv = c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g ** 2)
    p = torch.sigmoid(v)
    return g * p, p + g * dv * p * torch.sigmoid(-v)


def rounded(value, dtype):
    """Largest rounding error of `value` in dtype."""
    return value.abs() * HALF[dtype] + LEAST[dtype]


def product_bound(x, w, operand):
    """(x . w^T, bound) in fp64; operand: the largest relative rounding of a weight before the product."""
    k = x.shape[1]
    terms = x.abs() @ w.abs().t()
    edge = 2.0 ** -39 * (x.abs().amax(1, keepdim=True) * w.abs().sum(1) + x.abs().sum(1, keepdim=True) * w.abs().amax(1))
    return x @ w.t(), terms * (k * 2.0 ** -23 + operand) + edge + 2.0 ** -140


def block_bound(both, d, name, dtype):
    """(h, its bound, bound of g | u as stored) from the products and their bounds."""
    inter = both.shape[1] // 2
    g, u, dg, du = both[:, :inter], both[:, inter:], d[:, :inter], d[:, inter:]
    a, _ = act(name, g)
    h = a * u
    da = LIPSCHITZ * dg + (2 * g.abs() + 16) * 2.0 ** -23 * (a.abs() + dg) + 2.0 ** -126 * g.abs()
    e = da * (u.abs() + du) + a.abs() * du
    return h, e + rounded(h.abs() + e, dtype), d + rounded(both.abs() + d, dtype)


def gated_bound(x, w, name, dtype):
    both, d = product_bound(x.double(), w, 2.0 ** -11)
    h, eh, ep = block_bound(both, d, name, dtype)
    return h, eh, both, ep


def gated_grad_bound(dh, products, name):
    dtype = dh.dtype
    inter = dh.shape[1]
    g, u, f = products[:, :inter].double(), products[:, inter:].double(), dh.double()
    a, slope = act(name, g)
    # the slope's terms: p (at most 1) and g v' p (1 - p), each off by (2 |v(g)| + 16) 2^-23 of itself
    c = g.clamp(-30, 30)
    v = c if name == "silu" else 1.6 * (c + 0.044715 * c ** 3)
    dv = torch.ones_like(g) if name == "silu" else 1.6 * (1 + 0.134145 * c ** 2)
    p = torch.sigmoid(v)
    rel = (2 * v.abs() + 16) * 2.0 ** -23
    es = rel * (p + g.abs() * dv * p * torch.sigmoid(-v)) + 2.0 ** -23 * g.abs() * dv * p
    es = es + 2.0 ** -126 * (1 + g.abs() * dv)
    ref = torch.cat((f * u * slope, f * a), 1)
    e = torch.cat((f.abs() * u.abs() * es, f.abs() * (a.abs() * rel + 2.0 ** -126 * g.abs())), 1) + 2.0 ** -120
    return ref, e + rounded(ref.abs() + e, dtype)


def grad_bound(d, w):
    dtype = d.dtype
    ref, e = product_bound(d.double(), w.t(), HALF[dtype])
    # one exponent for the whole matrix in fp16
    e = e + 2.0 ** -39 * d.double().abs().sum(1, keepdim=True) * w.abs().max()
    return ref, e + rounded(ref.abs() + e, dtype)


def int8_rows(x):
    """(codes, scales) of the definition: scale the fp32 value of max|x| / 127, codes of the exact quotient."""
    x = x.double()
    s = (x.abs().amax(1) / 127).float()
    q = torch.where(s.unsqueeze(1) > 0, (x / s.double().unsqueeze(1)).round().clamp(-127, 127), 0.0)
    bad = ~torch.isfinite(x).all(1)
    s[bad], q[bad] = float("nan"), 0.0
    return q.to(torch.int8), s


def int8_codes(shape, seed):
    gen = torch.Generator().manual_seed(seed)
    return torch.randint(-128, 128, shape, generator=gen, dtype=torch.int8)


def int8_bound(xq, xs, wq, ws, dtype):
    """(product, bound): the sum is exact, its conversion and two products 2^-24 each."""
    ref = (xq.double() @ wq.double().t()) * xs.double().unsqueeze(1) * ws.double()
    e = ref.abs() * 3.1 * 2.0 ** -24
    return ref, e + (0 if dtype is torch.float32 else rounded(ref.abs() + e, dtype)) + LEAST[dtype] * 4


def check(got, ref, bound):
    got = got.cpu().double()
    assert got.shape == ref.shape
    assert torch.isfinite(got).all()
    worst = ((got - ref).abs() / bound).max().item() if got.numel() else 0.0
    assert worst <= 1.0, worst
    return worst


class Guarded:
    """An output tensor with marked elements before and after it: `whole()` says whether they are untouched."""

    def __init__(self, shape, dtype, dev, pad=64):
        n = math.prod(shape)
        self.flat = torch.full((n + 2 * pad,), 77, dtype=dtype, device=dev)
        self.t, self.pad = self.flat[pad:pad + n].view(shape), pad

    def whole(self):
        return bool((self.flat[:self.pad] == 77).all() and (self.flat[-self.pad:] == 77).all())


def formula_finite(x, w):
    """Where x . w^T of the formula is finite, where it is +-inf (sign) and where NaN, with infinities and NaN in x and w
    (a sum of infinities of one sign is that infinity, of both signs, or 0 times one, NaN)."""
    t = x.unsqueeze(1) * w.unsqueeze(0)
    return t.sum(2)


def assert_like(got, ref):
    """got is NaN where ref is, the same infinity where ref is one, finite elsewhere."""
    got = got.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), (torch.isnan(got) != torch.isnan(ref)).nonzero()[:5]
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf])
    assert torch.isfinite(got[torch.isfinite(ref)]).all()
