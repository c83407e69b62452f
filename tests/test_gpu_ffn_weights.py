"""The weights of the gated block and of the product's gradient, read out one by one and in differences of nearly equal
ones: what a kernel makes of a 4-bit weight before it multiplies shows up whole, not below the rounding of a long sum.

Bound: a result is rounded to its type once (half a step); before that a weight enters as fp32 or as the sum of 16-bit
terms that leave at most 2^-20.4 of it (the second term of two fp16 ones is below 2^-8.4 of the weight's binade, and half
a step of it 2^-20), code times scale is rounded to fp32 (2^-24), and the few additions are fp32's: 2^-21 of the terms.
Together 2^-19 of the terms' magnitudes."""
import numpy as np
import pytest
import torch

from tests import ffn_util as f
from tests.test_gpu_ffn_edges import _raw_weights

pytestmark = pytest.mark.gpu

TERMS = 2.0 ** -19
INEXACT = [x for x in f.FMTS if not x.startswith("mxfp4")]


def _w4():
    import bit_weight_only_w4_amd as w4

    return w4


def _hat(fmt, p, s):
    weight = fmt.split("_")[0]
    sc = s.cpu().numpy()
    sc = sc.view({"int4": np.uint16, "int4a": np.uint32}.get(weight, sc.dtype))
    return f.as_operands(fmt, p.cpu().numpy(), sc)[2].double()


def _bf16_bits(v):
    return v.view(torch.int32) >> 16 & 0xFFFF


def _blocks(fmt, rows, groups, seed):
    """[rows, groups] blocks of one code each: even groups any code and a scale of all its bits, odd ones the code 1 or -1
    with the scale that comes nearest to the weight before it from below in 12 bits (integers: the bf16 number).  Returns
    packed weights and scales."""
    weight = fmt.split("_")[0]
    gen = torch.Generator().manual_seed(seed)
    g = f.group(fmt)
    codes = torch.randint(0, 16, (rows, groups), generator=gen)
    codes[:, ::2] = (torch.arange(rows).unsqueeze(1) * 7 + torch.arange(0, groups, 2)) % 16  # every code
    s = torch.rand(rows, groups, generator=gen) * 3 + 1
    zero = torch.full((rows, groups), 8)
    if weight in ("int4", "int4a"):
        s = (s.view(torch.int32) & ~0xFFFF).view(torch.float32)
        zero[:, ::2] = torch.randint(0, 16, (rows, (groups + 1) // 2), generator=gen) if weight == "int4a" else 8
        value = (codes - zero) * s.double()
    else:
        table = torch.from_numpy(f.oracle.dequant(weight, np.array([[i * 17 for i in range(16)] + [0] * 16], np.uint8),
                                                  np.ones((1, 1), np.float32)))[0, :32:2].double()
        value = table[codes] * s.double()
    w = value[:, ::2].float()
    near = (w.abs().view(torch.int32) & ~(0xFFFF if weight.startswith("int4") else 0xFFF)).view(torch.float32)
    one = {"nf4": (15, 0), "fp4": (2, 10)}.get(weight, (9, 7))
    odd = near[:, :groups // 2]
    codes[:, 1::2] = torch.where(w[:, :groups // 2] < 0, one[1], one[0])
    s[:, 1::2] = torch.where(odd > 0, odd, torch.ones(()))
    codes = codes.to(torch.uint8)
    p = (codes * 17).repeat_interleave(g // 2, dim=1).contiguous()
    if weight == "int4":
        s = _bf16_bits(s.contiguous()).to(torch.int32).to(torch.int16)
    elif weight == "int4a":
        s = (_bf16_bits(s.contiguous()) | zero.int() << 16).int()
    return p, s.contiguous()


def _check(got, ref, terms):
    got = got.cpu()
    e = (ref.abs() + TERMS * terms) * f.HALF[got.dtype] + f.LEAST[got.dtype] + TERMS * terms
    f.check(got, ref, e)


@pytest.mark.parametrize("fmt", INEXACT)
@pytest.mark.parametrize("tokens", [1, 2, 7, 33, 64, 100, 128, 129, 200, 257, 400, 1100])
def test_gated_products_of_nearly_equal_weights(fmt, tokens):
    """Each token takes one weight of a block less one of the next, in every row."""
    w4, dev, dtype = _w4(), f.device(), f.DTYPES[fmt.split("_")[1]]
    inter, groups = 75, 6
    g = f.group(fmt)
    p, s = _blocks(fmt, 2 * inter, groups, tokens)
    hat = _hat(fmt, p, s)
    x = torch.zeros(tokens, groups * g, dtype=torch.float64)
    for t in range(tokens):
        pair = t % (groups // 2)
        x[t, 2 * pair * g + t * 5 % g] = 1.0
        x[t, (2 * pair + 1) * g + t * 3 % g] = -1.0
    _, pr = w4.gated(x.to(dtype).to(dev), p.to(dev), s.to(dev), fmt, save=True)
    _check(pr, x @ hat.t(), x.abs() @ hat.abs().t())


@pytest.mark.parametrize("fmt", INEXACT)
@pytest.mark.parametrize("tokens,n,steps", [(1, 70, 2), (16, 640, 3), (32, 333, 2), (33, 640, 2), (64, 1001, 2), (65, 129, 4),
                                            (130, 20000, 9), (300, 640, 4), (600, 9000, 9)])
def test_gradient_of_nearly_equal_weights(fmt, tokens, n, steps):
    """Each token takes the difference of two rows that are nearly equal in every column, the first and the last rows, and
    rows on both sides of steps among them."""
    w4, dev, dtype = _w4(), f.device(), f.DTYPES[fmt.split("_")[1]]
    p, s = _blocks(fmt, steps, 2 * ((n + 1) // 2), n)  # rows and blocks change places
    g = f.group(fmt)
    p = p.view(steps, -1, g // 2).transpose(0, 1).reshape(-1, steps * g // 2)[:n].contiguous()
    s = s.t()[:n].contiguous()
    hat = _hat(fmt, p, s)
    pairs = n // 2
    d = torch.zeros(tokens, n, dtype=torch.float64)
    terms = torch.zeros(tokens, steps * g, dtype=torch.float64)
    for t in range(tokens):
        at = (t // 2 if t % 2 == 0 else pairs - 1 - t // 2) if t % 3 else t * 16 + 15
        at %= pairs
        d[t, 2 * at], d[t, 2 * at + 1] = 1.0, -1.0
        terms[t] = hat[2 * at].abs() + hat[2 * at + 1].abs()
    dx = w4.gemm_grad(d.to(dtype).to(dev), p.to(dev), s.to(dev), fmt)
    _check(dx, d @ hat, terms)


@pytest.mark.parametrize("fmt", f.FMTS)
@pytest.mark.parametrize("tokens,n,k", [(1, 40, 384), (16, 1000, 512), (31, 4003, 384), (32, 28672, 1152), (64, 700, 640),
                                        (65, 8003, 2176), (130, 28000, 1152), (129, 200, 896), (333, 4001, 640),
                                        (512, 20000, 1664), (1000, 28672, 4224), (2049, 300, 384)])
def test_gradient_reads_weights_out(fmt, tokens, n, k):
    """Each token is one number in one row: a row of weights comes back, at one rounding.  The first, the last and the tail
    rows, rows on both sides of steps, and rows all over; other tokens' rows are far from it in value."""
    w4, dev, dtype = _w4(), f.device(), f.DTYPES[fmt.split("_")[1]]
    p, s = _raw_weights(fmt, n, k, tokens)
    edge = [0, n - 1, n - 2, 63, 64, 31, 32, n // 64 * 64 - 1, n // 64 * 64, n // 64 * 64 + 1, 127, 128, n // 2, n // 4, 3 * n // 4]
    rows = torch.tensor([(edge[t] if t < len(edge) else t * 7919) % n for t in range(tokens)])
    value = 2.0 ** (torch.arange(tokens) % 5).double() * (1 - 2 * (torch.arange(tokens) % 2))
    d = torch.zeros(tokens, n, dtype=dtype)
    d[torch.arange(tokens), rows] = value.to(dtype)
    dx = w4.gemm_grad(d.to(dev), p, s, fmt).cpu()
    at = rows.to(dev)
    ref = _hat(fmt, p[at], s[at]) * value.unsqueeze(1)
    if len(torch.unique(rows)) > 3:
        assert len(torch.unique(ref, dim=0)) > 3
    _check(dx, ref, ref.abs())


@pytest.mark.parametrize("fmt", f.FMTS)
@pytest.mark.parametrize("tokens,hidden,inter", [(1, 384, 40), (1, 4224, 77), (5, 640, 33), (64, 384, 100), (128, 1152, 77), (129, 640, 200),
                                                 (300, 2176, 333), (512, 4224, 40), (700, 640, 3000), (2049, 384, 90)])
def test_gated_products_read_weights_out(fmt, tokens, hidden, inter):
    w4, dev, dtype = _w4(), f.device(), f.DTYPES[fmt.split("_")[1]]
    p, s = _raw_weights(fmt, 2 * inter, hidden, tokens)
    edge = [0, hidden - 1, 63, 64, 31, 32, 127, 128, hidden - 64, hidden - 65, hidden // 2]
    cols = torch.tensor([(edge[t] if t < len(edge) else t * 7919) % hidden for t in range(tokens)])
    value = 2.0 ** (torch.arange(tokens) % 5).double() * (1 - 2 * (torch.arange(tokens) % 2))
    x = torch.zeros(tokens, hidden, dtype=dtype)
    x[torch.arange(tokens), cols] = value.to(dtype)
    _, pr = w4.gated(x.to(dev), p, s, fmt, save=True)
    ref = _hat(fmt, p, s)[:, cols].t() * value.unsqueeze(1)
    _check(pr, ref, ref.abs())
