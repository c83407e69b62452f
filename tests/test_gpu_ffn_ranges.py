"""Gated block and its gradients at the ends of their types' ranges, and operands at addresses of their own."""
import threading

import pytest
import torch

from tests import ffn_util as f
from tests.test_gpu_ffn import ACTS

pytestmark = pytest.mark.gpu


def _w4():
    import bit_weight_only_w4_amd as w4

    return w4


@pytest.mark.parametrize("act", ACTS)
def test_gated_grad_of_large_and_small_factors(act):
    """dh * u alone may leave fp32's range, and so may u * act'(g); their product with the third does not."""
    w4, dev = _w4(), f.device()
    mags = [1e20, 1e30, 3e38, 1e-20, 1e-30, 1e-38, 1.0]
    gates = [-200.0, -90.0, -60.0, -40.0, -8.0, -1.0, 0.0, 1.0, 40.0]
    rows = [(d, u, g) for d in mags for u in mags for g in gates]
    t = torch.tensor(rows, dtype=torch.float64).to(torch.bfloat16)
    dh, pr = t[:, :1].contiguous(), torch.stack((t[:, 2], t[:, 1]), 1).contiguous()
    got = w4.gated_grad(dh.to(dev), pr.to(dev), act).cpu().double()
    ref, bound = f.gated_grad_bound(dh, pr, act)
    assert not torch.isnan(got).any()
    inside = ref.abs() + bound < 3.38e38
    assert ((got - ref).abs() <= bound)[inside].all()
    assert inside.sum() > 600


@pytest.mark.parametrize("fmt", ["int4_f16", "int4_bf16", "mxfp4_f16", "mxfp4_bf16"])
@pytest.mark.parametrize("tokens,steps,inter", [(1, 3, 41), (1, 17, 130), (5, 3, 17), (40, 5, 33), (100, 3, 70), (200, 3, 65),
                                                (600, 3, 65)])
def test_gated_scales_two_bytes_into_a_dword(fmt, tokens, steps, inter):
    """Two-byte scales at an address that is no multiple of four, as every other call takes them."""
    w4, dev, dtype = _w4(), f.device(), f.DTYPES[fmt.split("_")[1]]
    p, s, hat = f.weights(fmt, 2 * inter, steps * f.group(fmt), tokens)
    x = f.normal((tokens, steps * f.group(fmt)), dtype, 2)
    raw = s.contiguous().view(torch.uint8).flatten()
    flat = torch.full((raw.numel() + 8,), 255, dtype=torch.uint8, device=dev)
    flat[2:2 + raw.numel()] = raw.to(dev)
    at = flat[2:2 + raw.numel()].view(s.dtype).view(s.shape)
    assert at.data_ptr() % 4 == 2
    h, pr = w4.gated(x.to(dev), p.to(dev), at, fmt, "silu", save=True)
    ref, eh, both, ep = f.gated_bound(x, hat, "silu", dtype)
    f.check(h, ref, eh)
    f.check(pr, both, ep)
    h2, pr2 = w4.gated(x.to(dev), p.to(dev), s.to(dev), fmt, "silu", save=True)
    assert torch.equal(h, h2) and torch.equal(pr, pr2)


def test_first_calls_of_several_threads():
    """Threads that make their first calls at the same time, of sizes that no other test launches."""
    w4, dev = _w4(), f.device()
    cases = []
    for i, (fmt, tokens, steps) in enumerate((("int4a_f16", 9, 2), ("int4a_f16", 30, 2), ("fp4_bf16", 50, 3), ("mxfp4_f16", 13, 1),
                                              ("nf4_f16", 100, 2), ("nf4_bf16", 19, 4), ("int4_bf16", 61, 5), ("int4_f16", 200, 3))):
        p, s, hat = f.weights(fmt, 2 * 45, steps * f.group(fmt), i)
        x = f.normal((tokens, steps * f.group(fmt)), f.DTYPES[fmt.split("_")[1]], i + 1)
        cases.append((fmt, x, p.to(dev), s.to(dev), hat, x.to(dev)))
    torch.cuda.synchronize()
    start, out = threading.Barrier(2 * len(cases)), {}

    def call(k):
        fmt, _, p, s, _, x = cases[k % len(cases)]
        stream = torch.cuda.Stream()
        start.wait()
        out[k] = w4.gated(x, p, s, fmt, stream=stream)
        stream.synchronize()

    threads = [threading.Thread(target=call, args=(k,)) for k in range(2 * len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for k in range(len(cases)):
        fmt, x, _, _, hat, _ = cases[k]
        ref, eh, _, _ = f.gated_bound(x, hat, "silu", x.dtype)
        f.check(out[k], ref, eh)
        assert torch.equal(out[k], out[k + len(cases)])


LARGEST = {"nf4": 1.0, "fp4": 6.0, "mxfp4": 6.0, "int4": 8.0, "int4a": 15.0}


def _spread(fmt, rows, blocks, seed):
    """Random codes; a row's first block has a scale of 1 to 2, block j one 2^(20 + j) times smaller.  Also the largest
    weight that each row's scales allow."""
    weight = fmt.split("_")[0]
    g = f.group(fmt)
    gen = torch.Generator().manual_seed(seed)
    p = torch.randint(0, 256, (rows, blocks * g // 2), generator=gen, dtype=torch.uint8)
    down = torch.arange(blocks).double() + 20
    down[0] = 0
    s = (1 + torch.rand(rows, blocks, generator=gen, dtype=torch.float64)) * 2.0 ** -down
    s = s.float()
    if weight == "mxfp4":
        e = (127 - down.long()).expand(rows, blocks).repeat_interleave(2, dim=1)
        return p, e.to(torch.uint8).contiguous(), torch.full((rows,), 6.0, dtype=torch.float64)
    if weight.startswith("int4"):
        bits = s.view(torch.int32) >> 16
        top = (bits[:, 0] << 16).view(torch.float32).double() * LARGEST[weight]
        if weight == "int4":
            return p, bits.to(torch.int16), top
        return p, bits | torch.randint(0, 16, bits.shape, generator=gen, dtype=torch.int32) << 16, top
    return p, s, s[:, 0].double() * LARGEST[weight]


@pytest.mark.parametrize("weight", ["nf4", "fp4", "mxfp4", "int4", "int4a"])
@pytest.mark.parametrize("tokens", [192, 700])
def test_gated_weights_far_below_the_largest(weight, tokens):
    """Weights read out one by one, down to 2^36 below the row's largest scale: off by at most 2^-20 of themselves, or 2^-39
    of what the row's largest scale and the format's largest code allow."""
    w4, dev, fmt = _w4(), f.device(), f"{weight}_bf16"
    g, blocks, inter = f.group(fmt), 16, 24
    p, s, top = _spread(fmt, 2 * inter, blocks, tokens)
    hat = f.as_operands(fmt, p.numpy(), s.numpy().view({"int4": "uint16", "int4a": "uint32"}.get(weight, s.numpy().dtype)))[2]
    cols = torch.arange(tokens) * 37 % (blocks * g)
    x = torch.zeros(tokens, blocks * g, dtype=torch.bfloat16)
    x[torch.arange(tokens), cols] = 1.0
    _, pr = w4.gated(x.to(dev), p.to(dev), s.to(dev), fmt, save=True)
    ref = hat.double()[:, cols].t()
    e = ref.abs() * 2.0 ** -20 + 2.0 ** -39 * top
    f.check(pr, ref, e + f.rounded(ref.abs() + e, torch.bfloat16))


@pytest.mark.parametrize("weight,xt", [("nf4", "bf16"), ("fp4", "bf16"), ("mxfp4", "bf16"), ("int4", "bf16"), ("int4a", "bf16")])
@pytest.mark.parametrize("tokens,rows", [(100, 40), (70, 16000)])
def test_gradient_weights_far_below_the_largest(weight, xt, tokens, rows):
    """The same along the weight rows, which share an exponent with the other rows of their columns only; some columns
    have small weights alone, and nothing is lost there."""
    w4, dev, fmt = _w4(), f.device(), f"{weight}_{xt}"
    g, groups = f.group(fmt), 5
    p, s, top = _spread(fmt, groups, rows, tokens + 1)
    p = p.view(groups, rows, g // 2).transpose(0, 1).reshape(rows, groups * g // 2).contiguous()
    per = s.shape[1] // rows
    s = s.view(groups, rows, per).transpose(0, 1).reshape(rows, groups * per).contiguous()
    if rows > 1000:  # (the scales of most rows would be 0)
        s[40:] = s[torch.arange(40, rows) % 39 + 1]
    first = {"mxfp4": 60, "int4": 0x2000, "int4a": 0x2000}.get(weight, 2.0 ** -60)
    s[:, -per:] = first  # the last group's: small in every row
    top[-1] = LARGEST[weight] * (2.0 ** -67 if weight == "mxfp4" else float(torch.tensor(0x2000 << 16, dtype=torch.int32).view(
        torch.float32)) if weight.startswith("int4") else 2.0 ** -60)
    hat = f.as_operands(fmt, p.numpy(), s.numpy().view({"int4": "uint16", "int4a": "uint32"}.get(weight, s.numpy().dtype)))[2]
    at = torch.arange(tokens) % min(rows, 40) if rows < 1000 else torch.arange(tokens) * 131 % rows
    d = torch.zeros(tokens, rows, dtype=torch.bfloat16)
    d[torch.arange(tokens), at] = 1.0
    dx = w4.gemm_grad(d.to(dev), p.to(dev), s.to(dev), fmt)
    ref = hat.double()[at]
    e = ref.abs() * 2.0 ** -20 + 2.0 ** -39 * top.repeat_interleave(g)
    f.check(dx, ref, e + f.rounded(ref.abs() + e, torch.bfloat16))


@pytest.mark.parametrize("tokens", [1, 3, 200])
@pytest.mark.parametrize("hidden", [1536, 4096, 6144])
@pytest.mark.parametrize("power", [-127, -118, -60, 90])
def test_gated_tokens_at_the_ends_of_bf16(tokens, hidden, power):
    """bf16 tokens near the smallest and the largest of their type, brought back by the weights' scales."""
    w4, dev, fmt = _w4(), f.device(), "nf4_bf16"
    p, s, _ = f.weights(fmt, 2 * 20, hidden, 3)
    s = (s * 2.0 ** min(-power, 120)).contiguous()
    hat = f.as_operands(fmt, p.numpy(), s.numpy())[2]
    x = (f.normal((tokens, hidden), torch.float64, 4) * 2.0 ** power).to(torch.bfloat16)
    h, pr = w4.gated(x.to(dev), p.to(dev), s.to(dev), fmt, "silu", save=True)
    ref, eh, both, ep = f.gated_bound(x, hat, "silu", torch.bfloat16)
    f.check(pr, both, ep)
    f.check(h, ref, eh)


def test_gated_tokens_subnormal_chunks_read_out():
    """One number in the smallest of bf16 in each chunk of a long token: nothing of it is lost."""
    w4, dev, fmt, hidden = _w4(), f.device(), "nf4_bf16", 4096
    p, s, _ = f.weights(fmt, 2 * 20, hidden, 5)
    s = (s * 2.0 ** 120).contiguous()
    hat = f.as_operands(fmt, p.numpy(), s.numpy())[2].double()
    for at, value in ((0, 2.0 ** -126), (33, 3 * 2.0 ** -133), (4095, 2.0 ** -120), (64, -2.0 ** -133), (1000, 1.9921875 * 2.0 ** -115)):
        x = torch.zeros(1, hidden, dtype=torch.bfloat16)
        x[0, at] = value
        x[0, at ^ 1] = value * 2.0 ** -6 if value > 2.0 ** -125 else 0.0
        _, pr = w4.gated(x.to(dev), p.to(dev), s.to(dev), fmt, "silu", save=True)
        ref = x.double() @ hat.t()
        e = 2.0 ** -22 * (x.double().abs() @ hat.abs().t())
        f.check(pr, ref, e + f.rounded(ref.abs() + e, torch.bfloat16))
