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
