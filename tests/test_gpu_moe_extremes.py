"""The largest calls that the expert layer, its router and MXFP4 accept: most tokens, slots and experts, longest
rows, matrices past 4 GiB, skewed and mostly absent slots."""
import numpy as np
import pytest

import oracle
import synth_inputs
from tests import gpu_util as g
from tests import moe_util as mu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _decode(packed, scales):
    """fp64 weights of MXFP4 bytes on the device."""
    import torch

    book = torch.tensor(oracle.fp4_codebook(), dtype=torch.float64, device=packed.device)
    p = packed.to(torch.int32)
    hat = torch.stack((book[p >> 4], book[p & 15]), dim=-1).flatten(-2)
    scale = torch.exp2(scales.double() - 127.0)
    return hat.view(*scale.shape, 32).mul_(scale.unsqueeze(-1)).view(hat.shape)


def test_router_of_the_most_tokens():
    import torch

    import bit_weight_only_w4_amd as w4

    tokens = (1 << 26) - 1
    v = torch.randn(tokens, 2, device=g.device()).half()
    ids, w = w4.moe_route(v, 1)
    assert torch.equal(ids[:, 0], (v[:, 1] > v[:, 0]).int())
    assert bool((w == 1.0).all())


@pytest.mark.parametrize("kind", ["even", "skewed", "mostly absent"])
@pytest.mark.parametrize("experts", [1024, 3])
def test_most_tokens_and_slots(kind, experts):
    import bit_weight_only_w4_amd as w4

    tokens, top_k = 4096, 16
    c = mu.case("mxfp4_bf16", 1, 64, 64, experts, 1, seed=experts)
    rng = np.random.default_rng(5)
    c["x"] = synth_inputs.activations(tokens, 64, "bf16", seed=9)
    c["weights"] = rng.random((tokens, top_k)).astype(np.float32)
    ids = rng.integers(0, experts, (tokens, top_k))  # an expert may stand in several slots
    if kind == "skewed":
        ids = np.minimum(rng.geometric(0.3, ids.shape) - 1, experts - 1)
    if kind == "mostly absent":
        ids = np.where(rng.random(ids.shape) < 0.9, -1, ids)
    c["ids"] = ids.astype(np.int32)
    y = w4.moe(*mu.to_device(c, g.device()))
    rows = np.unique(np.concatenate([[0, 1, tokens - 2, tokens - 1], rng.choice(tokens, 150)]))
    sub = dict(c, x=c["x"][rows], ids=c["ids"][rows], weights=c["weights"][rows])
    mu.check(y[rows], sub)


def _longest(tokens, hidden, inter, seed):
    """Random MXFP4 experts (two) and x; scales 2^-8 .. 2^-5."""
    import torch

    dev = g.device()
    gen = torch.Generator(device=dev).manual_seed(seed)

    def matrix(n, k):
        return (torch.randint(0, 256, (2, n, k // 2), dtype=torch.uint8, device=dev, generator=gen),
                torch.randint(119, 123, (2, n, k // 32), dtype=torch.uint8, device=dev, generator=gen))

    gu, dn = matrix(2 * inter, hidden), matrix(hidden, inter)
    x = torch.randn(tokens, hidden, device=dev, generator=gen).half()
    ids = torch.randint(0, 2, (tokens, 1), dtype=torch.int32, device=dev, generator=gen)
    w = torch.rand(tokens, 1, device=dev, generator=gen)
    return x, ids, w, gu, dn


@pytest.mark.parametrize("tokens", [1, 3, 40])
def test_longest_hidden(tokens):
    """hidden = 2^22 - 64: few activations are not zero, all rows of y are looked at."""
    import torch

    import bit_weight_only_w4_amd as w4

    hidden, inter = (1 << 22) - 64, 64
    x, ids, w, gu, dn = _longest(tokens, hidden, inter, seed=tokens)
    cols = torch.cat([torch.tensor([0, 31, 32, hidden - 65, hidden - 1]), torch.randint(0, hidden, (60,))]).unique()
    keep = torch.zeros(hidden, dtype=torch.bool)
    keep[cols] = True
    x = x * keep.to(x.device)
    y = w4.moe(x, ids, w, *gu, *dn, "mxfp4_f16")
    cols = cols.to(x.device)
    blocks = (cols // 32).unique()
    at = (blocks[:, None] * 16 + torch.arange(16, device=x.device)).flatten()
    xs = x.view(tokens, -1, 32)[:, blocks].reshape(tokens, -1).double()
    for e in (0, 1):
        t = torch.nonzero(ids[:, 0] == e).flatten()
        if t.numel() == 0:
            continue
        a = _decode(gu[0][e][:, at], gu[1][e][:, blocks])
        d = _decode(dn[0][e], dn[1][e])
        both, mag = torch.matmul(xs[t], a.t().contiguous()), torch.matmul(xs[t].abs(), a.abs().t().contiguous())
        gate, up = both[:, :inter], both[:, inter:]
        h = gate / (1 + torch.exp(-gate)) * up
        # at most 65 columns that are not zero: sums of 65 terms, and zeros add nothing
        err = (65 + 64) * U * mag
        dh = 1.1 * err[:, :inter] * (up.abs() + err[:, inter:]) + gate.abs() * err[:, inter:] + 2.0 ** -20 * h.abs()
        da = d.abs().t().contiguous()
        want = torch.matmul(h, d.t().contiguous())
        bound = torch.matmul(dh, da) + (64 / 32 + 64 + 3) * U * torch.matmul(h.abs() + dh, da)
        wt = w[t].double()
        assert bool(((y[t].double() - wt * want).abs() <= wt * bound + 2.0 ** -126 * inter).all())


@pytest.mark.parametrize("tokens", [1, 3, 40])
def test_longest_inter(tokens):
    """inter = 2^22 - 64; every product of the first is looked at through y."""
    import torch

    import bit_weight_only_w4_amd as w4

    hidden, inter = 64, (1 << 22) - 64
    x, ids, w, gu, dn = _longest(tokens, hidden, inter, seed=tokens + 9)
    y = w4.moe(x, ids, w, *gu, *dn, "mxfp4_f16")
    for t in sorted({0, tokens // 2, tokens - 1}):
        e = int(ids[t, 0])
        a = _decode(gu[0][e], gu[1][e])
        xt = x[t].double()
        both, mag = torch.mv(a, xt), torch.mv(a.abs_(), xt.abs())
        del a
        gate, up = both[:inter], both[inter:]
        h = gate / (1 + torch.exp(-gate)) * up
        err = (64 / 32 + 64) * U * mag
        dh = 1.1 * err[:inter] * (up.abs() + err[inter:]) + gate.abs() * err[inter:] + 2.0 ** -20 * h.abs()
        d = _decode(dn[0][e], dn[1][e])
        want, size = torch.mv(d, h), torch.mv(d.abs(), h.abs() + dh)
        bound = torch.mv(d.abs(), dh) + (inter / 32 + 64 + 3) * U * size
        wt = float(w[t, 0])
        assert bool(((y[t].double() - wt * want).abs() <= wt * bound + 2.0 ** -126 * inter).all()), t
