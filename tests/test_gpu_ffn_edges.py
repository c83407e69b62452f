"""Gated block, gradients and 8-bit products at their edges: infinities and NaN, magnitudes at either end, scales that
leave the types' ranges, tiles of every size, streams, graphs, several calls at once, and a block used as a whole."""
import math

import numpy as np
import pytest
import torch

import oracle
import synth_inputs
from tests import ffn_util as f
from tests.test_gpu_ffn import ACTS, _gated_case, _grad_case, _int8_case

pytestmark = pytest.mark.gpu


def _w4():
    import bit_weight_only_w4_amd as w4

    return w4


# ---- tiles

@pytest.mark.parametrize("fmt", ["mxfp4_bf16", "int4_f16"])
def test_gated_last_tiles_in_a_second_launch(fmt):
    """280 tiles of 256 x 256: the last 24 are covered with small ones."""
    _gated_case(fmt, 1000, 256, 8960, "silu", seed=11)


def test_gated_int8_last_tiles_in_a_second_launch():
    _int8_case(1000, 8960, 256, "bf16", gated=True, seed=12)
    _int8_case(1003, 8957, 320, "f16", gated=True, seed=13)


@pytest.mark.parametrize("tokens,n,k", [(2050, 8961, 192), (33, 128, 8192), (64, 128, 8192), (300, 700, 2048), (129, 33000, 64),
                                        (700, 256, 4096), (4096, 257, 128)])
def test_gemm_int8_tiles(tokens, n, k):
    """Large tiles with a sparse last round, split rows, one column of tiles, ragged ends of each."""
    for out in ("f32", "bf16"):
        _int8_case(tokens, n, k, out, seed=k)


@pytest.mark.parametrize("fmt", ["nf4_bf16", "fp4_f16"])
@pytest.mark.parametrize("tokens,n,k", [(65, 4160, 128), (400, 1000, 2048), (2100, 200, 4224), (1000, 64, 17920 // 128 * 128)])
def test_gemm_grad_tiles(fmt, tokens, n, k):
    _grad_case(fmt, tokens, n, k, seed=tokens)


def test_many_tokens():
    """The largest number of tokens of the 4-bit calls."""
    _gated_case("int4_bf16", 4096, 128, 24, "silu", seed=2)
    _grad_case("int4_bf16", 4096, 40, 128, seed=2)


# ---- infinities and NaN

def _poison(x, rows):
    """Tokens with one infinity, both, a NaN, and an untouched one between them."""
    x = x.clone()
    x[rows[0], 3] = float("inf")
    x[rows[1], 5], x[rows[1], 70 % x.shape[1]] = float("inf"), -float("inf")
    x[rows[2], x.shape[1] - 1] = float("nan")
    x[rows[3], 0] = -float("inf")
    return x


@pytest.mark.parametrize("fmt", f.FMTS)
@pytest.mark.parametrize("tokens", [1, 6, 40, 300])
def test_gated_nonfinite_tokens(fmt, tokens):
    """A token with an infinity or NaN gives what the formula gives, and nothing of it in the others.  Asymmetric INT4 in
    launches that stream the weights takes z sum(x) off apart: there some of an infinite token's infinite products are
    NaN, and the others the formula's."""
    w4, dev = _w4(), f.device()
    dtype, inter, hidden = f.DTYPES[fmt.split("_")[1]], 20, 256
    p, s, hat = f.weights(fmt, 2 * inter, hidden, 5)
    clean = f.normal((tokens, hidden), dtype, 6)
    for shift in range(4 if tokens == 1 else 1):
        rows = [(i + shift) % 4 if tokens > 1 else (0 if i == shift else -1) for i in range(4)]
        x = clean.clone()
        if tokens == 1:
            extra = _poison(torch.cat([clean] * 4), [0, 1, 2, 3])
            x = extra[shift:shift + 1]
        else:
            x = _poison(clean, rows)
        h, pr = w4.gated(x.to(dev), p.to(dev), s.to(dev), fmt, "silu", save=True)
        bad = ~torch.isfinite(x).all(1)
        both = f.formula_finite(x.double(), hat)
        if fmt.startswith("int4a") and tokens <= 128:
            got, ref = pr.cpu()[bad].double(), both[bad]
            assert not torch.isfinite(got).any() and torch.isnan(got[torch.isnan(ref)]).all()
            assert torch.equal(got[torch.isinf(got)], ref[torch.isinf(got)])
        else:
            f.assert_like(pr[bad.to(dev)], both[bad])
            g, u = both[bad].chunk(2, 1)
            f.assert_like(h[bad.to(dev)], g / (1 + torch.exp(-g)) * u)
        if (~bad).any():
            ref, eh, good, ep = f.gated_bound(x[~bad], hat, "silu", dtype)
            f.check(h[(~bad).to(dev)], ref, eh)
            f.check(pr[(~bad).to(dev)], good, ep)


@pytest.mark.parametrize("fmt", ["nf4_f16", "nf4_bf16", "fp4_f16", "int4a_f16", "int4_bf16", "mxfp4_f16"])
@pytest.mark.parametrize("tokens", [5, 20, 40, 100])
def test_gemm_grad_nonfinite(fmt, tokens):
    """Infinite and NaN gradients: what the formula gives in their tokens, nothing in the others."""
    w4, dev = _w4(), f.device()
    dtype, n, k = f.DTYPES[fmt.split("_")[1]], 100, 256
    p, s, hat = f.weights(fmt, n, k, 5)
    d = _poison(f.normal((tokens, n), dtype, 6, 0.2), [0, 1, 2, 3])
    dx = w4.gemm_grad(d.to(dev), p.to(dev), s.to(dev), fmt)
    bad = ~torch.isfinite(d).all(1)
    f.assert_like(dx[bad.to(dev)], f.formula_finite(d.double(), hat.t().contiguous())[bad])
    ref, e = f.grad_bound(d[~bad], hat)
    f.check(dx[(~bad).to(dev)], ref, e)


@pytest.mark.parametrize("tokens", [3, 40, 200])
@pytest.mark.parametrize("xt", ["f16", "bf16"])
def test_nan_scale_stays_in_its_row(tokens, xt):
    """MXFP4's scale byte 255: NaN in its channel (forward) and in its columns (gradient), nowhere else."""
    w4, dev = _w4(), f.device()
    fmt, dtype, inter, hidden = f"mxfp4_{xt}", f.DTYPES[xt], 24, 192
    p, s = oracle.quantize_mxfp4(synth_inputs.weights(2 * inter, hidden, sigma=0.05, seed=3))
    s = s.copy()
    s[5, 2] = 255
    s[inter + 9, 0] = 255
    pt, st, hat = f.as_operands(fmt, p, s)
    hat = hat.clone()
    hat[5, 64:96], hat[inter + 9, 0:32] = float("nan"), float("nan")
    x = f.normal((tokens, hidden), dtype, 4)
    h, pr = w4.gated(x.to(dev), pt.to(dev), st.to(dev), fmt, save=True)
    assert torch.equal(torch.isnan(pr.cpu()).all(0), torch.isnan(pr.cpu()).any(0))
    assert torch.isnan(pr.cpu()).any(0).nonzero().flatten().tolist() == [5, inter + 9]
    assert torch.isnan(h.cpu()).any(0).nonzero().flatten().tolist() == [5, 9]
    d = f.normal((tokens, 2 * inter), dtype, 5)
    dx = w4.gemm_grad(d.to(dev), pt.to(dev), st.to(dev), fmt).cpu()
    bad = sorted(set(range(64, 96)) | set(range(0, 32)))
    assert torch.isnan(dx).all(0).nonzero().flatten().tolist() == bad and torch.isnan(dx).any(0).sum() == len(bad)


# ---- magnitudes

@pytest.mark.parametrize("xt", ["f16", "bf16"])
@pytest.mark.parametrize("tokens", [1, 20, 200])
@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** 30])
def test_gated_scales_beyond_fp16(xt, tokens, scale):
    """Weights far outside fp16's range: their products are what counts, brought back by tokens as far out (bf16), or
    rounded as x's type rounds them (fp16: to 0, or past its range)."""
    w4, dev, dtype = _w4(), f.device(), f.DTYPES[xt]
    fmt, inter, hidden = f"fp4_{xt}", 18, 128
    p, s = oracle.quantize_fp4(synth_inputs.weights(2 * inter, hidden, sigma=0.05, seed=9))
    pt, st, hat = f.as_operands(fmt, p, (s * np.float32(scale)).astype(np.float32))
    x = f.normal((tokens, hidden), torch.float64, 10)
    x = (x / scale if xt == "bf16" else x).to(dtype)
    h, pr = w4.gated(x.to(dev), pt.to(dev), st.to(dev), fmt, "silu", save=True)
    ref, eh, both, ep = f.gated_bound(x, hat, "silu", dtype)
    if xt == "bf16" or scale < 1:
        f.check(pr, both, ep)
        f.check(h, ref, eh)
    else:
        far = both.abs() - ep > 65520  # what rounds past the type's range whatever the bound's error
        assert far.float().mean() > 0.9
        assert torch.equal(torch.isinf(pr.cpu())[far], torch.ones(int(far.sum()), dtype=torch.bool))


@pytest.mark.parametrize("tokens", [20, 200])
def test_gated_token_of_many_magnitudes(tokens):
    """bf16 tokens whose values span the type's range: off by at most 2^-39 of the token's largest times the weights."""
    w4, dev = _w4(), f.device()
    fmt, inter, hidden = "nf4_bf16", 16, 256
    p, s, hat = f.weights(fmt, 2 * inter, hidden, 21)
    x = f.normal((tokens, hidden), torch.float64, 22) * 2.0 ** (torch.arange(hidden) % 60 - 40).double()
    x = x.to(torch.bfloat16)
    _, pr = w4.gated(x.to(dev), p.to(dev), s.to(dev), fmt, save=True)
    _, _, both, ep = f.gated_bound(x, hat, "silu", torch.bfloat16)
    f.check(pr, both, ep)


@pytest.mark.parametrize("xt", ["f16", "bf16"])
@pytest.mark.parametrize("tokens", [5, 200])
@pytest.mark.parametrize("scale", [2.0 ** -40, 2.0 ** 20])
def test_gemm_grad_scales_beyond_fp16(xt, tokens, scale):
    w4, dev, dtype = _w4(), f.device(), f.DTYPES[xt]
    fmt, n, k = f"nf4_{xt}", 70, 192
    p, s = oracle.quantize_nf4(synth_inputs.weights(n, k, sigma=0.05, seed=9))
    pt, st, hat = f.as_operands(fmt, p, (s * np.float32(scale)).astype(np.float32))
    d = f.normal((tokens, n), torch.float64, 10, 0.1)
    d = (d / scale if xt == "bf16" else d * (1e-3 if scale > 1 else 1.0)).to(dtype)
    dx = w4.gemm_grad(d.to(dev), pt.to(dev), st.to(dev), fmt)
    f.check(dx, *f.grad_bound(d, hat))


def test_zero_weights_and_tokens():
    w4, dev = _w4(), f.device()
    for tokens in (1, 9, 200):
        for fmt in f.FMTS:
            dtype = f.DTYPES[fmt.split("_")[1]]
            p, s = w4.quantize(fmt, torch.zeros(12, 128, device=dev))
            x = f.normal((tokens, 128), dtype, 1).to(dev)
            h, pr = w4.gated(x, p, s, fmt, save=True)
            assert (h == 0).all() and (pr == 0).all()
            assert (w4.gemm_grad(f.normal((tokens, 12), dtype, 1).to(dev), p, s, fmt) == 0).all()
            p, s, _ = f.weights(fmt, 12, 128, 1)
            h, pr = w4.gated(x * 0, p.to(dev), s.to(dev), fmt, "gelu_tanh", save=True)
            assert (h == 0).all() and (pr == 0).all()


# ---- streams, graphs, calls at once

def _block(tokens, fmt="nf4_bf16", hidden=256, inter=192, seed=1):
    """A block's tensors on the GPU: x, gate_up, down and a gradient of its output."""
    dtype, dev = f.DTYPES[fmt.split("_")[1]], f.device()
    gu, dn = f.weights(fmt, 2 * inter, hidden, seed), f.weights(fmt, hidden, inter, seed + 1)
    x, dy = f.normal((tokens, hidden), dtype, seed + 2), f.normal((tokens, hidden), dtype, seed + 3, 0.3)
    return dict(fmt=fmt, x=x.to(dev), dy=dy.to(dev), gu=[t.to(dev) for t in gu[:2]], dn=[t.to(dev) for t in dn[:2]],
                hat=(gu[2], dn[2]))


def _step(b, act="silu"):
    """Forward and backward pass of the block as a training step makes them."""
    w4 = _w4()
    h, pr = w4.gated(b["x"], *b["gu"], b["fmt"], act, save=True)
    y = w4.gemm_smallbatch(h, *b["dn"], b["fmt"])
    dh = w4.gemm_grad(b["dy"], *b["dn"], b["fmt"])
    dp = w4.gated_grad(dh, pr, act)
    return y, h, pr, dh, dp, w4.gemm_grad(dp, *b["gu"], b["fmt"])


@pytest.mark.parametrize("fmt", ["nf4_bf16", "int4_f16", "mxfp4_bf16", "int4a_f16"])
@pytest.mark.parametrize("tokens", [1, 30, 200])
@pytest.mark.parametrize("act", ACTS)
def test_block_forward_and_backward(fmt, tokens, act):
    """Each result of a whole step against the formula at that step's own inputs."""
    b = _block(tokens, fmt, hidden=256, inter=256, seed=tokens)
    y, h, pr, dh, dp, dx = _step(b, act)
    dtype = b["x"].dtype
    gu, dn = b["hat"]
    ref, eh, both, ep = f.gated_bound(b["x"].cpu(), gu, act, dtype)
    f.check(h, ref, eh)
    f.check(pr, both, ep)
    hc = h.cpu().double()
    f.check(y, hc @ dn.t(), 2e-3 * (hc.abs() @ dn.abs().t()) + 1e-5)
    f.check(dh, *f.grad_bound(b["dy"].cpu(), dn))
    f.check(dp, *f.gated_grad_bound(dh.cpu(), pr.cpu(), act))
    f.check(dx, *f.grad_bound(dp.cpu(), gu))


@pytest.mark.parametrize("act", ACTS)
def test_block_gradient_against_differences(act):
    """dx of the whole step against central differences of sum(dy * block(x)) in 64 bits, along random directions.  The
    step rounds h's gradient, the products and their gradients to bf16, three roundings of 2^-8 of each term and the
    weights' two: 2^-5 of the sum of the magnitudes that make up the derivative along the direction."""
    b = _block(40, "nf4_bf16", seed=7)
    dx = _step(b, act)[-1].cpu().double()
    x, dy, (gu, dn) = b["x"].cpu().double(), b["dy"].cpu().double(), b["hat"]

    def value(z):
        g, u = (z @ gu.t()).chunk(2, 1)
        return (dy * ((f.act(act, g)[0] * u) @ dn.t())).sum(1)

    g, u = (x @ gu.t()).chunk(2, 1)
    a, slope = f.act(act, g)
    dh = dy.abs() @ dn.abs()
    mag = torch.cat((dh * (u.abs() + 1) * (slope.abs() + 0.5), dh * (a.abs() + 0.5)), 1) @ gu.abs()
    for seed in range(4):
        v = f.normal(x.shape, torch.float64, 100 + seed)
        num = (value(x + 1e-4 * v) - value(x - 1e-4 * v)) / 2e-4
        got = (dx * v).sum(1)
        assert ((got - num).abs() <= 2.0 ** -5 * (mag * v.abs()).sum(1) + 1e-6).all()


@pytest.mark.parametrize("tokens", [1, 40, 300])
def test_step_on_another_stream(tokens):
    b = _block(tokens)
    want = _step(b)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    w4 = _w4()
    h, pr = w4.gated(b["x"], *b["gu"], b["fmt"], save=True, stream=side)
    dh = w4.gemm_grad(b["dy"], *b["dn"], b["fmt"], stream=side)
    dp = w4.gated_grad(dh, pr, stream=side)
    dx = w4.gemm_grad(dp, *b["gu"], b["fmt"], stream=side)
    q, s = w4.quantize_int8(b["x"], stream=side)
    wq, ws = w4.quantize_int8(b["x"].new_ones(40, 256).cumsum(1), stream=side)
    y8 = w4.gemm_int8(q, s, wq, ws, stream=side)
    h8 = w4.gated_int8(q, s, wq, ws, stream=side)
    side.synchronize()
    for a, c in zip((h, pr, dh, dp, dx), want[1:]):
        assert torch.equal(a, c)
    q2, s2 = w4.quantize_int8(b["x"])
    assert torch.equal(q, q2) and torch.equal(s, s2)
    assert torch.equal(y8, w4.gemm_int8(q2, s2, wq, ws)) and torch.equal(h8, w4.gated_int8(q2, s2, wq, ws))


@pytest.mark.parametrize("tokens", [1, 24, 90, 300])
def test_step_in_a_graph(tokens):
    """Captured and replayed with new inputs and eager work between the replays."""
    w4 = _w4()
    b = _block(tokens, hidden=512, inter=320)
    wq, ws = w4.quantize_int8(f.normal((70, 512), torch.float32, 3).to(f.device()))
    gq, gs = w4.quantize_int8(f.normal((60, 512), torch.float32, 4, 0.05).to(f.device()))

    def all_of_it():
        q, s = w4.quantize_int8(b["x"])
        return (*_step(b), q, s, w4.gemm_int8(q, s, wq, ws, torch.bfloat16), *w4.gated_int8(q, s, gq, gs, save=True))

    all_of_it()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = all_of_it()
    for seed in (50, 60, 70):
        b["x"].copy_(f.normal(tuple(b["x"].shape), b["x"].dtype, seed).to(f.device()))
        b["dy"].copy_(f.normal(tuple(b["dy"].shape), b["dy"].dtype, seed + 1).to(f.device()))
        graph.replay()
        torch.cuda.synchronize()
        kept = [o.clone() for o in outs]
        for a, c in zip(kept, all_of_it()):
            assert torch.equal(a, c)
        torch.cuda.synchronize()


def test_two_streams_at_once():
    """The same calls on two streams, each with its own workspace: the same results as one after the other."""
    w4 = _w4()
    blocks = [_block(200, "fp4_f16", hidden=512, inter=512, seed=s) for s in (1, 20)]
    want = [_step(b) for b in blocks]
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for b, st in zip(blocks, streams):
            with torch.cuda.stream(st):
                got.append(_step(b))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for a, c in zip(g, w):
                assert torch.equal(a, c)


def test_workspaces_given_and_dirty():
    """A workspace of the stated size, filled with NaN patterns beforehand, and one that is too small."""
    w4, dev = _w4(), f.device()
    for fmt in ("nf4_bf16", "int4_f16"):
        b = _block(300, fmt, hidden=256, inter=128)
        n = w4.gated_workspace_bytes(fmt, 300, 256, 128)
        ws = torch.full((n,), 255, dtype=torch.uint8, device=dev)
        assert torch.equal(w4.gated(b["x"], *b["gu"], fmt, workspace=ws), w4.gated(b["x"], *b["gu"], fmt))
        with pytest.raises(w4.W4ValueError):
            w4.gated(b["x"], *b["gu"], fmt, workspace=ws[:n - 16])
        for tokens in (3, 300):
            d = f.normal((tokens, 256), b["x"].dtype, 5).to(dev)
            n = w4.gemm_grad_workspace_bytes(fmt, 256, 256, tokens)
            ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device=dev)
            assert torch.equal(w4.gemm_grad(d, *b["gu"], fmt, workspace=ws), w4.gemm_grad(d, *b["gu"], fmt))
    xq, wq = f.int8_codes((50, 8192), 1).to(dev), f.int8_codes((96, 8192), 2).to(dev)
    xs, ws_ = torch.rand(50, device=dev), torch.rand(96, device=dev)
    n = w4.int8_workspace_bytes(96, 8192, 50)
    assert n > 0
    ws = torch.full((n,), 255, dtype=torch.uint8, device=dev)
    assert torch.equal(w4.gemm_int8(xq, xs, wq, ws_, workspace=ws), w4.gemm_int8(xq, xs, wq, ws_))


def test_binding_refusals_on_the_gpu():
    w4, dev = _w4(), f.device()
    b = _block(4)
    x, (p, s) = b["x"], b["gu"]
    bad = [(x.half(), p, s, "nf4_bf16"), (x[:, ::2], p, s, "nf4_bf16"), (x, p[:-1], s[:-1], "nf4_bf16"), (x, p, s[:, :-1], "nf4_bf16"),
           (x, p, s.double(), "nf4_bf16"), (x, p.cpu(), s, "nf4_bf16"), (x, p, s, "nf5_bf16"), (x, p, s, "int4_bf16"),
           (x[:, :128].contiguous(), p, s, "nf4_bf16"), (x[0], p, s, "nf4_bf16")]
    for args in bad:
        with pytest.raises(ValueError):
            w4.gated(*args)
    with pytest.raises(ValueError):
        w4.gated(x, p, s, "nf4_bf16", act="relu")
    with pytest.raises(ValueError):
        w4.gated(x, p, s, "nf4_bf16", h=torch.empty(4, 192, device=dev))
    with pytest.raises(ValueError):
        w4.gated(x, p, s, "nf4_bf16", products=torch.empty(4, 192, dtype=x.dtype, device=dev))
    with pytest.raises(w4.W4ValueError):  # h on top of x
        w4.gated(x, p, s, "nf4_bf16", h=x.view(-1)[:4 * 192].view(4, 192))
    dh = x.new_zeros(4, 192)
    for args in ((dh, dh), (dh, x.new_zeros(4, 384).half()), (dh.float(), x.new_zeros(4, 384).float()),
                 (dh[:, ::2], x.new_zeros(4, 192))):
        with pytest.raises(ValueError):
            w4.gated_grad(*args)
    pr = x.new_zeros(4, 384)
    with pytest.raises(w4.W4ValueError):
        w4.gated_grad(dh, pr, d_products=pr)
    d = x.new_zeros(4, 384)
    for args in ((d[:, :-2].contiguous(), p, s, "nf4_bf16"), (d.half(), p, s, "nf4_bf16"), (d, p, s.half(), "nf4_bf16"),
                 (d.cpu(), p, s, "nf4_bf16"), (d, p, s, "x")):
        with pytest.raises(ValueError):
            w4.gemm_grad(*args)
    q, sc = w4.quantize_int8(x)
    for args in ((q.float(), sc, q, sc), (q, sc.double(), q, sc), (q, sc, q[:, :128], sc), (q, sc[:2], q, sc), (q, sc, q.cpu(), sc)):
        with pytest.raises(ValueError):
            w4.gemm_int8(*args)
    with pytest.raises(ValueError):
        w4.gemm_int8(q, sc, q, sc, torch.int32)
    with pytest.raises(ValueError):
        w4.gated_int8(q, sc, q[:3], sc[:3])
    with pytest.raises(ValueError):
        w4.gated_int8(q, sc, q, sc, dtype=torch.float32)
    with pytest.raises(w4.W4ValueError):  # K no multiple of 64
        w4.gemm_int8(q[:, :100].contiguous(), sc, q[:, :100].contiguous(), sc)
    with pytest.raises(ValueError):
        w4.quantize_int8(x.double())


def test_empty_batches_are_refused():
    w4, dev = _w4(), f.device()
    b = _block(2)
    with pytest.raises(w4.W4ValueError):
        w4.gated(b["x"][:0], *b["gu"], b["fmt"])
    with pytest.raises(w4.W4ValueError):
        w4.gemm_grad(b["dy"][:0], *b["dn"], b["fmt"])
    with pytest.raises(w4.W4ValueError):
        w4.quantize_int8(b["x"][:0])


@pytest.mark.parametrize("rows", [4, 4100])
def test_offsets_past_32_bits(rows):
    """Rows whose first element lies past 2^31 of its buffer."""
    w4, dev = _w4(), f.device()
    k = (1 << 31) // 4096 + 64
    if rows * k < 1 << 31:
        k = (1 << 23) + 64
    x = torch.zeros(rows, k, dtype=torch.float16, device=dev)
    x[-1, -1], x[-1, 0], x[0, 5] = 2.0, -1.0, 1.0
    codes, scales = w4.quantize_int8(x)
    assert codes[-1, -1] == 127 and codes[-1, 0] == -64 and codes[0, 5] == 127 and int((codes != 0).sum()) == 3
    assert math.isclose(float(scales[-1]), 2.0 / 127, rel_tol=1e-6)


def test_gated_grad_past_32_bits():
    w4, dev = _w4(), f.device()
    tokens, inter = 130, 1 << 23
    pr = torch.zeros(tokens, 2 * inter, dtype=torch.bfloat16, device=dev)
    dh = torch.zeros(tokens, inter, dtype=torch.bfloat16, device=dev)
    pr[-1, inter - 1], pr[-1, -1], dh[-1, -1] = 1.0, 3.0, 2.0
    dp = w4.gated_grad(dh, pr)
    assert int((dp != 0).sum()) == 2
    p = 1 / (1 + math.exp(-1))
    assert abs(float(dp[-1, inter - 1]) - 6 * p * (2 - p)) < 0.05 and abs(float(dp[-1, -1]) - 2 * p) < 0.01


def test_more_rows_than_one_launch_holds():
    """2^26 rows of one value: 2^32 threads."""
    w4, dev = _w4(), f.device()
    rows = (1 << 26) + 3
    x = (torch.arange(rows, dtype=torch.int32, device=dev) % 5 - 2).to(torch.bfloat16).view(rows, 1)
    codes, scales = w4.quantize_int8(x)
    assert torch.equal(codes.view(-1), (x.view(-1).sign() * 127).to(torch.int8))
    assert torch.equal(scales, x.view(-1).abs().float() / 127.0)


def test_gated_grad_of_more_than_2_32_single_channels():
    w4, dev = _w4(), f.device()
    tokens = (1 << 32) + 5
    pr = torch.zeros(tokens, 2, dtype=torch.bfloat16, device=dev)
    dh = torch.zeros(tokens, 1, dtype=torch.bfloat16, device=dev)
    at = [0, (1 << 31) - 1, 1 << 31, 1 << 32, tokens - 1]
    for t in at:
        pr[t, 0], pr[t, 1], dh[t, 0] = 1.0, 3.0, 2.0
    dp = w4.gated_grad(dh, pr)
    assert int((dp != 0).sum()) == 2 * len(at)
    p = 1 / (1 + math.exp(-1))
    for t in at:
        assert abs(float(dp[t, 0]) - 6 * p * (2 - p)) < 0.05 and abs(float(dp[t, 1]) - 2 * p) < 0.01


@pytest.mark.parametrize("rows,k", [(2048, 1536), (2049, 1535), (2047, 1536), (2050, 1544), (513, 2056), (512, 2056), (3, 2049),
                                    (600, 10250), (2, 16400), (5, 16384)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_quantize_int8_launches(dtype, rows, k):
    """Both sides of each bound of the launch's rule, rows that a workgroup does not hold, and quotients on and next to
    the borders between two codes."""
    w4, dev = _w4(), f.device()
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    g = torch.Generator().manual_seed(rows + k)
    x = torch.randn(rows, k, generator=g)
    half = torch.randint(-254, 255, (rows, k), generator=g).float() / 2
    half[:, 0] = 127.0  # scale 1: the others lie on integers and borders
    x[1::2] = half[1::2]
    if dtype == "f32":
        nudge = torch.randint(0, 3, (rows, k), generator=g)
        x = torch.where(nudge == 1, torch.nextafter(x, torch.zeros(())), x)
        x[1::2, 0] = 127.0
    x = x.to(dt)
    codes, scales = w4.quantize_int8(x.to(dev))
    q, s = f.int8_rows(x)
    assert torch.equal(scales.cpu(), s) and torch.equal(codes.cpu(), q)


# ---- weights decoded by the product itself

@pytest.mark.parametrize("fmt", f.FMTS)
@pytest.mark.parametrize("tokens,steps,inter", [(129, 1, 1), (256, 9, 333), (144, 4, 1030), (256, 40, 129), (257, 3, 140),
                                                (512, 5, 70), (513, 5, 70)])
def test_gated_decoded_in_the_product(fmt, tokens, steps, inter):
    """One step and many, ragged channels, one row of tiles, K split over workgroups; around each format's last number of
    tokens."""
    _gated_case(fmt, tokens, steps * f.group(fmt), inter, ACTS[inter % 2], seed=steps)


@pytest.mark.parametrize("fmt", ["mxfp4_f16", "mxfp4_bf16"])
@pytest.mark.parametrize("tokens,hidden,inter", [(2048, 320, 700), (2049, 320, 700), (700, 128, 9100), (511, 64, 4500)])
def test_gated_mxfp4_tiles(fmt, tokens, hidden, inter):
    _gated_case(fmt, tokens, hidden, inter, "silu", seed=hidden)


@pytest.mark.parametrize("fmt", ["nf4_f16", "nf4_bf16"])
@pytest.mark.parametrize("tokens", [129, 256, 257])
def test_gated_many_weights(fmt, tokens):
    """100 million NF4 weights, a sample of whose channels is compared."""
    w4, dev, dtype = _w4(), f.device(), f.DTYPES[fmt.split("_")[1]]
    hidden, inter = 1024, 48900
    g = torch.Generator(device=dev).manual_seed(tokens)
    p = torch.randint(0, 256, (2 * inter, hidden // 2), dtype=torch.uint8, device=dev, generator=g)
    s = torch.rand((2 * inter, hidden // 64), device=dev, generator=g) * 0.1
    x = f.normal((tokens, hidden), dtype, 3)
    h, pr = w4.gated(x.to(dev), p, s, fmt, "silu", save=True)
    at = torch.cat((torch.arange(0, inter, 1511), torch.tensor([inter - 1])))
    rows = torch.cat((at, at + inter))
    _, _, hat = f.as_operands(fmt, p[rows.to(dev)].cpu().numpy(), s[rows.to(dev)].cpu().numpy())
    ref, eh, both, ep = f.gated_bound(x, hat, "silu", dtype)
    f.check(pr[:, rows.to(dev)], both, ep)
    f.check(h[:, at.to(dev)], ref, eh)


@pytest.mark.parametrize("fmt", f.FMTS)
@pytest.mark.parametrize("tokens", [1, 20, 200, 300])
def test_gated_nonfinite_scales(fmt, tokens):
    """An infinite or NaN scale of a gate or up row gives no finite product of its row and leaves the others alone."""
    w4, dev, dtype = _w4(), f.device(), f.DTYPES[fmt.split("_")[1]]
    hidden, inter = 256, 70
    p, s, hat = f.weights(fmt, 2 * inter, hidden, 31)
    bad = [3, 64, inter + 5, 2 * inter - 1]
    weight = fmt.split("_")[0]
    s = s.clone()
    raw = s.view({"mxfp4": torch.uint8, "int4": torch.int16}.get(weight, torch.int32))
    for i, row in enumerate(bad):
        nan = i % 2 or weight == "mxfp4"
        raw[row, 1] = {"mxfp4": 255, "int4": 0x7FC0 if nan else 0x7F80,
                       "int4a": (0x7FC0 if nan else 0x7F80) | 3 << 16}.get(weight, 0x7FC00000 if nan else 0x7F800000)
    x = f.normal((tokens, hidden), dtype, 32)
    x = torch.where(x == 0, torch.ones_like(x), x)
    h, pr = w4.gated(x.to(dev), p.to(dev), s.to(dev), fmt, "silu", save=True)
    ref, eh, both, ep = f.gated_bound(x, hat, "silu", dtype)
    good = torch.ones(2 * inter, dtype=torch.bool)
    good[bad] = False
    f.check(pr.cpu()[:, good], both[:, good], ep[:, good])
    assert not torch.isfinite(pr.cpu()[:, ~good]).any()
    good = good[:inter] & good[inter:]
    f.check(h.cpu()[:, good], ref[:, good], eh[:, good])


# ---- gradients whose product decodes and transposes the weights itself: large matrices, a sample of whose columns is compared

def _raw_weights(fmt, n, k, seed):
    """Random packed weights and scales on the GPU (of about 0.02 to 0.1), as the binding takes them."""
    dev, weight = f.device(), fmt.split("_")[0]
    g = torch.Generator(device=dev).manual_seed(seed)
    p = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device=dev, generator=g)
    if weight == "mxfp4":
        return p, torch.randint(120, 124, (n, k // 32), dtype=torch.uint8, device=dev, generator=g)
    s = torch.rand((n, k // (128 if weight.startswith("int4") else 64)), device=dev, generator=g) * 0.08 + 0.02
    if weight in ("nf4", "fp4"):
        return p, s
    bits = s.bfloat16().view(torch.int16)
    if weight == "int4":
        return p, bits
    zero = torch.randint(0, 16, bits.shape, dtype=torch.int32, device=dev, generator=g)
    return p, bits.int() & 0xFFFF | zero << 16


def _columns(fmt, p, s, blocks):
    """fp64 values of the 128 columns of each of `blocks` (of 128), [n, 128 blocks]."""
    weight = fmt.split("_")[0]
    per = {"nf4": 2, "fp4": 2, "mxfp4": 4}.get(weight, 1)
    out = []
    for b in blocks:
        sc = s[:, b * per:(b + 1) * per].contiguous().cpu().numpy()
        sc = sc.view({"int4": np.uint16, "int4a": np.uint32}.get(weight, sc.dtype))
        out.append(f.as_operands(fmt, p[:, 64 * b:64 * (b + 1)].contiguous().cpu().numpy(), sc)[2])
    at = torch.cat([torch.arange(128 * b, 128 * b + 128) for b in blocks])
    return torch.cat(out, 1), at


@pytest.mark.parametrize("fmt", f.FMTS)
@pytest.mark.parametrize("tokens,n,k", [(65, 8003, 2176), (130, 28000, 1152), (512, 20000, 1664), (333, 11008, 4224),
                                        (1000, 28672, 4224), (2000, 28000, 4224)])
def test_gemm_grad_decoded_in_the_product(fmt, tokens, n, k):
    """Weight rows that end inside a step, an odd number of groups a row (scales on odd halves of a word), columns that end
    inside a tile, each tile, one and several splits."""
    w4, dev, dtype = _w4(), f.device(), f.DTYPES[fmt.split("_")[1]]
    p, s = _raw_weights(fmt, n, k, tokens)
    d = f.normal((tokens, n), dtype, 3, 0.3)
    dx = f.Guarded((tokens, k), dtype, dev)
    w4.gemm_grad(d.to(dev), p, s, fmt, dx=dx.t)
    torch.cuda.synchronize()
    assert dx.whole()
    hat, at = _columns(fmt, p, s, [0, k // 256, k // 128 - 1])
    few = torch.arange(0, tokens, max(1, tokens // 97))
    ref, e = f.grad_bound(d[few], hat)
    f.check(dx.t.cpu()[few][:, at], ref, e)
    assert torch.isfinite(dx.t).all()
    again = w4.gemm_grad(d.to(dev), p, s, fmt)
    assert torch.equal(again, dx.t)


@pytest.mark.parametrize("fmt", ["nf4_f16", "fp4_bf16", "int4_f16", "int4a_bf16", "mxfp4_f16", "mxfp4_bf16"])
def test_gemm_grad_decoded_in_the_product_nonfinite(fmt):
    """Infinite and NaN gradients stay in their tokens, non-finite scales in their blocks' columns."""
    w4, dev, dtype = _w4(), f.device(), f.DTYPES[fmt.split("_")[1]]
    weight, n, k = fmt.split("_")[0], 9001, 1152
    p, s = _raw_weights(fmt, n, k, 5)
    d = _poison(f.normal((100, n), dtype, 6, 0.2), [0, 20, 63, 64])
    dx = w4.gemm_grad(d.to(dev), p, s, fmt).cpu()
    bad = ~torch.isfinite(d).all(1)
    hat, at = _columns(fmt, p, s, [0, 8])
    for t in bad.nonzero().flatten().tolist():  # what an infinity or NaN meets decides: every other term is finite
        odd = ~torch.isfinite(d[t])
        ref = (d[t, odd].double().unsqueeze(1) * hat[odd]).sum(0)
        f.assert_like(dx[t:t + 1, at], ref.unsqueeze(0))
    ref, e = f.grad_bound(d[~bad], hat)
    f.check(dx[~bad][:, at], ref, e)
    raw = s.view({"mxfp4": torch.uint8, "int4": torch.int16}.get(weight, torch.int32))
    raw[7000, 2] = {"mxfp4": 255, "int4": 0x7FC0, "int4a": 0x7F80}.get(weight, 0x7F800000)
    raw[9000, raw.shape[1] - 1] = {"mxfp4": 255, "int4": 0x7F80, "int4a": 0x7FC0}.get(weight, 0x7FC00000)
    d = torch.where(d == 0, torch.ones_like(d), d)
    dx = w4.gemm_grad(d.to(dev), p, s, fmt).cpu()[~bad]
    g = k // raw.shape[1]
    hit = torch.zeros(k, dtype=torch.bool)
    hit[2 * g:3 * g], hit[k - g:] = True, True
    assert not torch.isfinite(dx[:, hit]).any() and torch.isfinite(dx[:, ~hit]).all()


@pytest.mark.parametrize("xt", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [2.0 ** -40, 2.0 ** 20])
def test_gemm_grad_decoded_in_the_product_beyond_fp16(xt, scale):
    w4, dev, dtype, fmt = _w4(), f.device(), f.DTYPES[xt], f"nf4_{xt}"
    p, s = _raw_weights(fmt, 9000, 1152, 8)
    s = s * scale
    d = (f.normal((80, 9000), torch.float64, 9, 0.3) / (scale if xt == "bf16" else 2.0 ** 14 if scale > 1 else 1)).to(dtype)
    dx = w4.gemm_grad(d.to(dev), p, s, fmt).cpu()
    hat, at = _columns(fmt, p, s, [0, 8])
    ref, e = f.grad_bound(d, hat)
    if xt == "bf16" or scale < 1:
        f.check(dx[:, at], ref, e)
    else:
        inside = ref.abs() + e < 65504
        assert inside.any() and bool(((dx[:, at].double() - ref).abs() <= e)[inside].all())


@pytest.mark.parametrize("fmt", f.FMTS)
@pytest.mark.parametrize("tokens", [31, 32, 33, 49, 64, 65])
def test_gemm_grad_around_the_last_few_tokens(fmt, tokens):
    _grad_case(fmt, tokens, 330, 3 * f.group(fmt), seed=tokens)


@pytest.mark.parametrize("fmt", ["nf4_bf16", "int4_f16", "int4_bf16", "fp4_bf16", "int4a_f16", "mxfp4_f16", "mxfp4_bf16"])
@pytest.mark.parametrize("tokens", [33, 48])
def test_gemm_grad_decoded_in_the_product_few(fmt, tokens):
    w4, dev, dtype = _w4(), f.device(), f.DTYPES[fmt.split("_")[1]]
    p, s = _raw_weights(fmt, 9537, 1152, tokens)
    d = f.normal((tokens, 9537), dtype, 3, 0.3)
    dx = w4.gemm_grad(d.to(dev), p, s, fmt)
    hat, at = _columns(fmt, p, s, [0, 4, 8])
    ref, e = f.grad_bound(d, hat)
    f.check(dx[:, at.to(dev)], ref, e)


@pytest.mark.parametrize("fmt", f.FMTS)
@pytest.mark.parametrize("tokens", [64, 65, 128, 129])
@pytest.mark.parametrize("steps,inter", [(1, 70), (8, 17000)])
def test_gated_around_the_last_few_tokens(fmt, tokens, steps, inter):
    """Small and large matrices (of which a sample of channels is compared)."""
    w4, dev, dtype = _w4(), f.device(), f.DTYPES[fmt.split("_")[1]]
    hidden = steps * 128
    p, s = _raw_weights(fmt, 2 * inter, hidden, tokens)
    x = f.normal((tokens, hidden), dtype, 3)
    h, pr = w4.gated(x.to(dev), p, s, fmt, "silu", save=True)
    at = torch.cat((torch.arange(0, inter, max(1, inter // 37)), torch.tensor([inter - 1])))
    rows = torch.cat((at, at + inter)).to(dev)
    hat, _ = _columns(fmt, p[rows], s[rows], range(steps))
    ref, eh, both, ep = f.gated_bound(x, hat, "silu", dtype)
    f.check(pr[:, rows], both, ep)
    f.check(h[:, at.to(dev)], ref, eh)


@pytest.mark.parametrize("fmt", ["nf4_f16", "int4_bf16", "mxfp4_f16"])
def test_gemm_grad_decoded_in_the_product_in_graphs_and_streams(fmt):
    """Captured and replayed with new inputs; two calls at once; a dirty workspace of the stated size, and none other."""
    w4, dev, dtype = _w4(), f.device(), f.DTYPES[fmt.split("_")[1]]
    tokens, n, k = 90, 9001, 1152
    p, s = _raw_weights(fmt, n, k, 7)
    d = [f.normal((tokens, n), dtype, 3 + i, 0.3).to(dev) for i in range(2)]
    want = [w4.gemm_grad(x, p, s, fmt) for x in d]
    size = w4.gemm_grad_workspace_bytes(fmt, n, k, tokens)
    ws = [torch.full((size + 64,), 0xFF, dtype=torch.uint8, device=dev) for _ in d]
    streams = [torch.cuda.Stream() for _ in d]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [w4.gemm_grad(x, p, s, fmt, workspace=w[:size], stream=st) for x, w, st in zip(d, ws, streams)]
        torch.cuda.synchronize()
        for a, b, w in zip(got, want, ws):
            assert torch.equal(a, b) and bool((w[size:] == 0xFF).all())
    with pytest.raises(w4.W4Error):
        w4.gemm_grad(d[0], p, s, fmt, workspace=ws[0][:size - 16])
    x = d[0].clone()
    w4.gemm_grad(x, p, s, fmt)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = w4.gemm_grad(x, p, s, fmt)
    for i in (1, 0, 1):
        x.copy_(d[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
        w4.gemm_grad(d[i], p, s, fmt)
        torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", ["nf4_bf16", "mxfp4_f16", "int4a_bf16", "fp4_f16"])
def test_gated_decoded_in_the_product_in_graphs_and_streams(fmt):
    w4, dev, dtype = _w4(), f.device(), f.DTYPES[fmt.split("_")[1]]
    tokens, hidden, inter = 200, 1024, 1500
    p, s = _raw_weights(fmt, 2 * inter, hidden, 7)
    xs = [f.normal((tokens, hidden), dtype, 3 + i).to(dev) for i in range(2)]
    want = [w4.gated(x, p, s, fmt, save=True) for x in xs]
    size = w4.gated_workspace_bytes(fmt, tokens, hidden, inter)
    assert 0 < size < 2 * inter * hidden * 2
    ws = [torch.full((size + 64,), 0xFF, dtype=torch.uint8, device=dev) for _ in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [w4.gated(x, p, s, fmt, save=True, workspace=w[:size], stream=st) for x, w, st in zip(xs, ws, streams)]
        torch.cuda.synchronize()
        for a, b, w in zip(got, want, ws):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and bool((w[size:] == 0xFF).all())
    x = xs[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = w4.gated(x, p, s, fmt)
    for i in (1, 0, 1):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i][0])
        w4.gated(xs[i], p, s, fmt)
        torch.cuda.synchronize()


@pytest.mark.parametrize("xt", ["f16", "bf16"])
@pytest.mark.parametrize("tokens,hidden,inter", [(2, 64, 1), (16, 6720, 781), (16, 192, 4801), (33, 448, 15), (64, 1600, 129),
                                                 (128, 320, 33)])
def test_gated_mxfp4_up_scales_inside_a_dword(xt, tokens, hidden, inter):
    """An odd number of channels times an odd number of 64-weight blocks: the up rows' scales start two bytes into a dword,
    and the tiles asked for ahead end past them."""
    _gated_case(f"mxfp4_{xt}", tokens, hidden, inter, "silu", seed=inter)


@pytest.mark.parametrize("tokens", [2, 16, 40, 128])
def test_grouped_mxfp4_scales_inside_a_dword(tokens):
    """The grouped small-batch product over members whose scales start two bytes into a dword, ragged row counts."""
    w4, dev, fmt, k = _w4(), f.device(), "mxfp4_f16", 320
    x = f.normal((tokens, k), torch.float16, 3).to(dev)
    packed, scales, hats = [], [], []
    for i, n in enumerate((17, 783, 5)):
        p, s, hat = f.weights(fmt, n, k, 40 + i)
        flat = torch.zeros(s.numel() + 8, dtype=torch.uint8, device=dev)
        flat[2:2 + s.numel()] = s.to(dev).flatten()
        packed.append(p.to(dev))
        scales.append(flat[2:2 + s.numel()].view(s.shape))
        hats.append(hat)
    ys = w4.gemm_smallbatch_grouped(x, packed, scales, fmt)
    torch.cuda.synchronize()
    for y, hat in zip(ys, hats):
        ref = x.cpu().double() @ hat.t()
        bound = 2.0 ** -11 * (x.cpu().double().abs() @ hat.t().abs()) + 1e-6
        assert ((y.cpu().double() - ref).abs() <= bound).all()
