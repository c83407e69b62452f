"""Gated block, its gradients and 8-bit products on the GPU against plain fp64 forms."""
import pytest
import torch

from tests import ffn_util as f

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu_tanh"]


def _w4():
    import bit_weight_only_w4_amd as w4

    return w4


def _gated_case(fmt, tokens, hidden, inter, act, seed=1, save=True):
    w4, dev = _w4(), f.device()
    dtype = f.DTYPES[fmt.split("_")[1]]
    p, s, hat = f.weights(fmt, 2 * inter, hidden, seed)
    x = f.normal((tokens, hidden), dtype, seed + 1)
    h, pr = f.Guarded((tokens, inter), dtype, dev), f.Guarded((tokens, 2 * inter), dtype, dev)
    out = w4.gated(x.to(dev), p.to(dev), s.to(dev), fmt, act, h=h.t, products=pr.t if save else None)
    torch.cuda.synchronize()
    ref, eh, both, ep = f.gated_bound(x, hat, act, dtype)
    f.check(h.t, ref, eh)
    assert h.whole() and pr.whole()
    if save:
        assert out[0] is h.t and out[1] is pr.t
        f.check(pr.t, both, ep)
    else:
        assert out is h.t
    return h.t, pr.t


@pytest.mark.parametrize("fmt", f.FMTS)
@pytest.mark.parametrize("tokens,steps,inter", [(1, 1, 1), (1, 3, 40), (2, 5, 17), (5, 2, 130), (16, 3, 33), (17, 2, 64),
                                                (31, 1, 15), (33, 3, 129), (64, 2, 80), (70, 4, 200), (130, 1, 16),
                                                (200, 7, 48), (257, 2, 300)])
def test_gated(fmt, tokens, steps, inter):
    _gated_case(fmt, tokens, steps * f.group(fmt), inter, ACTS[(tokens + inter) % 2], seed=tokens)


@pytest.mark.parametrize("fmt", ["nf4_bf16", "int4_f16", "mxfp4_bf16"])
@pytest.mark.parametrize("tokens", [1, 8, 24, 48, 96, 300])
def test_gated_long_rows(fmt, tokens):
    """Rows past one pass of a workgroup and an odd number of channels."""
    _gated_case(fmt, tokens, 4224, 77, "silu", seed=7, save=tokens % 16 == 0)


@pytest.mark.parametrize("fmt", ["nf4_f16", "int4a_bf16"])
def test_gated_many_tiles(fmt):
    """As many tiles as the largest tile needs before it is taken."""
    _gated_case(fmt, 1100, 256, 9000, "gelu_tanh", seed=3)


@pytest.mark.parametrize("fmt", f.FMTS)
@pytest.mark.parametrize("tokens", [1, 20, 300])
def test_gated_equals_itself(fmt, tokens):
    a = _gated_case(fmt, tokens, 256, 50, "silu")
    b = _gated_case(fmt, tokens, 256, 50, "silu")
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("xt", ["f16", "bf16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("tokens,inter", [(1, 1), (1, 8), (3, 7), (2, 4096), (33, 1409), (257, 264), (5, 24)])
@pytest.mark.parametrize("shift", [0, 1])
def test_gated_grad(xt, act, tokens, inter, shift):
    """shift: operands that start one element past an aligned address."""
    w4, dev, dtype = _w4(), f.device(), f.DTYPES[xt]
    dh, pr = f.normal((tokens, inter), dtype, 1, 0.3), f.normal((tokens, 2 * inter), dtype, 2, 3.0)

    def put(t):
        flat = torch.zeros(t.numel() + 8, dtype=dtype, device=dev)
        flat[shift:shift + t.numel()] = t.to(dev).flatten()
        return flat[shift:shift + t.numel()].view(t.shape)

    out = f.Guarded((tokens, 2 * inter), dtype, dev)
    assert w4.gated_grad(put(dh), put(pr), act, d_products=out.t) is out.t
    torch.cuda.synchronize()
    f.check(out.t, *f.gated_grad_bound(dh, pr, act))
    assert out.whole()


@pytest.mark.parametrize("act", ACTS)
def test_gated_grad_extremes(act):
    """Gates far out on either side, and the largest of bf16: the slope goes to 0 and 1, no NaN comes of it."""
    w4, dev = _w4(), f.device()
    g = torch.tensor([-3e38, -1e20, -1e5, -200.0, -88.0, -20.0, -0.0, 0.0, 20.0, 88.0, 200.0, 1e5, 1e20, 3e38])
    pr = torch.stack((g, torch.ones_like(g)), 0).reshape(1, -1).to(torch.bfloat16)
    dh = torch.ones(1, g.numel(), dtype=torch.bfloat16)
    got = w4.gated_grad(dh.to(dev), pr.to(dev), act).cpu().double()
    ref = torch.cat((torch.where(g > 10, 1.0, 0.0), torch.where(g > 10, pr[0, :g.numel()].float(), 0.0))).double()
    ref[[6, 7]] = 0.5
    assert ((got[0] - ref).abs() <= ref.abs() * 2.0 ** -8 + 1e-6).all(), got
    pr[0, 3] = float("nan")
    got = w4.gated_grad(dh.to(dev), pr.to(dev), act).cpu()
    assert torch.isnan(got[0, 3]) and torch.isnan(got[0, g.numel() + 3])
    assert torch.isfinite(got[0]).sum() == got.numel() - 2


def _grad_case(fmt, tokens, n, k, seed=1, shift=0):
    w4, dev = _w4(), f.device()
    dtype = f.DTYPES[fmt.split("_")[1]]
    p, s, hat = f.weights(fmt, n, k, seed)
    d = f.normal((tokens, n), dtype, seed + 1, 0.3)
    flat = torch.zeros(d.numel() + 8, dtype=dtype, device=dev)
    flat[shift:shift + d.numel()] = d.to(dev).flatten()
    dx = f.Guarded((tokens, k), dtype, dev)
    assert w4.gemm_grad(flat[shift:shift + d.numel()].view(d.shape), p.to(dev), s.to(dev), fmt, dx=dx.t) is dx.t
    torch.cuda.synchronize()
    f.check(dx.t, *f.grad_bound(d, hat))
    assert dx.whole()
    return dx.t


@pytest.mark.parametrize("fmt", f.FMTS)
@pytest.mark.parametrize("tokens,n,steps", [(1, 1, 1), (1, 64, 3), (2, 65, 1), (5, 200, 2), (16, 33, 5), (17, 128, 3),
                                            (33, 7, 2), (40, 320, 1), (65, 129, 4), (130, 64, 2), (200, 500, 3),
                                            (257, 63, 5)])
def test_gemm_grad(fmt, tokens, n, steps):
    _grad_case(fmt, tokens, n, steps * f.group(fmt), seed=tokens)


@pytest.mark.parametrize("fmt", ["nf4_bf16", "int4_f16", "fp4_f16"])
@pytest.mark.parametrize("tokens,n", [(1, 4097), (12, 2048), (48, 3001), (100, 4224)])
def test_gemm_grad_long_sums(fmt, tokens, n):
    _grad_case(fmt, tokens, n, 384, seed=5)


@pytest.mark.parametrize("tokens,n", [(3, 64), (70, 128), (300, 256)])
def test_gemm_grad_unaligned_rows(tokens, n):
    """d at an address that no 16-byte access takes."""
    _grad_case("nf4_bf16", tokens, n, 256, shift=1)
    _grad_case("int4_f16", tokens, n, 256, shift=3)


@pytest.mark.parametrize("fmt", ["nf4_f16", "nf4_bf16"])
def test_gemm_grad_many_tiles(fmt):
    _grad_case(fmt, 600, 256, 9024, seed=3)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 8), (3, 7), (2, 64), (5, 513), (1, 1024), (4, 1025), (3, 8960), (2, 10240),
                                    (2, 10241), (1, 40000), (300, 96)])
@pytest.mark.parametrize("shift", [0, 1])
def test_quantize_int8(dtype, rows, k, shift):
    w4, dev, dt = _w4(), f.device(), f.DTYPES[dtype]
    x = f.normal((rows, k), dt, rows + k, 3.0)
    flat = torch.zeros(x.numel() + 8, dtype=dt, device=dev)
    flat[shift:shift + x.numel()] = x.to(dev).flatten()
    codes, scales = f.Guarded((rows, k), torch.int8, dev), f.Guarded((rows,), torch.float32, dev)
    w4.quantize_int8(flat[shift:shift + x.numel()].view(x.shape), codes=codes.t, scales=scales.t)
    torch.cuda.synchronize()
    q, s = f.int8_rows(x)
    assert torch.equal(scales.t.cpu(), s) and torch.equal(codes.t.cpu(), q)
    assert codes.whole() and scales.whole()


def test_quantize_int8_borders():
    """Values on and next to the middle between two codes, for scales of many mantissas and magnitudes."""
    w4, dev = _w4(), f.device()
    rows = []
    for i in range(64):
        top = torch.tensor(2.0 ** (i * 3 - 140) * (1 + i / 64.0 + 2.0 ** -20), dtype=torch.float32)
        s = (top.double() / 127).float()
        mid = ((torch.arange(-126, 126, dtype=torch.float64) + 0.5) * s.double()).float()
        rows.append(torch.cat((mid, torch.nextafter(mid, torch.tensor(float("inf"))),
                               torch.nextafter(mid, torch.tensor(-float("inf"))), top.reshape(1), -top.reshape(1))))
    x = torch.stack(rows)
    x = torch.where(x.abs() > x[:, -2:-1], x[:, -2:-1], x)
    codes, scales = w4.quantize_int8(x.to(dev))
    q, s = f.int8_rows(x)
    assert torch.equal(scales.cpu(), s) and torch.equal(codes.cpu(), q)


def test_quantize_int8_odd_rows():
    """Rows of zeros, of the smallest and the largest numbers, with infinities and NaN."""
    w4, dev = _w4(), f.device()
    inf, nan = float("inf"), float("nan")
    least, most = 2.0 ** -149, torch.finfo(torch.float32).max
    x = torch.tensor([[0.0, -0.0, 0.0, 0.0], [least, -least, 0, 2 * least], [63 * least, 64 * least, -190 * least, least],
                      [most, -most, most / 2, 1.0], [inf, 1, 2, 3], [1, -inf, 2, 3], [nan, 1, 2, 3], [1, 2, 3, nan],
                      [1, 0.5, -0.5, -1], [1e-38, -1e-38, 5e-39, 1e-40]], dtype=torch.float32)
    codes, scales = w4.quantize_int8(x.to(dev))
    q, s = f.int8_rows(x)
    assert torch.equal(torch.nan_to_num(scales.cpu(), nan=-1.0), torch.nan_to_num(s, nan=-1.0))
    assert torch.equal(codes.cpu(), q)
    y = w4.gemm_int8(torch.zeros(10, 64, dtype=torch.int8, device=dev), scales, torch.ones(3, 64, dtype=torch.int8, device=dev),
                     torch.ones(3, device=dev))
    assert torch.isnan(y[4:8]).all() and (y[:4] == 0).all() and (y[8:] == 0).all()


def _int8_case(tokens, n, k, out, gated=False, act="silu", seed=1):
    w4, dev, dt = _w4(), f.device(), f.DTYPES[out]
    rows = 2 * n if gated else n
    xq, wq = f.int8_codes((tokens, k), seed), f.int8_codes((rows, k), seed + 1)
    # scales that keep gates of a few units, as normalized activations do
    xs = (f.normal((tokens,), torch.float64, seed + 2).abs() * 0.01 + 1e-3).float()
    ws = (f.normal((rows,), torch.float64, seed + 3).abs() * 0.02 / k ** 0.5 + 1e-5).float()
    ops = [t.to(dev) for t in (xq, xs, wq, ws)]
    y = f.Guarded((tokens, n), dt, dev)
    if not gated:
        assert w4.gemm_int8(*ops, y=y.t) is y.t
        torch.cuda.synchronize()
        f.check(y.t, *f.int8_bound(xq, xs, wq, ws, dt))
        assert y.whole()
        return y.t
    pr = f.Guarded((tokens, 2 * n), dt, dev)
    w4.gated_int8(*ops, act=act, h=y.t, products=pr.t)
    torch.cuda.synchronize()
    both, e = f.int8_bound(xq, xs, wq, ws, torch.float32)
    h, eh, ep = f.block_bound(both, e, act, dt)
    f.check(y.t, h, eh)
    f.check(pr.t, both, ep)
    assert y.whole() and pr.whole()
    return y.t


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tokens,n,k", [(1, 1, 64), (1, 300, 1536), (2, 17, 128), (3, 64, 192), (7, 200, 8960), (16, 31, 320),
                                        (17, 129, 64), (32, 100, 448), (33, 64, 576), (64, 65, 256), (70, 500, 1024),
                                        (129, 257, 704), (300, 80, 192)])
def test_gemm_int8(tokens, n, k, out):
    _int8_case(tokens, n, k, out, seed=tokens)


@pytest.mark.parametrize("out", ["f16", "bf16"])
@pytest.mark.parametrize("tokens,n,k", [(1, 1, 64), (1, 150, 1536), (5, 33, 192), (16, 65, 320), (18, 20, 4160), (40, 130, 256),
                                        (70, 64, 448), (260, 90, 128)])
def test_gated_int8(tokens, n, k, out):
    _int8_case(tokens, n, k, out, gated=True, act=ACTS[n % 2], seed=tokens)


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("n,k", [(1, 64), (7, 1024), (30, 1088), (129, 4160), (17, 896), (2, 9024)])
@pytest.mark.parametrize("tokens", [1, 2, 3, 4, 5])
def test_int8_few_tokens(tokens, n, k, gated, out):
    """Around the bounds of the launches: tokens held, rows of a wave, rows of a KiB and more."""
    if not (gated and out == "f32"):
        _int8_case(tokens, n, k, out, gated=gated, act=ACTS[n % 2], seed=tokens + n)


def test_int8_many_tiles():
    _int8_case(1030, 4400, 128, "bf16", seed=3)
    _int8_case(1030, 8800, 192, "bf16", gated=True, seed=4)


def test_int8_longest_rows():
    """The largest sums that int32 holds: every code -128 over the longest rows."""
    w4, dev = _w4(), f.device()
    for tokens in (1, 40):
        xq = torch.full((tokens, w4.INT8_MAX_K), -128, dtype=torch.int8, device=dev)
        wq = torch.full((3, w4.INT8_MAX_K), -128, dtype=torch.int8, device=dev)
        y = w4.gemm_int8(xq, torch.ones(tokens, device=dev), wq, torch.ones(3, device=dev))
        assert (y == float(128 * 128 * w4.INT8_MAX_K)).all()
