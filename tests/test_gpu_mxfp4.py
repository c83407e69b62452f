"""MXFP4 on the GPU: the quantizer bit for bit against the oracle, and every product against fp64.

Tolerance of the products.  Codes are exact in both 16-bit types, products of two 16-bit values are
exact in fp32 and scales are powers of two, so y differs from the fp64 product by fp32 accumulation
alone: along any path of a sum at most 32 additions inside a block, K/32 block additions and 32 of
the lane, wave, workgroup and split sums, each within 2^-24 of a partial sum that
T = sum_k |x_k w_k| bounds.  Hence |y - y_ref| <= (K/32 + 64) 2^-24 T (one in-order bound for every
kernel), plus 2^-126 for scales at the bottom of the range.
"""
import numpy as np
import pytest

import oracle
import synth_inputs
from tests import gpu_util as g

pytestmark = pytest.mark.gpu

FMTS = ["mxfp4_f16", "mxfp4_bf16"]


def _xdt(fmt):
    return fmt.split("_")[1]


def _check(y, x_bits, fmt, p, s, rows=None):
    w_hat = oracle.dequant_mxfp4(p, s)
    ref, t = oracle.gemv_reference(x_bits, _xdt(fmt), w_hat)
    bound = (w_hat.shape[1] / 32 + 64) * 2.0 ** -24 * t + 2.0 ** -126
    got = y.cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got))
    worst = np.max(np.abs(got - ref) / bound)
    assert worst <= 1.0, worst


def _case(fmt, n, k, b, seed, spread=0):
    import torch

    import bit_weight_only_w4_amd as w4

    w = synth_inputs.weights(n, k, seed=seed)
    if spread:  # block scales over many binades
        e = np.random.default_rng(seed).integers(-spread, spread + 1, (n, k // 32))
        w = (w * np.repeat(2.0 ** e, 32, axis=1)).astype(np.float32)
    x = synth_inputs.activations(b, k, _xdt(fmt), seed=seed + 1)
    p, s = w4.quantize(fmt, g.to_dev_f32(w))
    pr, sr = oracle.quantize_mxfp4(w)
    assert np.array_equal(p.cpu().numpy(), pr) and np.array_equal(s.cpu().numpy(), sr)
    assert s.dtype == torch.uint8
    return x, g.to_dev_x(x, _xdt(fmt)), p, s, pr, sr


def test_quantizer_bitexact_on_hard_blocks():
    import bit_weight_only_w4_amd as w4

    rng = np.random.default_rng(3)
    w = (rng.standard_normal((64, 512)) * np.exp2(rng.integers(-60, 60, (64, 512)))).astype(np.float32)
    w[0] = 0.0
    w[1] = -0.0
    w[2] = np.float32(2.0 ** -149)  # subnormal
    w[3] = np.float32(3.4028235e38)
    w[4] = np.tile(np.float32([4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5, -0.25, 7.99, -6, 0, 1, 2, 3]), 32)
    w[5] = np.float32(2.0 ** -126) * w[4]
    p, s = w4.quantize_mxfp4(g.to_dev_f32(w))
    pr, sr = oracle.quantize_mxfp4(w)
    assert np.array_equal(s.cpu().numpy(), sr)
    assert np.array_equal(p.cpu().numpy(), pr)


def test_quantizer_reports_nonfinite():
    import bit_weight_only_w4_amd as w4

    for bad in (np.nan, np.inf, -np.inf):
        w = synth_inputs.weights(5, 128, seed=1)
        w[4, 127] = bad
        with pytest.raises(w4.W4ValueError) as e:
            w4.quantize_mxfp4(g.to_dev_f32(w))
        assert e.value.status == -5


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,k,b", [(1, 64, 1), (33, 64, 8), (256, 1536, 1), (300, 1536, 3), (129, 8960, 5),
                                   (70, 320, 8), (8960, 1536, 1), (257, 16448, 2), (64, 28672, 1)])
def test_gemv(fmt, n, k, b):
    import bit_weight_only_w4_amd as w4

    x, xd, p, s, pr, sr = _case(fmt, n, k, b, seed=n + k + b)
    _check(w4.gemv(xd, p, s, fmt), x, fmt, pr, sr)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,k,b", [(1, 64, 1), (17, 192, 16), (300, 1536, 9), (130, 8960, 33), (77, 2048, 64),
                                   (1000, 320, 128), (45, 1600, 257), (5000, 512, 130), (16, 64, 4096)])
def test_mfma_and_the_automatic_choice(fmt, n, k, b):
    import bit_weight_only_w4_amd as w4

    x, xd, p, s, pr, sr = _case(fmt, n, k, b, seed=n + k + b, spread=6)
    _check(w4.matmul_ex(xd, p, s, fmt, path="mfma"), x, fmt, pr, sr)
    _check(w4.gemm_smallbatch(xd, p, s, fmt), x, fmt, pr, sr)
    _check(w4.gemm_prefill(xd, p, s, fmt), x, fmt, pr, sr)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("path,split,n,k,b", [("splitk", 4, 300, 1536, 2), ("splitk", 16, 129, 8960, 8),
                                              ("mfma", 4, 300, 8960, 16), ("mfma", 3, 77, 1088, 40)])
def test_k_ranges(fmt, path, split, n, k, b):
    import torch

    import bit_weight_only_w4_amd as w4

    x, xd, p, s, pr, sr = _case(fmt, n, k, b, seed=k + b)
    ws = torch.empty(w4.workspace_bytes(fmt, n, k, b, path, split), dtype=torch.uint8, device=g.device())
    _check(w4.matmul_ex(xd, p, s, fmt, path=path, split_k=split, workspace=ws), x, fmt, pr, sr)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("b", [1, 8, 32, 160])
def test_grouped_launches(fmt, b):
    import bit_weight_only_w4_amd as w4

    k = 1536
    cases = [_case(fmt, n, k, b, seed=5) for n in (1536, 256, 4100)]  # same seed: the same x
    xd = cases[0][1]
    for entry in (w4.gemm_smallbatch_grouped,) + ((w4.gemv_grouped,) if b <= 8 else ()):
        for c, y in zip(cases, entry(xd, [c[2] for c in cases], [c[3] for c in cases], fmt)):
            _check(y, c[0], fmt, c[4], c[5])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("path,b", [("gemv", 1), ("mfma", 16)])
def test_one_hot_exact_over_the_scale_range(fmt, path, b):
    """x = e_j returns column j exactly for every scale byte but 255 (also 0, 2^-127), as fp32 holds
    it: at byte 253 the codes 4 and 6 stand for 4 * 2^126 = 2^128 and more, past the largest fp32
    (2^128 - 2^104), and come out as infinities."""
    import torch

    import bit_weight_only_w4_amd as w4

    n, k = 254, 128
    rng = np.random.default_rng(8)
    pr = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
    sr = np.tile(np.arange(n, dtype=np.uint8)[:, None], (1, k // 32))  # rows 0..253: bytes 0..253
    w_hat = oracle.dequant_mxfp4(pr, sr)
    p, s = (torch.from_numpy(v).to(g.device()) for v in (pr, sr))
    xb = np.zeros((b, k), dtype=np.uint16)
    cols = [(37 * i + 5) % k for i in range(b)]
    for i, c in enumerate(cols):
        xb[i, c] = 0x3C00 if _xdt(fmt) == "f16" else 0x3F80
    y = w4.matmul_ex(g.to_dev_x(xb, _xdt(fmt)), p, s, fmt, path=path).cpu().numpy()
    for i, c in enumerate(cols):
        with np.errstate(over="ignore"):
            assert np.array_equal(y[i], w_hat[:, c].astype(np.float32))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("path,b", [("gemv", 2), ("mfma", 20)])
def test_nan_scale_and_nonfinite_activations_stay_in_their_rows(fmt, path, b):
    import torch

    import bit_weight_only_w4_amd as w4

    x, xd, p, s, pr, sr = _case(fmt, 50, 320, b, seed=4)
    s = s.clone()
    s[7, 3] = 255
    xd[1, 100] = float("nan")
    y = w4.matmul_ex(xd, p, s, fmt, path=path)
    assert torch.isnan(y[:, 7]).all() and torch.isnan(y[1]).all()
    keep_n = [i for i in range(50) if i != 7]
    keep_b = [i for i in range(b) if i != 1]
    _check(y[keep_b][:, keep_n], x[keep_b], fmt, pr[keep_n], sr[keep_n])


@pytest.mark.parametrize("fmt", FMTS)
def test_noalloc_split(fmt):
    import ctypes

    import torch

    import bit_weight_only_w4_amd as w4

    x, xd, p, s, pr, sr = _case(fmt, 300, 1536, 3, seed=6)
    y = torch.full((3, 300), float("nan"), device=g.device())
    vp = ctypes.c_void_p
    assert w4.lib().w4_matmul_splitk_noalloc(vp(xd.data_ptr()), vp(p.data_ptr()), vp(s.data_ptr()),
                                             w4.FORMATS[fmt], 300, 1536, 3, vp(y.data_ptr()), 4, None) == 0
    torch.cuda.synchronize()
    _check(y, x, fmt, pr, sr)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,k,b", [(33, 64, 16), (17, 1088, 5), (50, 320, 70), (300, 192, 2), (40, 4160, 130)])
def test_scales_that_start_inside_a_dword(fmt, n, k, b):
    """Rows 1 .. n of a matrix whose rows hold an odd number of scale pairs: the scales of the part start two bytes
    into a dword.  The bytes around them are 255 and must not be used.  Alone, and in a group beside a
    matrix whose scales start on a dword."""
    import torch

    import bit_weight_only_w4_amd as w4

    assert (k // 32) % 4 == 2
    x, xd, p, s, pr, sr = _case(fmt, n + 2, k, b, seed=n + k, spread=3)
    clean = s.clone()
    s[0] = 255
    s[-1] = 255
    part, scales = p[1:-1], s[1:-1]
    assert scales.data_ptr() % 4 == 2
    paths = ["mfma"] + (["gemv"] if b <= 8 else [])
    for path in paths:
        _check(w4.matmul_ex(xd, part, scales, fmt, path=path), x, fmt, pr[1:-1], sr[1:-1])
    _check(w4.gemm_smallbatch(xd, part, scales, fmt), x, fmt, pr[1:-1], sr[1:-1])
    torch.cuda.synchronize()
    ys = w4.gemm_smallbatch_grouped(xd, [part, p, part], [scales, clean, scales], fmt)
    _check(ys[0], x, fmt, pr[1:-1], sr[1:-1])
    _check(ys[1], x, fmt, pr, sr)
    _check(ys[2], x, fmt, pr[1:-1], sr[1:-1])
