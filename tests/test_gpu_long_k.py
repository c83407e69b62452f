"""Products whose rows pass three chunks of 32 weights for each lane of the widest GEMV team (K > 49152)."""
import numpy as np
import pytest

import oracle
import synth_inputs
from tests import gpu_util as g

pytestmark = pytest.mark.gpu

FMTS = ["nf4_f16", "nf4_bf16", "int4_f16", "fp4_bf16", "int4a_bf16", "mxfp4_f16", "mxfp4_bf16"]


def _case(fmt, n, k, b, seed):
    import bit_weight_only_w4_amd as w4

    weight, xdt = fmt.split("_")
    w = synth_inputs.weights(n, k, seed=seed)
    p, s = w4.quantize(fmt, g.to_dev_f32(w))
    x = synth_inputs.activations(b, k, xdt, seed=seed + 1)
    quantizer = {"nf4": oracle.quantize_nf4, "int4": oracle.quantize_int4, "fp4": oracle.quantize_fp4,
                 "int4a": oracle.quantize_int4_asym, "mxfp4": oracle.quantize_mxfp4}[weight]
    pr, sr = quantizer(w)
    assert np.array_equal(p.cpu().numpy(), pr)
    return x, g.to_dev_x(x, xdt), p, s, oracle.gemv_reference(x, xdt, oracle.dequant(weight, pr, sr))


def _check(fmt, y, ref):
    assert oracle.violation_ratio(y.cpu().numpy().astype(np.float64), *ref) <= 1.0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,k,b", [(33, 49152, 1), (33, 49280, 1), (17, 65536, 1), (600, 65536, 1), (9, 131072, 1),
                                   (5, 131200, 1), (33, 65536, 2), (9, 65664, 2), (20, 65536, 3), (20, 65536, 8)])
def test_long_rows(fmt, n, k, b):
    import bit_weight_only_w4_amd as w4

    x, xd, p, s, ref = _case(fmt, n, k, b, seed=n + b)
    _check(fmt, w4.gemv(xd, p, s, fmt), ref)
    _check(fmt, w4.gemm_smallbatch(xd, p, s, fmt), ref)


@pytest.mark.parametrize("fmt", ["nf4_bf16", "mxfp4_f16"])
def test_long_rows_grouped(fmt):
    import bit_weight_only_w4_amd as w4

    k = 65536
    cases = [_case(fmt, n, k, 1, seed=5) for n in (33, 7)]
    for c, y in zip(cases, w4.gemv_grouped(cases[0][1], [c[2] for c in cases], [c[3] for c in cases], fmt)):
        _check(fmt, y, c[4])


@pytest.mark.parametrize("fmt", ["int4_f16", "mxfp4_bf16"])
@pytest.mark.parametrize("split", [2, 4])
def test_long_rows_in_ranges(fmt, split):
    import torch

    import bit_weight_only_w4_amd as w4

    n, k = 21, 131072
    x, xd, p, s, ref = _case(fmt, n, k, 1, seed=3)
    ws = torch.empty(w4.workspace_bytes(fmt, n, k, 1, "splitk", split), dtype=torch.uint8, device=g.device())
    _check(fmt, w4.matmul_ex(xd, p, s, fmt, path="splitk", split_k=split, workspace=ws), ref)


def test_mxfp4_matrix_past_4_gib():
    """131200 x 65536: more than 2^33 weights, packed bytes past 2^32 and two quantizer launches (rows of 2^32
    weights each); rows around every border against the oracle and the fp64 products."""
    import torch

    import bit_weight_only_w4_amd as w4

    dev = g.device()
    n, k = 131200, 65536
    w = torch.empty(n, k, device=dev)
    gen = torch.Generator(device=dev).manual_seed(2)
    for r in range(0, n, 16384):
        w[r:r + 16384].normal_(0.0, 0.02, generator=gen)
    p, s = w4.quantize_mxfp4(w)
    assert p.numel() > 2 ** 32
    rows = [0, 1, 65535, 65536, 65537, 131071, 131072, n - 17, n - 2, n - 1]
    pr, sr = oracle.quantize_mxfp4(w[rows].cpu().numpy())
    assert np.array_equal(p[rows].cpu().numpy(), pr) and np.array_equal(s[rows].cpu().numpy(), sr)
    del w
    hat = oracle.dequant_mxfp4(pr, sr)
    for b in (1, 3, 40):
        x = synth_inputs.activations(b, k, "bf16", seed=b)
        y = w4.gemm_smallbatch(g.to_dev_x(x, "bf16"), p, s, "mxfp4_bf16")
        ref, t = oracle.gemv_reference(x, "bf16", hat)
        got = y[:, rows].cpu().numpy().astype(np.float64)
        assert np.all(np.abs(got - ref) <= (k / 32 + 64) * 2.0 ** -24 * t + 2.0 ** -126), b
