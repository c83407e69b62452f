"""Pins of the oracle's MXFP4 (E2M1 codes, one power-of-two scale byte per 32 weights)."""
import numpy as np
import pytest

import oracle
import synth_inputs


def test_code_points_round_trip_at_every_scale():
    """Weights that are code points times 2^e, with the top code in each block, come back exactly."""
    rng = np.random.default_rng(0)
    grid = oracle.fp4_codebook().astype(np.float64)
    for e in (-120, -20, -3, 0, 5, 100):
        w = grid[rng.integers(0, 16, (7, 128))]
        w[:, ::32] = 6.0
        w = (w * 2.0 ** e).astype(np.float32)
        p, s = oracle.quantize_mxfp4(w)
        assert np.all(s == e + 127)
        assert np.array_equal(oracle.dequant_mxfp4(p, s), w.astype(np.float64))


def test_rounding_is_within_half_a_step():
    """Inside the grid a magnitude moves by at most half its interval; above 6 * 2^e (the block's
    maximum may reach just under 8 * 2^e) it saturates to 6 * 2^e."""
    w = synth_inputs.weights(64, 512, seed=1)
    p, s = oracle.quantize_mxfp4(w)
    step = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=1)
    r, q = np.abs(w) / step, np.abs(oracle.dequant_mxfp4(p, s)) / step
    assert np.all(r < 8.0)
    half = np.where(r < 2, 0.25, np.where(r < 4, 0.5, 1.0))
    inside = r <= 6
    assert np.all(np.abs(r - q)[inside] <= half[inside])
    assert np.all(q[~inside] == 6.0)


@pytest.mark.parametrize("ratio,code", [(0.25, 0.0), (0.75, 1.0), (1.25, 1.0), (1.75, 2.0), (2.5, 2.0),
                                        (3.5, 4.0), (5.0, 4.0), (7.99, 6.0)])
def test_ties_go_to_even_codes(ratio, code):
    w = np.zeros((1, 64), dtype=np.float32)
    w[0, 0], w[0, 1], w[0, 2] = 4.0, ratio, -ratio  # scale 1
    p, s = oracle.quantize_mxfp4(w)
    assert s[0, 0] == 127
    d = oracle.dequant_mxfp4(p, s)
    assert d[0, 1] == code and d[0, 2] == -code


def test_zero_and_subnormal_blocks():
    w = np.zeros((1, 64), dtype=np.float32)
    w[0, 32] = np.float32(2.0 ** -140)  # far below the smallest scale
    w[0, 33] = np.float32(2.0 ** -127)
    p, s = oracle.quantize_mxfp4(w)
    assert np.all(s == 0) and np.all(p[0, :16] == 0)
    d = oracle.dequant_mxfp4(p, s)
    assert d[0, 32] == 0.0 and d[0, 33] == 2.0 ** -127


def test_nan_scale_and_layout():
    p = np.full((1, 32), 0x2F, dtype=np.uint8)  # 1.0 then -6.0
    s = np.array([[128, 255]], dtype=np.uint8)
    d = oracle.dequant_mxfp4(p, s)
    assert np.array_equal(d[0, :4], [2.0, -12.0, 2.0, -12.0]) and np.all(np.isnan(d[0, 32:]))
    with pytest.raises(ValueError):
        oracle.quantize_mxfp4(np.full((1, 64), np.inf, dtype=np.float32))
    with pytest.raises(ValueError):
        oracle.quantize_mxfp4(np.zeros((1, 96), dtype=np.float32))
