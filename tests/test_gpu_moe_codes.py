"""The codes and scales of the expert kernels read out one by one, through both products of the layer.

x is one-hot, so a gate or up sum is one code times one scale; gate = 64 and silu(64) = 64 (1 + exp(-64) rounds to
1).  NF4 codes are held as two 16-bit terms after a factor.  Their bound: the two bf16 terms are off by at most
4.2e-7 over the sixteen codes (rms 1.8e-7, 3.4e-7 of the codes' rms), 2.74e-6 without the factor; the gate's and
the reading row's codes of 1 add 1.4 u each (u = 2^-24), and one result passes at most 11 roundings (its product's scale,
gate and up, the factor's reciprocal twice, the sums of three planes and of two terms, the weight): 14 u of its value
in all.  A kernel without the factor misses the bound at the code -0.525 (2.74e-6 against 8.6e-7)."""
import numpy as np
import pytest

import oracle
from tests import gpu_util as g
from tests import moe_util as mu

pytestmark = pytest.mark.gpu

# a wave per pair; shared products with packed planes, with three tiles; sorted pairs
LAUNCHES = [(1, 2, 1, 0), (2, 2, 1, 1), (9, 4, 2, 1), (40, 2, 2, 2), (150, 2, 2, 2)]
U = 2.0 ** -24


def _run(fmt, tokens, top_k, x, gu, gus, dn, dns):
    """The layer with weight 1 for each token's expert 1 (slot 0; the other slots absent)."""
    import bit_weight_only_w4_amd as w4

    ids = np.full((tokens, top_k), -1, np.int32)
    ids[:, 0] = 1
    pack = lambda nib: ((nib[..., 0::2] << 4) | nib[..., 1::2]).astype(np.uint8)
    c = dict(fmt=fmt, x=x, ids=ids, weights=np.ones((tokens, top_k), np.float32), gu=(pack(gu), gus), dn=(pack(dn), dns))
    return w4.moe(*mu.to_device(c, g.device())).cpu().numpy().astype(np.float64)


def _plan(fmt, tokens, hidden, inter, experts, top_k, kind):
    import bit_weight_only_w4_amd as w4

    g.device()
    assert w4.moe_plan(fmt, tokens, hidden, inter, experts, top_k)["kind"] == kind


def _one_hot(fmt, tokens, hidden, bits_f16, bits_bf16):
    x = np.zeros((tokens, hidden), np.uint16)
    cols = (np.arange(tokens) * 37 + 5) % hidden
    x[np.arange(tokens), cols] = bits_f16 if fmt.endswith("_f16") else bits_bf16
    return x, cols


def _nf4_bound(code):
    return 4.2e-7 + 14 * U * np.abs(code)


@pytest.mark.parametrize("fmt", ["nf4_f16", "nf4_bf16"])
@pytest.mark.parametrize("tokens,experts,top_k,kind", LAUNCHES)
def test_nf4_codes_of_up_rows(fmt, tokens, experts, top_k, kind):
    hidden, inter = 320, 192
    _plan(fmt, tokens, hidden, inter, experts, top_k, kind)
    rng = np.random.default_rng(tokens)
    book = oracle.nf4_codebook().astype(np.float64)
    x, cols = _one_hot(fmt, tokens, hidden, 0x3C00, 0x3F80)
    gu = np.full((experts, 2 * inter, hidden), 15)
    gu[:, inter:] = rng.integers(0, 16, (experts, inter, hidden))
    gu[:, inter:inter + 16] = np.arange(16)[:, None]
    gus = np.ones((experts, 2 * inter, hidden // 64), np.float32)
    gus[:, :inter] = 64.0
    dn = np.full((experts, hidden, inter), 7)  # the code 0
    dn[:, np.arange(inter), np.arange(inter)] = 15
    dns = np.ones((experts, hidden, inter // 64), np.float32)
    y = _run(fmt, tokens, top_k, x, gu, gus, dn, dns)
    for t in range(tokens):
        want = book[gu[1, inter:, cols[t]]]
        assert np.all(np.abs(y[t, :inter] / 64 - want) <= _nf4_bound(want)), t
        assert np.all(y[t, inter:] == 0.0)


@pytest.mark.parametrize("fmt", ["nf4_f16", "nf4_bf16"])
@pytest.mark.parametrize("tokens,experts,top_k,kind", LAUNCHES)
def test_nf4_codes_of_down_rows(fmt, tokens, experts, top_k, kind):
    hidden, inter = 320, 192
    _plan(fmt, tokens, hidden, inter, experts, top_k, kind)
    rng = np.random.default_rng(tokens)
    book = oracle.nf4_codebook().astype(np.float64)
    x, _ = _one_hot(fmt, tokens, hidden, 0x3C00, 0x3F80)
    row = 101  # the one row of h that is not zero
    gu = np.full((experts, 2 * inter, hidden), 7)
    gu[:, [row, inter + row]] = 15
    gus = np.full((experts, 2 * inter, hidden // 64), 64.0, np.float32)
    gus[:, inter:] = 1.0
    dn = rng.integers(0, 16, (experts, hidden, inter))
    dn[:, :16, row] = np.arange(16)
    dns = np.ones((experts, hidden, inter // 64), np.float32)
    y = _run(fmt, tokens, top_k, x, gu, gus, dn, dns)
    want = book[dn[1, :, row]]
    for t in range(tokens):
        assert np.all(np.abs(y[t] / 64 - want) <= _nf4_bound(want)), t


@pytest.mark.parametrize("fmt", ["mxfp4_f16", "mxfp4_bf16"])
@pytest.mark.parametrize("tokens,experts,top_k,kind", LAUNCHES)
@pytest.mark.parametrize("hidden,inter", [(256, 256), (1088, 320)])
@pytest.mark.parametrize("first,gate_byte,shift", [(0, 133, 0), (64, 141, 8)])
def test_mxfp4_scale_bytes_of_up_rows(fmt, tokens, experts, top_k, kind, hidden, inter, first, gate_byte, shift):
    """Up row n has the scale byte first + n % (255 - first), up to 254, and x is 2^-shift: every value is a
    code times a power of two inside fp32's range and comes out exactly."""
    _plan(fmt, tokens, hidden, inter, experts, top_k, kind)
    rng = np.random.default_rng(tokens + hidden)
    book = oracle.fp4_codebook().astype(np.float64)
    x, cols = _one_hot(fmt, tokens, hidden, (15 - shift) << 10, (127 - shift) << 7)
    gu = np.full((experts, 2 * inter, hidden), 2)  # the code 1
    gu[:, inter:] = rng.integers(0, 16, (experts, inter, hidden))
    byte = first + np.arange(inter) % ((200 if first == 0 else 255) - first)
    gus = np.full((experts, 2 * inter, hidden // 32), gate_byte, np.uint8)
    gus[:, inter:] = byte[None, :, None]
    dn = np.zeros((experts, hidden, inter), np.int64)
    n = min(hidden, inter)
    dn[:, np.arange(n), np.arange(n)] = 2
    dns = np.full((experts, hidden, inter // 32), 121, np.uint8)  # 2^-6: the gate's 64 taken off
    y = _run(fmt, tokens, top_k, x, gu, gus, dn, dns)
    for t in range(tokens):
        want = book[gu[1, inter:, cols[t]]] * 2.0 ** (byte - 127.0 - shift)
        assert np.array_equal(y[t, :n], want[:n]), t


@pytest.mark.parametrize("fmt", ["mxfp4_f16", "mxfp4_bf16"])
@pytest.mark.parametrize("tokens,experts,top_k,kind", LAUNCHES)
@pytest.mark.parametrize("hidden,inter", [(256, 256), (320, 1088)])
def test_mxfp4_scale_bytes_of_down_rows(fmt, tokens, experts, top_k, kind, hidden, inter):
    """Down row n has the scale byte n % 255 and h is one-hot 1: exact, and infinite past fp32's range."""
    _plan(fmt, tokens, hidden, inter, experts, top_k, kind)
    rng = np.random.default_rng(tokens + inter)
    book = oracle.fp4_codebook().astype(np.float64)
    x, _ = _one_hot(fmt, tokens, hidden, 0x3C00, 0x3F80)
    row = inter - 27
    gu = np.zeros((experts, 2 * inter, hidden), np.int64)
    gu[:, [row, inter + row]] = 2
    gus = np.full((experts, 2 * inter, hidden // 32), 133, np.uint8)  # gate 64
    gus[:, inter:] = 121                                              # up 2^-6
    dn = rng.integers(0, 16, (experts, hidden, inter))
    byte = np.arange(hidden) % 255
    dns = np.repeat(byte.astype(np.uint8)[None, :, None], inter // 32, axis=2).repeat(experts, axis=0)
    y = _run(fmt, tokens, top_k, x, gu, gus, dn, dns)
    with np.errstate(over="ignore"):
        want = (book[dn[1, :, row]] * 2.0 ** (byte - 127.0)).astype(np.float32).astype(np.float64)
    for t in range(tokens):
        assert np.array_equal(y[t], want), t
