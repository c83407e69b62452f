"""Infinities and NaN in the expert layer: they come where the definition has them, and nowhere else.

The expected values are the definition's in fp64: a product of zero and infinity is NaN, a sum of infinities of both
signs is NaN, h is kept in fp32's range.  Outputs that are finite by the definition are finite here and inside
the layer's error bound (tests/moe_util.py)."""
import numpy as np
import pytest

import oracle
from tests import gpu_util as g
from tests import moe_util as mu

pytestmark = pytest.mark.gpu

FMTS = [f"{w}_{x}" for w in ("nf4", "int4", "fp4", "int4a", "mxfp4") for x in ("f16", "bf16")]
# a wave per pair; shared products with packed planes, with three tiles; sorted pairs
LAUNCHES = [(1, 2, 2, 0), (2, 2, 1, 1), (9, 4, 2, 1), (40, 2, 2, 2), (150, 2, 2, 2)]
GROUP = {"nf4": 64, "fp4": 64, "int4": 128, "int4a": 128, "mxfp4": 32}
POSITIVE = {"nf4": (8, 15), "fp4": (1, 7), "int4": (9, 15), "int4a": (6, 15), "mxfp4": (1, 7)}
NEGATIVE = {"nf4": (0, 6), "fp4": (9, 15), "int4": (0, 7), "int4a": (0, 4), "mxfp4": (9, 15)}  # int4a: z = 5


def _scales(weight, value):
    """Powers of two `value` [rows, K / group] in the format's storage (int4a: zero point 5)."""
    value = np.asarray(value, dtype=np.float64)
    if weight == "mxfp4":
        return (np.log2(value).astype(np.int64) + 127).astype(np.uint8)
    if weight in ("nf4", "fp4"):
        return value.astype(np.float32)
    bits = oracle.f32_to_bf16_rne_bits(value.astype(np.float32))
    return bits.astype(np.uint16) if weight == "int4" else (bits.astype(np.uint32) | (5 << 16))


def _matrix(weight, nibbles, scale):
    """(packed, scales, fp64 weights, magnitudes) of nibbles [E, N, K] and power-of-two scales [E, N, K / group]."""
    e, n, k = nibbles.shape
    flat = nibbles.reshape(e * n, k).astype(np.uint8)
    packed = (flat[:, 0::2] << 4) | flat[:, 1::2]
    s = _scales(weight, scale.reshape(e * n, -1))
    hat = oracle.dequant(weight, packed, s).reshape(e, n, k)
    sc = np.repeat(scale, GROUP[weight], axis=2)
    mag = np.abs(hat) if weight[:3] != "int" else hat + (32 + 2 * (5 if weight == "int4a" else 8)) * sc
    return packed.reshape(e, n, k // 2), s.reshape(e, n, -1), hat, mag


def _layer(fmt, tokens, experts, top_k, seed, hidden=384, inter=256):
    """Nibbles and scales of a layer that a test changes before it is put together."""
    weight, xdt = fmt.split("_")
    rng = np.random.default_rng(seed)
    grp = GROUP[weight]
    ids = np.stack([rng.permutation(experts)[:top_k] for _ in range(tokens)]).astype(np.int32)
    x = rng.standard_normal((tokens, hidden)).astype(np.float32)
    bits = oracle.f32_to_bf16_rne_bits(x).astype(np.uint16) if xdt == "bf16" else x.astype(np.float16).view(np.uint16)
    return dict(fmt=fmt, x=bits, ids=ids, weights=(0.25 + rng.random((tokens, top_k))).astype(np.float32),
                gn=rng.integers(0, 16, (experts, 2 * inter, hidden)), gs=np.full((experts, 2 * inter, hidden // grp), 2.0 ** -5),
                dnib=rng.integers(0, 16, (experts, hidden, inter)), ds=np.full((experts, hidden, inter // grp), 2.0 ** -5))


def _expected(c):
    """The definition in fp64, h in fp32's range."""
    x = oracle.x_bits_to_f64(c["x"], c["fmt"].split("_")[1])
    gu, dn = c["gu"][2], c["dn"][2]
    inter = dn.shape[2]
    y = np.zeros((x.shape[0], dn.shape[1]))
    with np.errstate(all="ignore"):
        for t in range(x.shape[0]):
            for j, e in enumerate(c["ids"][t]):
                both = (gu[e] * x[t]).sum(1)
                gate, up = both[:inter], both[inter:]
                h = gate / (1 + np.exp(-gate)) * up
                h = np.where(np.abs(h) > 3.4e38, np.copysign(np.inf, h), h)
                y[t] += float(c["weights"][t, j]) * (dn[e] * h).sum(1)
    return y


def _check(c, need):
    """Runs the layer; `need` names the kinds of outputs that have to be among the expected ones."""
    import bit_weight_only_w4_amd as w4

    weight = c["fmt"].split("_")[0]
    c["gu"], c["dn"] = _matrix(weight, c["gn"], c["gs"]), _matrix(weight, c["dnib"], c["ds"])
    want = _expected(c)
    kinds = dict(nan=np.isnan(want), plus=want == np.inf, minus=want == -np.inf, finite=np.isfinite(want))
    for k in need:
        assert kinds[k].any(), k
    got = w4.moe(*mu.to_device(c, g.device())).cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), kinds["nan"])
    assert np.array_equal(got == np.inf, kinds["plus"]) and np.array_equal(got == -np.inf, kinds["minus"])
    rows = np.flatnonzero(kinds["finite"].all(1))
    if rows.size:
        with np.errstate(all="ignore"):
            ref, bound = mu.reference(c)
        assert np.all(np.abs(got[rows] - ref[rows]) <= bound[rows])


def _signed(rng, weight, sign, shape):
    lo, hi = (POSITIVE if sign > 0 else NEGATIVE)[weight]
    return rng.integers(lo, hi + 1, shape)


def _overflow_in(c, row):
    """Large scales in gate and up row `row`; a large activation meets the gate row's largest code: gate > 0."""
    for r in (row, c["dnib"].shape[2] + row):
        c["gs"][:, r] = 2.0 ** 80
    weight, xdt = c["fmt"].split("_")
    c["x"][:, 5] = np.float16(50).view(np.uint16) if xdt == "f16" else 0x4248
    c["gn"][:, row, 5] = POSITIVE[weight][1]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,experts,top_k,kind", LAUNCHES)
def test_infinite_activations(fmt, tokens, experts, top_k, kind):
    """Gate and up rows have positive codes at the infinite column, so h is +inf throughout; down rows of one sign
    give its infinity, rows of both signs or with a code of zero NaN."""
    import bit_weight_only_w4_amd as w4

    c = _layer(fmt, tokens, experts, top_k, seed=tokens)
    hidden, inter = c["dnib"].shape[1:]
    g.device()
    assert w4.moe_plan(fmt, tokens, hidden, inter, experts, top_k)["kind"] == kind
    rng = np.random.default_rng(1)
    weight = fmt.split("_")[0]
    col = 77
    c["gn"][:, :, col] = _signed(rng, weight, 1, c["gn"].shape[:2])
    c["dnib"][:, 0:20] = _signed(rng, weight, 1, (experts, 20, inter))
    c["dnib"][:, 20:40] = _signed(rng, weight, -1, (experts, 20, inter))
    odd = sorted({0, tokens // 2, tokens - 1})
    for t in odd:
        c["x"][t, col] = 0x7C00 if fmt.endswith("_f16") else 0x7F80
    _check(c, ["nan", "plus", "minus"] + (["finite"] if tokens > len(odd) else []))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,experts,top_k,kind", LAUNCHES)
def test_products_between_the_matrices_past_fp32(fmt, tokens, experts, top_k, kind):
    """One gate and up row whose product leaves fp32's range: that h is infinite, the others finite."""
    c = _layer(fmt, tokens, experts, top_k, seed=tokens + 1)
    _overflow_in(c, 30)
    _check(c, ["plus", "minus"])


@pytest.mark.parametrize("fmt", ["nf4_bf16", "int4_bf16", "int4a_bf16", "fp4_bf16", "mxfp4_bf16"])
@pytest.mark.parametrize("tokens,experts,top_k,kind", LAUNCHES)
@pytest.mark.parametrize("exponent", [120, 124, 125])
def test_activations_at_the_top_of_the_range(fmt, tokens, experts, top_k, kind, exponent):
    """One activation near bf16's largest and small scales: every sum of the definition is finite (codes are
    at most 15 in magnitude before their scale), and so is every output."""
    c = _layer(fmt, tokens, experts, top_k, seed=tokens + 2)
    c["x"][:] = 0
    c["x"][np.arange(tokens), np.arange(tokens) % c["x"].shape[1]] = (exponent + 127) << 7 | 0x3F
    c["gs"][:] = 2.0 ** (2 - exponent)
    _check(c, ["finite"])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,experts,top_k,kind", LAUNCHES)
def test_nan_activations_stay_in_their_token(fmt, tokens, experts, top_k, kind):
    c = _layer(fmt, tokens, experts, top_k, seed=tokens + 3)
    c["x"][tokens - 1, 300] = 0x7FFF
    _check(c, ["nan"] + (["finite"] if tokens > 1 else []))


@pytest.mark.parametrize("fmt", ["nf4_f16", "int4_bf16", "int4a_f16"])
@pytest.mark.parametrize("tokens,hidden,inter,experts,top_k", [(1, 2432, 1664, 2, 1), (5, 2432, 1280, 4, 1),
                                                               (14, 512, 2432, 4, 2), (40, 1280, 640, 2, 1)])
def test_long_rows(fmt, tokens, hidden, inter, experts, top_k):
    """K ranges, windows and several quads."""
    c = _layer(fmt, tokens, experts, top_k, seed=5, hidden=hidden, inter=inter)
    rng = np.random.default_rng(2)
    weight = fmt.split("_")[0]
    c["gn"][:, :, hidden - 3] = _signed(rng, weight, 1, c["gn"].shape[:2])
    c["dnib"][:, 100:300] = _signed(rng, weight, -1, (experts, 200, inter))
    c["x"][0, hidden - 3] = 0x7C00 if fmt.endswith("_f16") else 0x7F80
    _check(c, ["nan", "minus"])
    c["x"][0, hidden - 3] = 0
    _overflow_in(c, inter - 1)
    _check(c, ["plus", "minus"])
