"""Seeded inputs and the plain fp64 mixture-of-experts layer of the tests, with its error bound.

The bound is the sum of the layer's roundings, each taken at its largest.  With u = 2^-24:

* a sum over K of one matrix: |d| <= eps(K) T, eps(K) = (K/32 + 64) u and T the sum of the
  magnitudes of its terms (32 additions inside a block, K/32 block additions, 32 for the sums over
  waves and column planes); the integer formats add (16 + q) x and -(16 + z) x (z = 8 for INT4)
  apart, so their terms are |x| s (32 + q + z).  Products are exact in fp32 except the scale's (2 u, inside the
  64), NF4's codes are two 16-bit terms, off by at most 2^-18 |code|;
* silu has |silu'| <= 1.1; exp, the division and two products are off by at most 2^-20 |h|;
* h is kept whole; the sum over slots adds (top_k + 2) u of its magnitudes;
* 2^-126 for results below the normal numbers, times K.
"""
import numpy as np

import oracle
import synth_inputs

U = 2.0 ** -24


def quantize_experts(weight, w):
    """fp32 [E, N, K] -> packed, scales and the fp64 weights, term magnitudes of the oracle."""
    e, n, k = w.shape
    q = {"nf4": oracle.quantize_nf4, "int4": oracle.quantize_int4, "fp4": oracle.quantize_fp4,
         "int4a": oracle.quantize_int4_asym, "mxfp4": oracle.quantize_mxfp4}[weight]
    p, s = q(w.reshape(e * n, k))
    hat = oracle.dequant(weight, p, s).reshape(e, n, k)
    mag = np.abs(hat)
    if weight in ("int4", "int4a"):
        sc = np.repeat(oracle.bf16_bits_to_f64((s & 0xFFFF).astype(np.uint16)), 128, axis=1).reshape(e, n, k)
        z = np.repeat((s >> 16) & 15, 128, axis=1).astype(np.float64).reshape(e, n, k) if weight == "int4a" else 8.0
        mag = hat + (32 + 2 * z) * sc  # s (16 + q) + s (16 + z), hat = s (q - z)
    return p.reshape(e, n, k // 2), s.reshape(e, n, -1), hat, mag


def case(fmt, tokens, hidden, inter, experts, top_k, seed, sigma=0.05):
    """Host arrays of one layer: x bits, ids, weights, and both quantized matrices."""
    weight, xdt = fmt.split("_")
    rng = np.random.default_rng(seed)
    gu = synth_inputs.weights(experts * 2 * inter, hidden, sigma=sigma, seed=seed).reshape(experts, 2 * inter, hidden)
    dn = synth_inputs.weights(experts * hidden, inter, sigma=sigma, seed=seed + 1).reshape(experts, hidden, inter)
    x = synth_inputs.activations(tokens, hidden, xdt, seed=seed + 2)
    ids = np.stack([rng.permutation(experts)[:top_k] if top_k <= experts else rng.integers(0, experts, top_k)
                    for _ in range(tokens)]).astype(np.int32)
    w = rng.random((tokens, top_k)).astype(np.float32)
    return dict(fmt=fmt, x=x, ids=ids, weights=w, gu=quantize_experts(weight, gu), dn=quantize_experts(weight, dn))


def _eps(k):
    return (k / 32 + 64) * U


def reference(c):
    """(y, bound) in fp64."""
    weight, xdt = c["fmt"].split("_")
    code = 2.0 ** -18 if weight == "nf4" else 0.0
    x = oracle.x_bits_to_f64(c["x"], xdt)
    (_, _, gu, gum), (_, _, dn, dnm) = c["gu"], c["dn"]
    experts, hidden, inter = dn.shape
    y = np.zeros((x.shape[0], hidden))
    bound = np.full_like(y, 2.0 ** -126 * inter)
    for t in range(x.shape[0]):
        for j, e in enumerate(c["ids"][t]):
            if e < 0 or e >= experts:
                continue
            w = float(c["weights"][t, j])
            both, mag = gu[e] @ x[t], gum[e] @ np.abs(x[t])
            d = (_eps(hidden) + code) * mag + 2.0 ** -126 * hidden
            g, u, dg, du = both[:inter], both[inter:], d[:inter], d[inter:]
            with np.errstate(over="ignore"):
                s = g / (1 + np.exp(-g))
            h = s * u
            dh = 1.1 * dg * (np.abs(u) + du) + np.abs(s) * du + 2.0 ** -20 * np.abs(h)
            out, om = dn[e] @ h, dnm[e] @ (np.abs(h) + dh)
            y[t] += w * out
            bound[t] += abs(w) * (np.abs(dn[e]) @ dh + (_eps(inter) + code + (c["ids"].shape[1] + 2) * U) * om)
    return y, bound


def to_device(c, dev):
    """The tensors of a w4.moe call, in order."""
    import torch

    xdt = torch.float16 if c["fmt"].endswith("_f16") else torch.bfloat16

    def mat(m):
        p, s = m[0], m[1]
        s = s.view(np.int16) if s.dtype == np.uint16 else s.view(np.int32) if s.dtype == np.uint32 else s
        return torch.from_numpy(p).to(dev), torch.from_numpy(np.ascontiguousarray(s)).to(dev)

    x = torch.from_numpy(c["x"].view(np.int16)).view(xdt).to(dev)
    return (x, torch.from_numpy(c["ids"]).to(dev), torch.from_numpy(c["weights"]).to(dev), *mat(c["gu"]),
            *mat(c["dn"]), c["fmt"])


def check(y, c, rows=None):
    ref, bound = reference(c)
    got = y.cpu().numpy().astype(np.float64)
    if rows is not None:
        ref, bound, got = ref[rows], bound[rows], got[rows]
    assert got.shape == ref.shape and np.all(np.isfinite(got))
    worst = float(np.max(np.abs(got - ref) / bound)) if got.size else 0.0
    assert worst <= 1.0, worst
    return worst
