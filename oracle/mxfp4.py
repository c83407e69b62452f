"""MXFP4 of the oracle: E2M1 codes in blocks of 32 along K, one E8M0 scale byte per block.

Test infrastructure only (see the package docstring).

The block form of the OCP microscaling formats (OCP Microscaling Formats specification 1.0):
a block's scale is a power of two, 2^(e - 127) for the stored byte e (255 is NaN), and its
elements are E2M1.  Quantization takes e - 127 = floor(log2(max |w|)) - 2, 2 being E2M1's largest
exponent, and rounds |w| / 2^(e - 127) to the nearest code, ties to even codes, magnitudes past the
grid to its last (quotients lie below 8).  An all-zero block stores byte 0.  Sign bit = (w < 0),
nibble order and the code table as in ``oracle.fp4``.
"""
from __future__ import annotations

import numpy as np

from .fp4 import fp4_codebook, fp4_magnitude_index

MXFP4_BLOCK = 32


def quantize_mxfp4(w: np.ndarray):
    """Quantize fp32 ``w[N, K]``: ``(packed uint8[N, K/2], scale uint8[N, K/32])``."""
    w = np.ascontiguousarray(w, dtype=np.float32)
    n, k = w.shape
    if n < 1 or k < 1 or k % 64:
        raise ValueError("K must be a positive multiple of 64")
    if not np.all(np.isfinite(w)):
        raise ValueError("non-finite weight")
    blocks = w.astype(np.float64).reshape(n, k // MXFP4_BLOCK, MXFP4_BLOCK)
    absmax = np.abs(blocks).max(axis=2)
    _, exponent = np.frexp(absmax)  # absmax = m 2^exponent, 1/2 <= m < 1
    e = np.where(absmax > 0.0, np.clip(exponent - 1 - 2, -127, 127), -127)
    mag = fp4_magnitude_index(np.abs(blocks) / np.ldexp(1.0, e)[..., None])
    nib = (mag | np.where(blocks < 0.0, 8, 0).astype(np.uint8)).astype(np.uint8).reshape(n, k)
    packed = ((nib[:, 0::2] << 4) | nib[:, 1::2]).astype(np.uint8)
    return packed, (e + 127).astype(np.uint8)


def dequant_mxfp4(packed: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """fp64 [N, K] decoded weights (exact; NaN where the scale byte is 255)."""
    from .gemv import unpack_nibbles

    idx = unpack_nibbles(packed)
    s = np.asarray(scale, dtype=np.uint8)
    if s.shape != (idx.shape[0], idx.shape[1] // MXFP4_BLOCK):
        raise ValueError("scale shape does not match [N, K/32]")
    value = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 127))
    return fp4_codebook().astype(np.float64)[idx] * np.repeat(value, MXFP4_BLOCK, axis=1)
