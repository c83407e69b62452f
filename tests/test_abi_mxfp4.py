"""Host-side refusals of the MXFP4 format (no launch is made)."""
import ctypes

import pytest

FAKE = 0x10000  # a non-null, well-aligned address that is never dereferenced
F16, BF16 = 16, 17


def _lib():
    import bit_weight_only_w4_amd as w4

    return w4, w4.lib()


def vp(a):
    return ctypes.c_void_p(a)


def _ex(L, path, fmt=F16, n=64, k=256, b=1, split=0):
    return L.w4_matmul_ex(vp(FAKE), vp(FAKE * 2), vp(FAKE * 3), fmt, n, k, b, vp(FAKE * 4), path, split,
                          None, 0, None)


def test_quantizer_refusals():
    _, L = _lib()
    q = L.w4_quantize_mxfp4
    assert q(None, 4, 64, vp(FAKE * 2), vp(FAKE * 3), None) == -1
    assert q(vp(FAKE), 4, 64, vp(FAKE * 2), None, None) == -1
    assert q(vp(FAKE), 0, 64, vp(FAKE * 2), vp(FAKE * 3), None) == -2
    assert q(vp(FAKE), 4, 96, vp(FAKE * 2), vp(FAKE * 3), None) == -2
    assert q(vp(FAKE), 4, 64, vp(FAKE * 2 + 8), vp(FAKE * 3), None) == -3
    assert q(vp(FAKE), 4, 64, vp(FAKE * 2), vp(FAKE * 3 + 1), None) == -3
    assert q(vp(FAKE), 4, 64, vp(FAKE), vp(FAKE * 3), None) == -9


@pytest.mark.parametrize("fmt", [F16, BF16])
def test_shapes_alignment_and_paths(fmt):
    w4, L = _lib()
    assert L.w4_gemv(vp(FAKE), vp(FAKE * 2), vp(FAKE * 3), fmt, 64, 96, 1, vp(FAKE * 4), None) == -2
    assert L.w4_gemv(vp(FAKE), vp(FAKE * 2), vp(FAKE * 3 + 1), fmt, 64, 256, 1, vp(FAKE * 4), None) == -3
    assert L.w4_gemv(vp(FAKE), vp(FAKE * 2), vp(FAKE * 3), fmt, 64, 256, 1, vp(FAKE * 3), None) == -9
    for path in ("twopass", "tiled", "tiled_f16"):
        assert _ex(L, w4.PATHS[path], fmt) == -7
        assert L.w4_workspace_bytes(fmt, 64, 256, 1, w4.PATHS[path], 2) == 0
    assert _ex(L, w4.PATHS["splitk"], fmt, split=4) == -6  # no workspace
    for f in range(9, 16):
        assert _ex(L, 0, f) == -4
    assert _ex(L, 0, 18) == -4


def test_automatic_path_never_leaves_the_two_kernels():
    w4, _ = _lib()
    for n in (1, 256, 1536, 8960, 151936):
        for k in (64, 1536, 8960):
            for b in (1, 2, 8, 32, 128, 512, 4096):
                path, _ = w4.auto_path("mxfp4_f16", n, k, b, 1 << 30)
                assert path in ("gemv", "mfma")
    assert w4.weight_format("mxfp4_bf16") == "mxfp4"
