"""Host-side refusals of the gated block, its gradients and the 8-bit products (no launch is made)."""
import ctypes

import pytest

FAKE = 0x100000  # a non-null, well-aligned address that is never dereferenced


def _lib():
    import bit_weight_only_w4_amd as w4

    return w4, w4.lib()


def vp(a):
    return ctypes.c_void_p(a)


def _gated(L, fmt=1, act=0, t=2, h=128, i=100, wsb=None, ws=FAKE * 9, **p):
    a = dict(x=FAKE, w=FAKE * 2, s=FAKE * 3, out=FAKE * 4, pr=FAKE * 5)
    a.update(p)
    if wsb is None:
        wsb = L.w4_gated_workspace_bytes(fmt, t, h, i)
    return L.w4_gated(vp(a["x"]), vp(a["w"]), vp(a["s"]), fmt, act, t, h, i, vp(a["out"]), vp(a["pr"]), vp(ws), wsb, None)


def test_gated_refusals():
    _, L = _lib()
    for name in ("x", "w", "s", "out"):
        assert _gated(L, **{name: 0}) == -1, name
    assert _gated(L, fmt=0) == -4 and _gated(L, fmt=9) == -4 and _gated(L, act=2) == -4 and _gated(L, act=-1) == -4
    for bad in (dict(t=0), dict(t=4097), dict(h=0), dict(h=96), dict(fmt=3, h=192), dict(fmt=8, h=64),
                dict(h=1 << 21), dict(i=0), dict(i=1 << 24), dict(i=-1)):
        assert _gated(L, wsb=1 << 60, **bad) == -2, bad
        assert L.w4_gated_workspace_bytes(bad.get("fmt", 1), bad.get("t", 2), bad.get("h", 128), bad.get("i", 100)) == 0
    for bad in (dict(x=FAKE + 8), dict(w=FAKE * 2 + 4), dict(s=FAKE * 3 + 2), dict(out=FAKE * 4 + 1),
                dict(pr=FAKE * 5 + 1)):
        assert _gated(L, **bad) == -3, bad
    big = dict(t=4096, h=256, i=512)
    used = L.w4_gated_workspace_bytes(1, 4096, 256, 512)
    assert used >= 2 * 512 * 256 * 2
    assert _gated(L, ws=0, **big) == -6 and _gated(L, wsb=used - 1, **big) == -6
    assert _gated(L, ws=FAKE * 9 + 8, **big) == -3
    for name, at in (("x", FAKE), ("w", FAKE * 2), ("s", FAKE * 3)):
        assert _gated(L, out=at) == -9 and _gated(L, pr=at) == -9 and _gated(L, ws=at, **big) == -9, name
    assert _gated(L, out=FAKE * 5) == -9 and _gated(L, pr=FAKE * 4 + 2) == -9
    assert _gated(L, ws=FAKE * 4, **big) == -9 and _gated(L, ws=FAKE * 5, **big) == -9
    assert _gated(L, out=FAKE * 2 + 2 * 100 * 64 - 2) == -9  # the last bytes of the weights


def _grad(L, type=1, act=0, t=3, i=5, **p):
    a = dict(dh=FAKE, pr=FAKE * 2, out=FAKE * 3)
    a.update(p)
    return L.w4_gated_grad(vp(a["dh"]), vp(a["pr"]), type, act, t, i, vp(a["out"]), None)


def test_gated_grad_refusals():
    _, L = _lib()
    for name in ("dh", "pr", "out"):
        assert _grad(L, **{name: 0}) == -1
        assert _grad(L, **{name: FAKE * 7 + 1}) == -3
    assert _grad(L, type=0) == -4 and _grad(L, type=3) == -4 and _grad(L, act=2) == -4
    for t, i in ((0, 5), (3, 0), (-1, 5), (1 << 38, 1), (1, 1 << 38), (1 << 20, 1 << 18), (1 << 62, 1 << 62)):
        assert _grad(L, t=t, i=i) == -2, (t, i)
    assert _grad(L, out=FAKE) == -9 and _grad(L, out=FAKE + 28) == -9 and _grad(L, out=FAKE * 2 + 58) == -9


def _gemm_grad(L, fmt=1, n=70, k=128, b=3, wsb=None, ws=FAKE * 9, **p):
    a = dict(d=FAKE, w=FAKE * 2, s=FAKE * 3, out=FAKE * 4)
    a.update(p)
    if wsb is None:
        wsb = L.w4_gemm_grad_workspace_bytes(fmt, n, k, b)
    return L.w4_gemm_grad(vp(a["d"]), vp(a["w"]), vp(a["s"]), fmt, n, k, b, vp(a["out"]), vp(ws), wsb, None)


def test_gemm_grad_refusals():
    _, L = _lib()
    for name in ("d", "w", "s", "out"):
        assert _gemm_grad(L, **{name: 0}) == -1, name
    assert _gemm_grad(L, fmt=0) == -4 and _gemm_grad(L, fmt=18) == -4
    for bad in (dict(b=0), dict(b=4097), dict(k=0), dict(k=96), dict(fmt=4, k=192), dict(k=1 << 22), dict(n=0),
                dict(n=1 << 21)):
        assert _gemm_grad(L, wsb=1 << 60, **bad) == -2, bad
        assert L.w4_gemm_grad_workspace_bytes(bad.get("fmt", 1), bad.get("n", 70), bad.get("k", 128), bad.get("b", 3)) == 0
    for bad in (dict(d=FAKE + 1), dict(w=FAKE * 2 + 8), dict(s=FAKE * 3 + 2), dict(out=FAKE * 4 + 1)):
        assert _gemm_grad(L, **bad) == -3, bad
    assert _gemm_grad(L, fmt=3, s=FAKE * 3 + 1) == -3
    big = dict(n=4096, k=256, b=4096)
    used = L.w4_gemm_grad_workspace_bytes(1, 4096, 256, 4096)
    assert used >= 2 * 4096 * 256
    assert _gemm_grad(L, ws=0, **big) == -6 and _gemm_grad(L, wsb=used - 1, **big) == -6
    assert _gemm_grad(L, ws=FAKE * 9 + 8, **big) == -3
    for name, at in (("d", FAKE), ("w", FAKE * 2), ("s", FAKE * 3)):
        assert _gemm_grad(L, out=at) == -9 and _gemm_grad(L, ws=at, **big) == -9, name
    assert _gemm_grad(L, ws=FAKE * 4, **big) == -9


def test_quantize_int8_refusals():
    _, L = _lib()

    def call(type=0, r=3, k=40, x=FAKE, c=FAKE * 2, s=FAKE * 3):
        return L.w4_quantize_int8(vp(x), type, r, k, vp(c), vp(s), None)

    assert call(x=0) == -1 and call(c=0) == -1 and call(s=0) == -1
    assert call(type=3) == -4 and call(type=-1) == -4
    for r, k in ((0, 40), (1 << 31, 40), (3, 0), (3, 1 << 24), (-3, 40)):
        assert call(r=r, k=k) == -2
    assert call(x=FAKE + 2) == -3 and call(type=1, x=FAKE + 1) == -3 and call(s=FAKE * 3 + 2) == -3
    assert call(c=FAKE) == -9 and call(s=FAKE + 476) == -9 and call(s=FAKE * 2 + 116) == -9


def _int8(L, gated=False, type=1, act=0, n=30, k=128, b=5, work=FAKE * 900, wsb=None, **p):
    a = dict(xq=FAKE, xs=FAKE * 2, wq=FAKE * 3, ws=FAKE * 400, out=FAKE * 500, pr=FAKE * 600)
    a.update(p)
    v = {q: vp(z) for q, z in a.items()}
    if wsb is None:
        wsb = L.w4_int8_workspace_bytes(n, k, b, int(gated))
    if gated:
        return L.w4_gated_int8(v["xq"], v["xs"], v["wq"], v["ws"], act, b, k, n, v["out"], v["pr"], type, vp(work), wsb,
                               None)
    return L.w4_gemm_int8(v["xq"], v["xs"], v["wq"], v["ws"], n, k, b, v["out"], type, vp(work), wsb, None)


@pytest.mark.parametrize("gated", [False, True])
def test_int8_refusals(gated):
    w4, L = _lib()
    assert w4.INT8_MAX_K * 128 * 128 < 1 << 31 and w4.INT8_MAX_K % 64 == 0
    for name in ("xq", "xs", "wq", "ws", "out"):
        assert _int8(L, gated, **{name: 0}) == -1, name
    assert _int8(L, gated, type=3) == -4 and _int8(L, gated, type=-1) == -4
    if gated:
        assert _int8(L, gated, type=0) == -4 and _int8(L, gated, act=2) == -4
    for bad in (dict(b=0), dict(b=1 << 16), dict(k=0), dict(k=96), dict(k=131072), dict(n=0), dict(n=1 << 24),
                dict(b=1 << 15, n=1 << (21 if gated else 22))):
        assert _int8(L, gated, wsb=1 << 60, **bad) == -2, bad
        assert L.w4_int8_workspace_bytes(bad.get("n", 30), bad.get("k", 128), bad.get("b", 5), int(gated)) == 0
    for bad in (dict(xq=FAKE + 8), dict(xs=FAKE * 2 + 2), dict(wq=FAKE * 3 + 4), dict(ws=FAKE * 400 + 1),
                dict(out=FAKE * 500 + 1)):
        assert _int8(L, gated, **bad) == -3, bad
    long = dict(n=40, k=131008, b=64)  # few results of long rows: K is split
    used = L.w4_int8_workspace_bytes(40, 131008, 64, int(gated))
    assert used and used % (64 * 40 * (8 if gated else 4)) == 0
    assert _int8(L, gated, work=0, **long) == -6 and _int8(L, gated, wsb=used - 1, **long) == -6
    assert _int8(L, gated, work=FAKE * 900 + 8, **long) == -3
    for at in (FAKE, FAKE * 2, FAKE * 3, FAKE * 400, FAKE * 500):
        assert _int8(L, gated, work=at, **long) == -9, at
    for name, at in (("xq", FAKE), ("xs", FAKE * 2), ("wq", FAKE * 3), ("ws", FAKE * 400)):
        assert _int8(L, gated, out=at) == -9, name
        if gated:
            assert _int8(L, gated, pr=at) == -9, name
    assert _int8(L, gated, out=FAKE * 3 + 128 * 30 * (2 if gated else 1) - 2) == -9
    if gated:
        assert _int8(L, gated, pr=FAKE * 500) == -9 and _int8(L, gated, pr=FAKE * 600 + 1) == -3


def test_binding_refuses_host_tensors():
    import torch

    w4, _ = _lib()
    z, u8, i8, f16 = torch.zeros, torch.uint8, torch.int8, torch.float16
    with pytest.raises(ValueError):
        w4.gated(z(1, 64, dtype=f16), z(4, 32, dtype=u8), z(4, 1), "nf4_f16")
    with pytest.raises(ValueError):
        w4.gated_grad(z(1, 4, dtype=f16), z(1, 8, dtype=f16))
    with pytest.raises(ValueError):
        w4.gemm_grad(z(1, 4, dtype=f16), z(4, 32, dtype=u8), z(4, 1), "nf4_f16")
    with pytest.raises(ValueError):
        w4.quantize_int8(z(1, 4))
    for call in (w4.gemm_int8, w4.gated_int8):
        with pytest.raises(ValueError):
            call(z(1, 64, dtype=i8), z(1), z(4, 64, dtype=i8), z(4))
