"""Host-side refusals of the expert layer and its router (no launch is made)."""
import ctypes

import pytest

FAKE = 0x100000  # a non-null, well-aligned address that is never dereferenced


def _lib():
    import bit_weight_only_w4_amd as w4

    return w4, w4.lib()


def vp(a):
    return ctypes.c_void_p(a)


def _route(L, logits=FAKE, kind=0, t=4, e=8, k=2, ids=FAKE * 2, w=FAKE * 3):
    return L.w4_moe_route(vp(logits), kind, t, e, k, 1, vp(ids), vp(w), None)


def test_route_refusals():
    _, L = _lib()
    for name in ("logits", "ids", "w"):
        assert _route(L, **{name: 0}) == -1
    assert _route(L, kind=3) == -4
    assert _route(L, t=0) == -2 and _route(L, t=1 << 26) == -2
    assert _route(L, e=0) == -2 and _route(L, e=1025) == -2
    assert _route(L, k=0) == -2 and _route(L, k=9) == -2 and _route(L, e=64, k=17) == -2
    assert _route(L, logits=FAKE + 2) == -3 and _route(L, ids=FAKE * 2 + 2) == -3 and _route(L, w=FAKE + 1) == -3
    assert _route(L, kind=1, logits=FAKE + 1) == -3
    assert _route(L, ids=FAKE) == -9 and _route(L, w=FAKE + 64) == -9 and _route(L, ids=FAKE * 3) == -9


def _moe(L, fmt=1, t=2, h=128, i=128, e=4, k=2, y=FAKE * 8, ws=FAKE * 9, wsb=None, **p):
    a = dict(x=FAKE, ids=FAKE * 2, w=FAKE * 3, gu=FAKE * 4, gus=FAKE * 5, d=FAKE * 6, ds=FAKE * 7)
    a.update(p)
    if wsb is None:
        wsb = L.w4_moe_workspace_bytes(fmt, t, h, i, e, k)
    return L.w4_moe(vp(a["x"]), vp(a["ids"]), vp(a["w"]), vp(a["gu"]), vp(a["gus"]), vp(a["d"]), vp(a["ds"]),
                    fmt, t, h, i, e, k, vp(y), vp(ws), wsb, None)


def test_layer_refusals():
    _, L = _lib()
    for name in ("x", "ids", "w", "gu", "gus", "d", "ds"):
        assert _moe(L, **{name: 0}) == -1, name
    assert _moe(L, y=0) == -1
    assert _moe(L, fmt=0) == -4 and _moe(L, fmt=9) == -4
    for bad in (dict(t=0), dict(t=4097), dict(e=0), dict(e=1025), dict(k=0), dict(k=17), dict(h=0), dict(h=96),
                dict(i=96), dict(i=0), dict(fmt=3, h=192), dict(fmt=8, i=192), dict(h=1 << 22)):
        assert _moe(L, wsb=1 << 40, **bad) == -2, bad
        assert L.w4_moe_workspace_bytes(bad.get("fmt", 1), bad.get("t", 2), bad.get("h", 128), bad.get("i", 128),
                                        bad.get("e", 4), bad.get("k", 2)) == 0
    # offsets inside x and the planes of h stay below 2^31
    assert _moe(L, t=4096, h=1 << 18, wsb=1 << 60) == -2
    assert _moe(L, t=4096, k=16, i=8192, wsb=1 << 60) == -2
    for bad in (dict(x=FAKE + 8), dict(gu=FAKE * 4 + 8), dict(d=FAKE * 6 + 4), dict(gus=FAKE * 5 + 2),
                dict(ds=FAKE * 7 + 1), dict(ids=FAKE * 2 + 2), dict(w=FAKE * 3 + 2), dict(y=FAKE * 8 + 2),
                dict(ws=FAKE * 9 + 8)):
        assert _moe(L, **bad) == -3, bad
    assert _moe(L, ws=0) == -6 and _moe(L, wsb=16) == -6
    for name in ("x", "ids", "w", "gu", "gus", "d", "ds"):
        at = dict(x=FAKE, ids=FAKE * 2, w=FAKE * 3, gu=FAKE * 4, gus=FAKE * 5, d=FAKE * 6, ds=FAKE * 7)[name]
        assert _moe(L, y=at) == -9 and _moe(L, ws=at) == -9, name
    assert _moe(L, y=FAKE * 9 + 64) == -9
    assert _moe(L, gu=FAKE * 4, ds=FAKE * 4, y=FAKE * 4 + 4 * 128 * 128 - 4) == -9  # its last bytes


def test_workspace_grows_with_the_pairs():
    w4, _ = _lib()
    a = w4.moe_workspace_bytes("nf4_f16", 1, 512, 256, 8, 2)
    assert a >= 2 * (6 * 256 + 4 * 512)
    assert w4.moe_workspace_bytes("nf4_f16", 8, 512, 256, 8, 2) > 4 * a


def test_binding_refuses_host_tensors():
    import torch

    w4, _ = _lib()
    with pytest.raises(ValueError):
        w4.moe_route(torch.zeros(2, 4), 2)
    with pytest.raises(ValueError):
        w4.moe_route(torch.zeros(2, 4, dtype=torch.float64), 2)
    z = torch.zeros
    with pytest.raises(ValueError):
        w4.moe(z(1, 64, dtype=torch.float16), z(1, 1, dtype=torch.int32), z(1, 1), z(1, 128, 32, dtype=torch.uint8),
               z(1, 128, 1), z(1, 64, 32, dtype=torch.uint8), z(1, 64, 1), "nf4_f16")
    with pytest.raises(ValueError):
        w4.moe(*[z(1, 1)] * 7, "nf5_f16")
