"""The expert layer's shared products where the activations of a chunk come in several windows."""
import pytest

from tests import gpu_util as g
from tests import moe_util as mu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["nf4_f16", "mxfp4_bf16", "int4_bf16"])
@pytest.mark.parametrize("tokens,hidden,inter,experts,top_k", [
    (14, 512, 1280, 8, 2), (14, 1024, 2048, 4, 2), (7, 256, 2304, 2, 1), (7, 512, 2560, 2, 2), (14, 256, 1280, 4, 1),
    (6, 128, 3200, 2, 2), (10, 256, 1920, 4, 2), (11, 256, 2304, 4, 1), (13, 128, 1664, 4, 2), (15, 256, 2432, 4, 2),
    (15, 1664, 1280, 5, 2)])
def test_windows_of_three_planes(fmt, tokens, hidden, inter, experts, top_k):
    import bit_weight_only_w4_amd as w4

    dev = g.device()
    p = w4.moe_plan(fmt, tokens, hidden, inter, experts, top_k)
    assert p["kind"] == 1 and tokens * top_k > 2 * experts  # three planes, a tile each
    quads = (inter + 255) // 256
    assert p["down_window"] < 3 * tokens * quads * 512  # more than one window
    c = mu.case(fmt, tokens, hidden, inter, experts, top_k, seed=tokens + inter)
    mu.check(w4.moe(*mu.to_device(c, dev)), c)


@pytest.mark.parametrize("fmt", ["nf4_bf16", "int4a_f16", "mxfp4_f16"])
@pytest.mark.parametrize("tokens,hidden,inter,experts,top_k,kind", [
    (8, 512, 640, 1, 1, 1), (13, 2304, 1280, 1, 1, 1), (14, 512, 640, 1, 1, 2), (27, 256, 640, 2, 1, 1),
    (28, 256, 640, 2, 1, 2), (26, 384, 2304, 4, 2, 1), (6, 640, 384, 1, 2, 1), (7, 640, 384, 1, 2, 2)])
def test_few_experts_around_the_rule(fmt, tokens, hidden, inter, experts, top_k, kind):
    import bit_weight_only_w4_amd as w4

    dev = g.device()
    assert w4.moe_plan(fmt, tokens, hidden, inter, experts, top_k)["kind"] == kind
    c = mu.case(fmt, tokens, hidden, inter, experts, top_k, seed=tokens + inter)
    mu.check(w4.moe(*mu.to_device(c, dev)), c)
