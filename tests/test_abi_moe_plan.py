"""The expert layer's launch rules on the host: every accepted size has launches whose LDS fits."""
import pytest

LDS = 160 * 1024          # of a CU
TABLE = 32 * 1024         # NF4's decode table
WINDOW = 80 * 1024        # the most that the shared products keep activations in


def _w4():
    import bit_weight_only_w4_amd as w4

    return w4


def _check(p, tokens, experts, top_k, fmt="nf4_f16"):
    up_tiles = 1
    down_tiles = 1 if tokens * top_k <= 2 * experts else 3
    for window, tiles in ((p["up_window"], up_tiles), (p["down_window"], down_tiles)):
        assert 0 < window <= WINDOW
        assert TABLE + window + 2 * 8 * tiles * 1024 <= LDS
    assert p["up_groups"] in (1, 2, 4) and p["down_groups"] in (1, 2, 4)


@pytest.mark.parametrize("tokens,hidden,inter,experts,top_k", [
    (14, 512, 1280, 8, 2), (14, 1024, 2048, 4, 2), (7, 256, 2304, 2, 1), (7, 512, 2560, 2, 2), (14, 256, 1280, 4, 1)])
def test_windows_of_three_planes_that_do_not_divide_the_row(tokens, hidden, inter, experts, top_k):
    p = _w4().moe_plan("nf4_f16", tokens, hidden, inter, experts, top_k)
    assert p["kind"] == 1
    _check(p, tokens, experts, top_k)


@pytest.mark.parametrize("tokens", range(1, 17))
def test_every_size_of_few_tokens_fits(tokens):
    """Rows of 1 to 64 quads (256 values) and some longer, few and many row tiles, one and three planes."""
    w4 = _w4()
    lengths = [64 * i for i in range(1, 65)] + [256 * q + r for q in range(1, 65) for r in (0, 64)] + \
        [20480, 28672, 65536, (1 << 22) - 64]
    shared = 0
    for experts, top_k in ((1, 1), (2, 1), (2, 2), (3, 1), (4, 1), (4, 2), (8, 2), (8, 4), (16, 4), (64, 6), (128, 8)):
        for other in (64, 256, 1024, 4096, 16384):
            for length in lengths:
                for hidden, inter in ((other, length), (length, other)):
                    if w4.moe_workspace_bytes("nf4_f16", tokens, hidden, inter, experts, top_k) == 0:
                        continue  # not an accepted size
                    p = w4.moe_plan("nf4_f16", tokens, hidden, inter, experts, top_k)
                    if p["kind"] == 1:
                        _check(p, tokens, experts, top_k)
                        shared += 1
                    else:
                        assert p["up_window"] == p["down_window"] == 0
    assert shared > 0 or tokens == 1


def test_larger_batches_of_shared_products_fit():
    w4 = _w4()
    for tokens in (17, 31, 63, 64, 100, 250, 700):
        for experts, top_k in ((128, 1), (128, 2), (256, 2), (1024, 1), (1024, 2)):
            for hidden, inter in ((64, 1280), (256, 20480), (2048, 768), (4096, 1408), (1280, 2304)):
                p = w4.moe_plan("nf4_bf16", tokens, hidden, inter, experts, top_k)
                if p["kind"] == 1:
                    _check(p, tokens, experts, top_k)


def test_refusals():
    w4 = _w4()
    with pytest.raises(w4.W4Error) as e:
        w4.moe_plan("nf4_f16", 0, 64, 64, 1, 1)
    assert e.value.status == -2
    with pytest.raises(w4.W4Error):
        w4.moe_plan("int4_f16", 1, 64, 128, 1, 1)
    assert w4.lib().w4_moe_plan(9, 1, 64, 64, 1, 1, None, None, None, None, None) == -4
    assert w4.lib().w4_moe_plan(1, 1, 64, 64, 1, 1, None, None, None, None, None) == 0


@pytest.mark.parametrize("tokens,experts,top_k,kind", [
    (8, 1, 1, 1), (13, 1, 1, 1), (14, 1, 1, 2), (16, 2, 1, 1), (27, 2, 1, 1), (28, 2, 1, 2), (16, 4, 2, 1),
    (27, 4, 2, 1), (28, 4, 2, 2), (31, 8, 2, 1), (32, 8, 2, 2), (15, 16, 8, 1), (16, 16, 8, 2), (95, 256, 8, 1),
    (96, 256, 8, 2)])
def test_sorted_pairs_start_where_they_were_measured_to_pay(tokens, experts, top_k, kind):
    """2048 x 2048: fewer than eight experts from 14 pairs each, more from eight, those that fill the card from three."""
    assert _w4().moe_plan("int4_f16", tokens, 1024 if experts == 16 else 2048, 2048, experts, top_k)["kind"] == kind
