"""Which way a gated block takes, told by the workspace that it asks for: none where the weights are streamed, little where
the product decodes them, two or four bytes a weight where they are decoded first."""
import pytest


def _bytes(fmt, tokens, hidden, inter):
    import bit_weight_only_w4_amd as w4

    return w4.gated_workspace_bytes(fmt, tokens, hidden, inter)


@pytest.mark.parametrize("xt", ["f16", "bf16"])
def test_streamed_where_that_is_faster(xt):
    for weight, tokens, hidden, inter, streamed in (
            ("mxfp4", 32, 4096, 11008, True), ("mxfp4", 48, 4096, 11008, False), ("mxfp4", 64, 8192, 28672, False),
            ("mxfp4", 64, 1536, 8960, True), ("mxfp4", 96, 1536, 8960, False), ("mxfp4", 96, 896, 4864, False),
            ("int4", 64, 8192, 28672, True), ("int4", 96, 8192, 28672, False), ("int4", 128, 1536, 8960, True),
            ("nf4", 128, 4096, 11008, True), ("fp4", 128, 8192, 28672, True), ("int4a", 128, 4096, 11008, True),
            ("nf4", 192, 4096, 11008, False)):
        assert (_bytes(f"{weight}_{xt}", tokens, hidden, inter) == 0) == streamed, (weight, tokens, hidden)


@pytest.mark.parametrize("xt", ["f16", "bf16"])
def test_decoded_first_only_where_that_is_faster(xt):
    for weight, tokens, hidden, inter, first in (
            ("nf4", 512, 8192, 28672, False), ("nf4", 512, 4096, 11008, False), ("nf4", 192, 8192, 28672, False),
            ("nf4", 2048, 4096, 11008, True), ("nf4", 512, 1536, 8960, True), ("fp4", 512, 8192, 28672, False),
            ("int4", 512, 8192, 28672, False), ("int4", 4096, 8192, 28672, True), ("mxfp4", 1000, 8192, 28672, False),
            ("mxfp4", 4096, 4096, 11008, True)):
        got = _bytes(f"{weight}_{xt}", tokens, hidden, inter)
        assert got > 0 and (got >= 2 * inter * hidden * 2) == first, (weight, tokens, hidden)
