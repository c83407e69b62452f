"""Launch shapes of the fused GEMV on long rows: no team passes the largest workgroup that it is built for."""
import pytest


@pytest.mark.parametrize("fmt", ["nf4_f16", "int4_bf16", "int4a_f16", "fp4_bf16", "mxfp4_f16"])
@pytest.mark.parametrize("batch", range(1, 9))
def test_teams_fit_a_workgroup(fmt, batch):
    import bit_weight_only_w4_amd as w4

    planned = 0
    for n in (1, 64, 5000, 131200):
        for k in [128 * i for i in range(1, 400, 7)] + [49152, 49280, 65536, 131072, 131200, 1 << 20]:
            for split in (1, 2, 4):
                try:
                    p = w4.gemv_plan(fmt, n, k, batch, split)
                except w4.W4Error as e:
                    assert e.status == -7
                    continue
                planned += 1
                assert p["threads"] in (256, 512) and p["threads"] % p["team"] == 0
                assert p["team"] * p["iters"] >= p["chunks_per_split"]
    assert planned > 0
    if batch == 1:
        assert w4.gemv_plan(fmt, 64, 131072, 1)["iters"] == 8
