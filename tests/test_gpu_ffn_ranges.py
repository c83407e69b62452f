"""Gated block and its gradients at the ends of their types' ranges, and operands at addresses of their own."""
import pytest
import torch

from tests import ffn_util as f
from tests.test_gpu_ffn import ACTS

pytestmark = pytest.mark.gpu


def _w4():
    import bit_weight_only_w4_amd as w4

    return w4


@pytest.mark.parametrize("act", ACTS)
def test_gated_grad_of_large_and_small_factors(act):
    """dh * u alone may leave fp32's range, and so may u * act'(g); their product with the third does not."""
    w4, dev = _w4(), f.device()
    mags = [1e20, 1e30, 3e38, 1e-20, 1e-30, 1e-38, 1.0]
    gates = [-200.0, -90.0, -60.0, -40.0, -8.0, -1.0, 0.0, 1.0, 40.0]
    rows = [(d, u, g) for d in mags for u in mags for g in gates]
    t = torch.tensor(rows, dtype=torch.float64).to(torch.bfloat16)
    dh, pr = t[:, :1].contiguous(), torch.stack((t[:, 2], t[:, 1]), 1).contiguous()
    got = w4.gated_grad(dh.to(dev), pr.to(dev), act).cpu().double()
    ref, bound = f.gated_grad_bound(dh, pr, act)
    assert not torch.isnan(got).any()
    inside = ref.abs() + bound < 3.38e38
    assert ((got - ref).abs() <= bound)[inside].all()
    assert inside.sum() > 600
