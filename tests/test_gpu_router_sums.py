"""Sums over tokens of the router losses at magnitudes and lengths where 32 bits alone would not hold them."""
import numpy as np
import pytest

from oracle import router as orouter

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("T,E,k", [(50, 4, 2), (512, 4, 2), (9000, 8, 2), (9000, 24, 4), (9000, 48, 4), (9000, 48, 8),
                                   (9000, 100, 2), (9000, 100, 8), (9000, 256, 8), (9000, 250, 20),
                                   (60000, 48, 8), (60000, 100, 2), (60000, 100, 8), (60000, 256, 8), (60000, 250, 20)])
def test_squares_whose_sum_passes_fp32(T, E, k):
    """lse near 4e18, its square 2e37: twenty of them pass fp32, their mean does
    not.  lse is off by one rounding, 2^-24 (log(sum) is nothing beside 4e18), its
    square by twice that; at most 13 tokens per lane, 5 lanes' and 8 warps' sums and
    the loss itself round once each, all terms positive: 29 2^-24."""
    import torch
    from mxfp8_grouped_gemm_x32_b200.layer import GroupedMLP
    rng = np.random.default_rng(E + k)
    z = (rng.normal(size=(T, E)) + rng.uniform(3e18, 5e18, size=(T, 1))).astype(np.float32)
    mask = rng.random(T) < 0.9
    layer = GroupedMLP(T, 32, 64, E, k, backward=False, mxfp8=False, guard=4096)
    for m in (None, mask):
        f = orouter.route_losses(z, k, m)
        _, _, losses = layer.route_losses(torch.from_numpy(z).cuda(), None if m is None else torch.from_numpy(m).cuda())
        got = float(losses[1])
        assert np.isfinite(f["losses"][1].astype(np.float32))
        assert abs(got - f["losses"][1]) <= 32 * 2.0 ** -24 * f["losses"][1]
    assert layer.check_guards() == []
