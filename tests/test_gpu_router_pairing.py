"""route_backward belongs to the last route_losses: another routing in between leaves it alone, and the mask need not be
given twice.  Bit for bit against the two calls in a row."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _case(seed, T, E, k, dtype):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(T, E, device="cuda", generator=g).to(dtype)
    return z, torch.randn(T, k, device="cuda", generator=g), torch.tensor([0.3, 0.1], device="cuda"), \
        torch.rand(T, device="cuda", generator=g) < 0.7


@pytest.mark.parametrize("E,k", [(8, 2), (100, 4)])
@pytest.mark.parametrize("between", ["route", "route_permute"])
@pytest.mark.parametrize("masked", [False, True])
def test_another_routing_in_between(E, k, between, masked):
    import torch
    from mxfp8_grouped_gemm_x32_b200.layer import GroupedMLP
    T, H = 333, 64
    z, dp, dl, mask = _case(E, T, E, k, torch.float32)
    other = _case(E + 1, T, E, k, torch.float32)[0]
    layer = GroupedMLP(T, H, 64, E, k, backward=False, guard=4096)
    idx, prob, _ = layer.route_losses(z, mask if masked else None)
    want = layer.route_backward(z, dp, dl, mask if masked else None).clone()
    keep = idx.clone(), prob.clone()
    if between == "route":
        i2, p2 = layer.route(other)
    else:
        i2, p2 = layer.route_permute(other, torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"))
    got = layer.route_backward(z, dp, dl, mask if masked else None)
    assert torch.equal(got, want)
    assert torch.equal(idx, keep[0]) and torch.equal(prob, keep[1])
    # the layer's ids and probabilities are the last routing's, whichever call made it
    assert layer.topk_idx.data_ptr() == i2.data_ptr() and torch.equal(layer.topk_prob, p2)
    assert not torch.equal(i2, idx)
    idx, prob, _ = layer.route_losses(z, mask if masked else None)
    assert layer.topk_idx.data_ptr() == idx.data_ptr() and layer.topk_prob.data_ptr() == prob.data_ptr()
    assert torch.equal(idx, keep[0]) and layer.check_guards() == []


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("E,k", [(8, 2), (60, 6), (256, 8)])
def test_the_mask_of_the_losses_is_the_gradients(E, k, dtype):
    import torch
    from mxfp8_grouped_gemm_x32_b200.layer import GroupedMLP
    T = 500
    z, dp, dl, mask = _case(E, T, E, k, getattr(torch, dtype))
    z[~mask] = float("nan")
    layer = GroupedMLP(T, 32, 64, E, k, backward=False, mxfp8=False)
    layer.route_losses(z, mask)
    want = layer.route_backward(z, dp, dl, mask).clone()
    assert torch.equal(layer.route_backward(z, dp, dl), want) and bool((want[~mask] == 0).all())
    # and after losses without one there is none
    z = torch.nan_to_num(z)
    layer.route_losses(z)
    every = layer.route_backward(z, dp, dl)
    assert bool((every[~mask] != 0).any(1).all())
    assert torch.equal(every, layer.route_backward(z, dp, dl, torch.ones(T, dtype=torch.bool, device="cuda")))
