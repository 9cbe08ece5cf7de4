"""A layer without tokens: the permutation's kernels write the empty maps and nothing past the workspace, whose size
moe_workspace_size states (256 bytes for no slots, less than one block's counts of more than 64 experts)."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("E", [1, 64, 65, 128, 256])
@pytest.mark.parametrize("recipe", ["mxfp4", "mxfp8", "bf16"])
def test_no_tokens(E, recipe):
    import torch
    from mxfp8_grouped_gemm_x32_b200 import lib
    from mxfp8_grouped_gemm_x32_b200.layer import GroupedMLP
    H, I, k = 32, 64, 1
    layer = GroupedMLP(0, H, I, E, k, backward=False, mxfp8=recipe == "mxfp8", guard=4096)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    w1, w2, x = torch.zeros(E, 2 * I, H, **bf), torch.zeros(E, H, I, **bf), torch.empty(0, H, **bf)
    idx, prob = torch.empty(0, k, dtype=torch.int32, device="cuda"), torch.empty(0, k, device="cuda")
    layer.split_sizes.fill_(7)
    layer.group_offsets.fill_(7)
    layer.row_to_slot.fill_(7)
    layer.prob_perm.fill_(7.0)
    if recipe == "mxfp8":
        layer.quantize_weights(w1, w2)
        layer.permute(x, idx, prob)
        out = layer.forward()
    else:
        layer.permute_index(idx, prob)
        if recipe == "mxfp4":
            layer.quantize_weights_mxfp4(w1, w2)
            out = layer.forward_mxfp4(x)
        else:
            out = layer.forward_bf16(x, w1, w2)
    torch.cuda.synchronize()
    assert out.shape == (0, H) and layer.check_guards() == [] and lib.moe_get_device_status(0) == 0
    assert not layer.split_sizes.any() and not layer.group_offsets.any() and not layer.prob_perm.any()
    assert bool((layer.row_to_slot == -1).all())
