"""Permutation and combine across the sizes at which their kernels change:
slots up to 1024 in one launch, more of them through histogram, scan and
scatter; few or many output rows.  Plain numpy is the reference; the index
maps are exact, out is the fp32 sum in ascending j rounded once to bf16 (the
same bits)."""
import numpy as np
import pytest

from mxfp8_grouped_gemm_x32_b200.workloads import bf16_bits_from_f32, bf16_bits_to_f32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _permutation(idx, prob, E, rows_cap):
    T, k = idx.shape
    flat = idx.reshape(-1)
    ok = (flat >= 0) & (flat < E)
    split = np.bincount(flat[ok], minlength=E)
    offs = np.concatenate([[0], np.cumsum((split + 127) // 128 * 128)])
    slot_to_row = np.full(T * k, -1)
    row_to_slot, prob_perm = np.full(rows_cap, -1), np.zeros(rows_cap, np.float32)
    for e in range(E):
        slots = np.flatnonzero(ok & (flat == e))
        rows = offs[e] + np.arange(len(slots))
        slot_to_row[slots], row_to_slot[rows], prob_perm[rows] = rows, slots, prob.reshape(-1)[slots]
    return split, offs, slot_to_row, row_to_slot, prob_perm


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 8), (1, 8, 128), (1, 1, 256), (31, 1, 5), (16, 2, 256), (33, 1, 3),
                                   (128, 1, 1), (129, 1, 1), (64, 4, 32), (1023, 1, 7), (512, 2, 256), (1024, 1, 1),
                                   (256, 4, 4), (1025, 1, 7), (205, 5, 256), (2048, 1, 1), (3001, 3, 40)])
@pytest.mark.parametrize("kind", ["spread", "one expert", "some rejected", "all rejected"])
def test_permutation(T, k, E, kind):
    import torch
    from mxfp8_grouped_gemm_x32_b200 import lib
    from mxfp8_grouped_gemm_x32_b200.layer import GroupedMLP
    rng = np.random.default_rng(T * k + E)
    idx = rng.integers(0, E, (T, k)).astype(np.int32)
    if kind == "one expert":
        idx[:] = E - 1
    elif kind == "some rejected":
        idx[rng.random((T, k)) < 0.3] = -1
        idx[rng.random((T, k)) < 0.1] = E
    elif kind == "all rejected":
        idx[:] = E
    prob = rng.random((T, k)).astype(np.float32)
    layer = GroupedMLP(T, 32, 64, E, k, backward=False, mxfp8=False, guard=4096)
    layer.row_to_slot.fill_(77)
    layer.prob_perm.fill_(7.0)
    layer.permute_index(torch.from_numpy(idx).cuda(), torch.from_numpy(prob).cuda())
    torch.cuda.synchronize()
    assert lib.moe_get_device_status(0) == (5 if np.any((idx < 0) | (idx >= E)) else 0)
    assert layer.check_guards() == []
    for name, want in zip(("split_sizes", "group_offsets", "slot_to_row", "row_to_slot", "prob_perm"),
                          _permutation(idx, prob, E, layer.rows_cap)):
        assert np.array_equal(getattr(layer, name).cpu().numpy().reshape(-1), want), name


@pytest.mark.parametrize("T,H", [(1, 32), (1, 2880), (7, 96), (64, 2880), (300, 4096), (2500, 2048)])
@pytest.mark.parametrize("k", [1, 3, 4, 5, 8])
def test_combine(T, H, k):
    import torch
    from mxfp8_grouped_gemm_x32_b200 import lib
    rng = np.random.default_rng(T + k)
    y = bf16_bits_from_f32(rng.normal(size=(T * k, H)).astype(np.float32))
    dy = torch.from_numpy(y.view(np.int16)).view(torch.bfloat16).cuda()
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    lib.moe_combine(dy.data_ptr(), T, k, H, out.data_ptr())
    torch.cuda.synchronize()
    rows = bf16_bits_to_f32(y).reshape(T, k, H)
    want = np.zeros((T, H), np.float32)
    for j in range(k):
        want += rows[:, j]
    assert np.array_equal(out.view(torch.int16).cpu().numpy().view(np.uint16), bf16_bits_from_f32(want))


@pytest.mark.parametrize("recipe", ["bf16", "mxfp4"])
def test_a_token_alone_and_among_many(recipe):
    """A token's output does not depend on the others' number."""
    import torch
    from mxfp8_grouped_gemm_x32_b200.layer import GroupedMLP
    H, I, E, k, T = 256, 128, 4, 3, 5000
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    w1 = (torch.randn(E, 2 * I, H, device="cuda", generator=g) / 16).bfloat16()
    w2 = (torch.randn(E, H, I, device="cuda", generator=g) / 11).bfloat16()
    idx = torch.argsort(torch.rand(T, E, device="cuda", generator=g), 1)[:, :k].int().contiguous()
    prob = torch.rand(T, k, device="cuda", generator=g)
    outs = []
    for n in (T, 6):
        layer = GroupedMLP(n, H, I, E, k, backward=False, mxfp8=False)
        layer.permute_index(idx[:n].contiguous(), prob[:n].contiguous())
        if recipe == "mxfp4":
            layer.quantize_weights_mxfp4(w1, w2)
            outs.append(layer.forward_mxfp4(x[:n].contiguous())[:6].clone())
        else:
            outs.append(layer.forward_bf16(x[:n].contiguous(), w1, w2)[:6].clone())
    assert torch.equal(outs[0], outs[1])
