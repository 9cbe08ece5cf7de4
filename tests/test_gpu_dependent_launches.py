"""Kernels that start while the one before them runs: passes over two inputs
with different routings in turn on one layer, nothing waited for in between, so
that every buffer a kernel could read too early holds the other input's values.
Results bit for bit those of a layer of its own for each input, synchronised
after every call."""
import numpy as np
import pytest

from tests import test_gpu_mxfp4 as mx

pytestmark = pytest.mark.gpu

H, I = 256, 192


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _inputs(seed, T, E, k):
    """Skewed towards other experts for each seed: other group sizes, offsets and row numbers."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(T, E, device="cuda", generator=g) + 2 * torch.randn(E, device="cuda", generator=g)
    return dict(z=z, x=torch.randn(T, H, device="cuda", generator=g).bfloat16(),
                mask=torch.rand(T, device="cuda", generator=g) < 0.8,
                dp=torch.randn(T, k, device="cuda", generator=g), dl=torch.tensor([0.3, 0.1], device="cuda"))


def _weights(E):
    import torch
    g = torch.Generator(device="cuda").manual_seed(99)
    return ((torch.randn(E, 2 * I, H, device="cuda", generator=g) / 16).bfloat16(),
            (torch.randn(E, H, I, device="cuda", generator=g) / 14).bfloat16())


def _layer(recipe, T, E, k, w):
    from mxfp8_grouped_gemm_x32_b200.layer import GroupedMLP
    layer = GroupedMLP(T, H, I, E, k, backward=False, mxfp8=recipe == "mxfp8")
    if recipe == "mxfp4":
        layer.quantize_weights_mxfp4(*w)
    elif recipe == "mxfp8":
        layer.quantize_weights(*w)
    return layer


def _pass(recipe, layer, t, w, wait=lambda: None):
    """Router losses, permutation, experts, the logits' gradient; clones made on the stream."""
    idx, prob, losses = layer.route_losses(t["z"], t["mask"])
    wait()
    if recipe == "mxfp8":
        layer.permute(t["x"], idx, prob)
        wait()
        out = layer.forward()
    else:
        layer.permute_index(idx, prob)
        wait()
        out = layer.forward_mxfp4(t["x"]) if recipe == "mxfp4" else layer.forward_bf16(t["x"], *w)
    wait()
    got = [out.clone(), losses.clone(), layer.expert_counts.clone(), layer.group_offsets.clone(), layer.row_to_slot.clone()]
    got.append(layer.route_backward(t["z"], t["dp"], t["dl"]).clone())
    wait()
    return got


# slots up to 1024 (one launch) and above (three); one and several row tiles per expert
SIZES = [(1, 8, 2), (64, 16, 4), (256, 32, 4), (900, 16, 4), (3000, 8, 3)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("recipe", ["mxfp4", "bf16", "mxfp8"])
def test_two_inputs_in_turn(recipe, T, E, k):
    import torch
    from mxfp8_grouped_gemm_x32_b200 import lib
    w = _weights(E)
    ins = [_inputs(s, T, E, k) for s in (1, 2)]
    want = [_pass(recipe, _layer(recipe, T, E, k, w), t, w, torch.cuda.synchronize) for t in ins]
    assert not torch.equal(want[0][3], want[1][3]) or T == 1
    layer = _layer(recipe, T, E, k, w)
    torch.cuda.synchronize()
    got = [_pass(recipe, layer, ins[n % 2], w) for n in range(40)]
    torch.cuda.synchronize()
    for n, outs in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(outs, want[n % 2])), n
    assert lib.moe_get_device_status(0) == 0


@pytest.mark.parametrize("T,E,k", SIZES)
def test_in_one_graph_with_branches(T, E, k):
    """Captured: both inputs in turn, the second's ids and probabilities copied
    on another stream, which joins right before the permutation (the node that
    a dependent launch follows is then a copy, or one of two)."""
    import torch
    w = _weights(E)
    ins = [_inputs(s, T, E, k) for s in (3, 4)]
    want = [_pass("mxfp4", _layer("mxfp4", T, E, k, w), t, w, torch.cuda.synchronize) for t in ins]
    layer = _layer("mxfp4", T, E, k, w)
    router = _layer("mxfp4", T, E, k, w)
    _pass("mxfp4", layer, ins[0], w)                      # buffers made before the capture
    router.route_losses(ins[1]["z"], ins[1]["mask"])
    idx, prob = torch.empty_like(router.topk_idx), torch.empty_like(router.topk_prob)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            i, p, _ = router.route_losses(ins[1]["z"], ins[1]["mask"])
            idx.copy_(i)
            prob.copy_(p)
        first = _pass("mxfp4", layer, ins[0], w)
        main.wait_stream(side)
        layer.permute_index(idx, prob)
        second = layer.forward_mxfp4(ins[1]["x"]).clone()
        maps = [layer.group_offsets.clone(), layer.row_to_slot.clone()]
    for _ in range(5):
        for t in first + maps + [second, idx, prob, layer.out, layer.slot_to_row]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, want[0]))
        assert torch.equal(second, want[1][0])
        assert torch.equal(maps[0], want[1][3]) and torch.equal(maps[1], want[1][4])


@pytest.mark.parametrize("order", ["rising", "falling"])
def test_groups_of_every_size(order):
    """Groups of 1 to 70 rows: every number of lanes without a token in the last
    warp of a group, several blocks of columns."""
    import torch
    E = 70
    sizes = np.arange(1, E + 1) if order == "rising" else np.arange(E, 0, -1)
    idx = np.repeat(np.arange(E), sizes)
    T = len(idx)
    idx = np.random.default_rng(1).permutation(idx).reshape(T, 1)
    x, w1, w2, idx, prob = mx._problem(T, 160, 320, E, 1, seed=2, idx=idx)
    layer = mx._layer(T, 160, 320, E, 1, w1, w2)
    layer.permute_index(torch.from_numpy(idx).cuda(), torch.from_numpy(prob).cuda())
    out = layer.forward_mxfp4(mx._bf(x))
    torch.cuda.synchronize()
    assert mx._status() == 0 and layer.check_guards() == []
    mx._check_out(out, x, w1, w2, idx, prob)


@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (40, 256, 8), (700, 256, 4), (500, 128, 8), (2500, 200, 1)])
def test_many_experts(T, E, k):
    import torch
    x, w1, w2, idx, prob = mx._problem(T, 64, 128, E, k, seed=T)
    idx[idx % 7 == 3] = E - 1                             # empty groups among them, and the last one large
    layer = mx._layer(T, 64, 128, E, k, w1, w2)
    layer.permute_index(torch.from_numpy(idx).cuda(), torch.from_numpy(prob).cuda())
    out = layer.forward_mxfp4(mx._bf(x))
    torch.cuda.synchronize()
    assert mx._status() == 0 and layer.check_guards() == []
    mx._check_out(out, x, w1, w2, idx, prob)


@pytest.mark.parametrize("T,Hd,Id,E,k", [(3, 96, 64, 4, 2), (150, 288, 192, 7, 3), (1200, 416, 832, 5, 2)])
@pytest.mark.parametrize("byte", [0x00, 0x7F, 0xFF])
def test_what_the_buffers_held_before(T, Hd, Id, E, k, byte):
    """The workspace's and the row maps' earlier bytes (NaN scales, largest codes, ids) reach no output."""
    import torch
    x, w1, w2, idx, prob = mx._problem(T, Hd, Id, E, k, seed=T)
    outs = []
    for fill in (0x55, byte):
        layer = mx._layer(T, Hd, Id, E, k, w1, w2)
        layer.permute_index(torch.from_numpy(idx).cuda(), torch.from_numpy(prob).cuda())
        layer.forward_mxfp4(mx._bf(x))
        for t in (layer.ws_mxfp4, layer.ws_perm, layer.split_sizes, layer.group_offsets, layer.row_to_slot,
                  layer.slot_to_row, layer.prob_perm, layer.out):
            t.view(torch.uint8).fill_(fill)
        layer.permute_index(torch.from_numpy(idx).cuda(), torch.from_numpy(prob).cuda())
        outs.append(layer.forward_mxfp4(mx._bf(x)).clone())
        assert layer.check_guards() == []
    assert torch.equal(outs[0], outs[1]) and mx._status() == 0
