"""The router in a training step: losses, permutation, the layer's forward and
backward, and the gradient of the logits from d(prob) and the losses, against
the oracles of the parts; and the operators used side by side."""
import numpy as np
import pytest

from mxfp8_grouped_gemm_x32_b200.workloads import bf16_bits_from_f32, bf16_bits_to_f32
from oracle import moe as omoe
from oracle import router as orouter

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _bf(bits):
    import torch
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


def _inputs(T, H, I, E, seed):
    rng = np.random.default_rng(seed)
    x = bf16_bits_from_f32(rng.normal(size=(T, H)).astype(np.float32))
    w1 = bf16_bits_from_f32((rng.normal(size=(E, 2 * I, H)) / np.sqrt(H)).astype(np.float32))
    w2 = bf16_bits_from_f32((rng.normal(size=(E, H, I)) / np.sqrt(I)).astype(np.float32))
    dy = bf16_bits_from_f32(rng.normal(size=(T, H)).astype(np.float32))
    logits = rng.normal(size=(T, E)).astype(np.float32)
    return x, w1, w2, dy, logits, rng.random(T) < 0.8


@pytest.mark.parametrize("recipe", ["mxfp8", "bf16"])
def test_step(recipe):
    import torch
    from mxfp8_grouped_gemm_x32_b200 import lib
    from mxfp8_grouped_gemm_x32_b200.layer import GroupedMLP
    T, H, I, E, k = 300, 256, 128, 8, 2
    x, w1, w2, dy, logits, mask = _inputs(T, H, I, E, 1)
    layer = GroupedMLP(T, H, I, E, k, mxfp8=recipe == "mxfp8", guard=4096)
    dz, dm = torch.from_numpy(logits).cuda(), torch.from_numpy(mask).cuda()
    dl = torch.tensor([0.01, 0.001], device="cuda")
    idx, prob, losses = layer.route_losses(dz, dm)
    if recipe == "mxfp8":
        layer.quantize_weights(_bf(w1), _bf(w2))
        layer.permute(_bf(x), idx, prob)
        layer.forward()
        dprob = layer.backward(_bf(dy))[3]
    else:
        layer.permute_index(idx, prob)
        layer.forward_bf16(_bf(x), _bf(w1), _bf(w2))
        dprob = layer.backward_bf16(_bf(dy), _bf(x), _bf(w1), _bf(w2))[3]
    grad = layer.route_backward(dz, dprob, dl, dm)
    torch.cuda.synchronize()
    assert lib.moe_get_device_status(0) == 0 and layer.check_guards() == []

    f = orouter.route_losses(logits, k, mask)
    assert np.array_equal(idx.cpu().numpy(), f["idx"])
    f64 = lambda b: bf16_bits_to_f32(b).astype(np.float64)
    p32 = prob.cpu().numpy()
    mode = dict(quantize=False, h_bf16=True) if recipe == "bf16" else {}
    fw = omoe.forward(f64(x), f64(w1), f64(w2), f["idx"], p32, **mode)
    mode = dict(quantize=False, bf16_held=True) if recipe == "bf16" else {}
    bw = omoe.backward(fw, f64(x), f64(w1), f64(w2), p32, f64(dy), **mode)
    dl64 = dl.cpu().numpy().astype(np.float64)
    got = grad.cpu().numpy().astype(np.float64)
    # the last step alone, from the device's own d(prob): fp32 arithmetic
    own = orouter.route_backward(f, dprob.cpu().numpy(), dl64)
    assert np.sqrt(np.mean((got - own) ** 2)) <= 1e-5 * np.sqrt(np.mean(own ** 2))
    # the whole step: d(prob) is held to 1e-2 of its rms, a masked token's too,
    # and the gradient is linear in it with |dz_e| <= 2 p |dprob|_max, k <= 2
    ref = orouter.route_backward(f, bw["dprob_f64"], dl64)
    assert np.all(got[~mask] == 0.0)
    assert np.sqrt(np.mean((got - ref) ** 2)) <= 2e-2 * np.sqrt(np.mean(bw["dprob_f64"] ** 2))
    # masked tokens leave no trace in the layer: probability 0, so no gradient of theirs
    assert np.all(p32[~mask] == 0.0)


def test_gradients_of_two_types_keep_their_buffers():
    """fp32 and bf16 logits of one layer: the first gradient stays as it was."""
    import torch
    from mxfp8_grouped_gemm_x32_b200.layer import GroupedMLP
    T, E, k = 257, 24, 3
    layer = GroupedMLP(T, 32, 64, E, k, backward=False, mxfp8=False)
    z = torch.randn(T, E, device="cuda")
    dp, dl = torch.randn(T, k, device="cuda"), torch.ones(2, device="cuda")
    layer.route_losses(z)
    want = layer.route_backward(z, dp, dl).clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        layer.route_losses(z)
        g32 = layer.route_backward(z, dp, dl)
    zb = z.bfloat16()
    layer.route_losses(zb)
    g16 = layer.route_backward(zb, dp, dl)
    assert g16.dtype == torch.bfloat16 and g32.dtype == torch.float32
    half = g16.clone()
    g32.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(g32, want) and torch.equal(g16, half)
    assert layer.route_backward(z, dp, dl).data_ptr() == g32.data_ptr()


def test_two_layers_on_two_streams():
    """Router, permutation and MXFP4 experts of two layers at the same time give
    what each gives alone."""
    import torch
    from mxfp8_grouped_gemm_x32_b200 import lib
    from mxfp8_grouped_gemm_x32_b200.layer import GroupedMLP
    H, I, E, k = 512, 256, 16, 4
    layers, calls, want = [], [], []
    for seed, T in ((1, 900), (2, 64)):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
        layer = GroupedMLP(T, H, I, E, k, backward=False, mxfp8=False)
        layer.quantize_weights_mxfp4((rand(E, 2 * I, H) / 22).bfloat16(), (rand(E, H, I) / 16).bfloat16())
        x, z, dp, dl = rand(T, H).bfloat16(), rand(T, E), rand(T, k), torch.ones(2, device="cuda")

        def call(layer=layer, x=x, z=z, dp=dp, dl=dl):
            idx, prob, losses = layer.route_losses(z)
            layer.permute_index(idx, prob)
            return layer.forward_mxfp4(x), losses, layer.route_backward(z, dp, dl)
        layers.append(layer)
        calls.append(call)
        want.append([t.clone() for t in call()])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(20):
        outs = []
        for s, call in zip(streams, calls):
            with torch.cuda.stream(s):
                outs.append(call())
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w))
    assert lib.moe_get_device_status(0) == 0


@pytest.mark.parametrize("H,I", [(32, 64), (288, 192), (416, 832), (2880, 64)])
def test_loaded_weights_with_tails(H, I):
    """Codes and plain scales as a checkpoint holds them, K past a multiple of
    256 in both GEMMs, against the layer's own quantiser."""
    import torch
    from mxfp8_grouped_gemm_x32_b200 import lib, mxfp4
    from mxfp8_grouped_gemm_x32_b200.layer import GroupedMLP
    T, E, k = 70, 3, 2
    g = torch.Generator(device="cuda").manual_seed(H)
    w1 = (torch.randn(E, 2 * I, H, device="cuda", generator=g) / 16).bfloat16()
    w2 = (torch.randn(E, H, I, device="cuda", generator=g) / 16).bfloat16()
    x = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    idx = torch.argsort(torch.rand(T, E, device="cuda", generator=g), 1)[:, :k].int().contiguous()
    prob = torch.rand(T, k, device="cuda", generator=g)

    def plain(w):
        codes, blocked = mxfp4.quantize(w)
        m, n, K = w.shape
        scales = torch.empty(m, n, K // 32, dtype=torch.uint8, device="cuda")
        lib.moe_mx_scales_from_blocked(blocked.data_ptr(), m, n, K, scales.data_ptr(), K // 32)
        return codes, scales
    a = GroupedMLP(T, H, I, E, k, backward=False, mxfp8=False, guard=4096)
    b = GroupedMLP(T, H, I, E, k, backward=False, mxfp8=False, guard=4096)
    a.quantize_weights_mxfp4(w1, w2)
    b.load_weights_mxfp4(*plain(w1), *plain(w2))
    outs = []
    for layer in (a, b):
        layer.permute_index(idx, prob)
        outs.append(layer.forward_mxfp4(x).clone())
        assert layer.check_guards() == []
    assert torch.equal(outs[0], outs[1]) and bool(torch.isfinite(outs[0].float()).all())
