"""Every call of the layer launches with the layer's device current, whichever
device the caller has current.  On the CPU: the library's functions and the
device context are replaced by recorders."""
import contextlib

import pytest
import torch

from mxfp8_grouped_gemm_x32_b200 import layer as layer_module
from mxfp8_grouped_gemm_x32_b200 import lib

T, H, I, E, k = 4, 32, 64, 2, 1
SIZES = ("moe_mx_scale_bytes", "moe_padded_rows", "moe_workspace_size", "moe_mxfp4_tiled_scale_bytes")


@pytest.fixture
def recorded(monkeypatch):
    """[(function, device that was current, stream)] of the library calls made."""
    current, calls = [], []

    @contextlib.contextmanager
    def on_device(dev):
        current.append(dev)
        yield
        current.pop()

    monkeypatch.setattr(layer_module, "on_device", on_device)
    monkeypatch.setattr(layer_module, "_raw_stream", lambda index: 99)
    for name in lib.EXPORTED:
        if name not in SIZES and hasattr(lib, name):
            monkeypatch.setattr(lib, name, lambda *a, _n=name: calls.append((_n, current[-1] if current else None, a[-1])) or 0)
    return calls


def _tensors():
    bf = dict(dtype=torch.bfloat16)
    return dict(x=torch.zeros(T, H, **bf), w1=torch.zeros(E, 2 * I, H, **bf), w2=torch.zeros(E, H, I, **bf),
                dY=torch.zeros(T, H, **bf), idx=torch.zeros(T, k, dtype=torch.int32), prob=torch.zeros(T, k),
                z=torch.zeros(T, E), mask=torch.ones(T, dtype=torch.bool), dl=torch.zeros(2),
                c1=torch.zeros(E, 2 * I, H // 2, dtype=torch.uint8), s1=torch.zeros(E, 2 * I, H // 32, dtype=torch.uint8),
                c2=torch.zeros(E, H, I // 2, dtype=torch.uint8), s2=torch.zeros(E, H, I // 32, dtype=torch.uint8))


CALLS = {
    "quantize_weights": lambda L, t: L.quantize_weights(t["w1"], t["w2"]),
    "route": lambda L, t: L.route(t["z"]),
    "route_permute": lambda L, t: L.route_permute(t["z"], t["x"]),
    "permute": lambda L, t: L.permute(t["x"], t["idx"], t["prob"], with_cols=True),
    "permute_index": lambda L, t: L.permute_index(t["idx"], t["prob"]),
    "forward": lambda L, t: L.forward(),
    "backward": lambda L, t: L.backward(t["dY"], t["x"]),
    "forward_bf16": lambda L, t: L.forward_bf16(t["x"], t["w1"], t["w2"]),
    "backward_bf16": lambda L, t: L.backward_bf16(t["dY"], t["x"], t["w1"], t["w2"]),
    "fp8_tensor": lambda L, t: (L.forward_fp8_tensor(t["x"], t["w1"], t["w2"]),
                                L.backward_fp8_tensor(t["dY"], t["x"], t["w1"], t["w2"])),
    "router training": lambda L, t: (L.route_losses(t["z"], t["mask"]), L.route_backward(t["z"], t["prob"], t["dl"])),
    "mxfp4": lambda L, t: (L.quantize_weights_mxfp4(t["w1"], t["w2"]), L.permute_index(t["idx"], t["prob"]),
                           L.forward_mxfp4(t["x"])),
    "mxfp4 loaded": lambda L, t: L.load_weights_mxfp4(t["c1"], t["s1"], t["c2"], t["s2"]),
    "step": lambda L, t: L.step(t["x"], t["idx"], t["prob"], t["w1"], t["w2"], t["dY"]),
    "device_status": lambda L, t: L.device_status(),
}


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("backward", [False, True])
def test_launches_on_the_layers_device(recorded, name, backward):
    if not backward and ("backward" in name or name in ("fp8_tensor", "step")):
        pytest.skip("needs the backward's buffers")
    L = layer_module.GroupedMLP(T, H, I, E, k, device="cpu", backward=backward)
    CALLS[name](L, _tensors())
    assert recorded
    assert all(dev == L.dev for _, dev, _ in recorded), recorded
    assert all(stream == 99 for _, _, stream in recorded), recorded


def test_forward_mxfp4_needs_a_permutation(recorded):
    """Without one the row maps hold whatever the memory held, and the kernels would read by it."""
    t = _tensors()
    L = layer_module.GroupedMLP(T, H, I, E, k, device="cpu", backward=False, mxfp8=False)
    L.load_weights_mxfp4(t["c1"], t["s1"], t["c2"], t["s2"])
    recorded.clear()
    with pytest.raises(RuntimeError, match="permute"):
        L.forward_mxfp4(t["x"])
    assert recorded == []
    L.route(t["z"])
    with pytest.raises(RuntimeError, match="permute"):
        L.forward_mxfp4(t["x"])
    L.permute_index(t["idx"], t["prob"])
    L.forward_mxfp4(t["x"])
    assert recorded[-1][0] == "moe_grouped_mlp_fwd_mxfp4"
    for permute in ("permute", "route_permute"):
        L = layer_module.GroupedMLP(T, H, I, E, k, device="cpu", backward=False)
        L.load_weights_mxfp4(t["c1"], t["s1"], t["c2"], t["s2"])
        CALLS[permute](L, t)
        L.forward_mxfp4(t["x"])
        assert recorded[-1][0] == "moe_grouped_mlp_fwd_mxfp4"
