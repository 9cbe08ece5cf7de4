"""MXFP4 on the GPU against the oracle: codes and scale bytes bit for bit, the
values they stand for exactly, and the expert MLP's forward within what fp32
accumulation leaves open.

Bar of the MLP, element by element and from oracle values only.  The GEMMs'
products of E2M1 values and power-of-two scales are exact; their fp32
accumulation is within acc_band (2^-22 sqrt(K sum t^2)) of the oracle's sum.
gate and up inside that band, and 2^-19 |h| for the fast exponential and
division, bound h; where h lies that near to a border between two codes, or its
block's |max| that near to a scale's border, either neighbour is right: D is the
largest change of the dequantised h over those alternatives, and |W_down| carries
it to the output.  The down GEMM adds its own band, the 24-bit rows drop less
than 2^-15 of a row's value, and the output's rounding to bf16 is half a step,
2^-8 relative.
"""
import numpy as np
import pytest

from mxfp8_grouped_gemm_x32_b200.workloads import bf16_bits_from_f32, bf16_bits_to_f32
from oracle import moe as omoe
from oracle import mxfp4 as o4
from tests.ambiguity import ACT, acc_band
from tests.mxutil import sf_padding_offsets, sf_unblock

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _bf(bits):
    import torch
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


def _status():
    from mxfp8_grouped_gemm_x32_b200 import lib
    return lib.moe_get_device_status(0)


# ---------------------------------------------------------------------- codec
def _check_codec(x64, dev, groups, rows, K):
    """x64 [groups*rows, K] float64 values of the device tensor `dev`."""
    import torch
    from mxfp8_grouped_gemm_x32_b200 import mxfp4
    codes, scales = mxfp4.quantize(dev)
    back = mxfp4.dequantize(codes, scales, dev.dtype)
    wide = mxfp4.dequantize(codes, scales, torch.float32)
    torch.cuda.synchronize()
    rc, rb = o4.quantize_rows(x64)
    sf = scales.cpu().numpy()
    gb = sf_unblock(sf, groups, rows, K).reshape(rb.shape)
    assert np.array_equal(gb, rb)
    assert np.all(sf[sf_padding_offsets(groups, rows, K)] == 0)
    gc = o4.unpack(codes.cpu().numpy().reshape(groups * rows, K // 2))
    fine = np.repeat(rb != o4.SCALE_NAN, 32, axis=1)
    # a zero code may carry the sign of what rounded to it on either side
    same = (gc == rc) | ((gc & 7 == 0) & (rc & 7 == 0))
    assert np.all(same[fine])
    assert np.array_equal(np.signbit(x64[fine]), (gc[fine] & 8) != 0)
    # a |max| above 1.75 * 2^127 has the scale 2^126 and rounds to the code of 4:
    # 2^128, which is infinity in both result types
    with np.errstate(over="ignore"):
        ref = o4.dequantize_rows(rc, rb).astype(np.float32).astype(np.float64)
    for t in (back, wide):
        got = t.float().cpu().numpy().astype(np.float64).reshape(ref.shape)
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        assert np.array_equal(got[fine], ref[fine])


@pytest.mark.parametrize("shape", [(1, 32), (32,), (3, 96), (127, 64), (128, 128), (129, 160), (5, 2880), (2, 70, 256),
                                   (3, 2, 33, 224), (1000, 1056), (257, 4096)])
@pytest.mark.parametrize("bf16", [True, False])
def test_quantize_shapes(shape, bf16):
    import torch
    rng = np.random.default_rng(sum(shape))
    x = rng.normal(size=shape) * np.exp(rng.uniform(-20, 20, size=shape[:-1] + (1,)))
    x = np.where(rng.random(shape[:-1] + (shape[-1] // 32,)).repeat(32, axis=-1) < 0.1, 0.0, x)
    if bf16:
        bits = bf16_bits_from_f32(x.astype(np.float32))
        dev, x64 = _bf(bits), bf16_bits_to_f32(bits).astype(np.float64)
    else:
        x = x.astype(np.float32)
        dev, x64 = torch.from_numpy(x).cuda(), x.astype(np.float64)
    rows = shape[-2] if len(shape) > 1 else 1
    groups = int(np.prod(shape)) // (rows * shape[-1])
    _check_codec(x64.reshape(groups * rows, shape[-1]), dev, groups, rows, shape[-1])


def test_every_bf16_value_and_every_border():
    """Each finite bf16 value as the largest of its block next to fractions
    that fall on every border between two codes; NaN and infinities."""
    bits = np.arange(1 << 16, dtype=np.uint16)
    top = bf16_bits_to_f32(np.where((bits & 0x7F80) == 0x7F80, 0, bits).astype(np.uint16)).astype(np.float64)
    frac = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.24, 0.26, 4.9, 5.1, 0.5, 1.0, 2.0]) / 6.0
    with np.errstate(over="ignore", under="ignore"):
        vals = bf16_bits_from_f32((top[:, None] * np.concatenate([frac, -frac])).astype(np.float32))
    x = np.concatenate([bits[:, None], vals, vals[:, :1]], axis=1).astype(np.uint16)
    with np.errstate(invalid="ignore"):
        x64 = bf16_bits_to_f32(x).astype(np.float64)
    _check_codec(x64, _bf(x), 1, 1 << 16, 32)


def test_fp32_extremes():
    import torch
    x = np.zeros((16, 32), np.float32)
    x[0, 0], x[1, 0], x[2, 0] = 1.4e-45, 1.17549435e-38, 3.4028235e38
    x[3, :2] = [3.4028235e38, -1e38]
    x[4, 0] = np.float32(6.0) * np.float32(2.0) ** 20
    x[5, 0] = np.nextafter(x[4, 0], np.float32(np.inf))
    x[6, 5], x[7, 6], x[8, 7] = np.nan, np.inf, -np.inf
    x[9] = 2.0 ** -127
    x[10] = 3e-45
    _check_codec(x.astype(np.float64), torch.from_numpy(x).cuda(), 1, 16, 32)


def test_empty_and_refusals():
    import torch
    from mxfp8_grouped_gemm_x32_b200 import mxfp4
    for shape in ((0, 64), (4, 0), (0, 3, 32)):
        c, s = mxfp4.quantize(torch.empty(shape, dtype=torch.bfloat16, device="cuda"))
        assert mxfp4.dequantize(c, s).shape == torch.Size(shape)
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    c, s = mxfp4.quantize(x)
    with pytest.raises(ValueError):
        mxfp4.quantize(x[:, :33].contiguous())
    with pytest.raises(ValueError):
        mxfp4.quantize(torch.zeros(64, 64, device="cuda").t()[:, :32])      # not contiguous
    with pytest.raises(TypeError):
        mxfp4.quantize(x.half())
    with pytest.raises(ValueError):
        mxfp4.dequantize(c, s[:-1])
    with pytest.raises(TypeError):
        mxfp4.dequantize(c, s, torch.float16)
    with pytest.raises(TypeError):
        mxfp4.dequantize(c.float(), s)
    buf = torch.zeros(8 * 64 + 1, dtype=torch.bfloat16, device="cuda")
    from mxfp8_grouped_gemm_x32_b200.lib import MoeError
    with pytest.raises(MoeError):
        mxfp4.quantize(buf[1:].view(8, 64))                                  # off a 16-byte boundary


# ------------------------------------------------------------------------ MLP
def _round_trip_with(v, s):
    return o4.decode(o4.encode(np.clip(v / s, -6.0, 6.0))) * s


def _h_ambiguity(h, band):
    """Largest change of the dequantised h over the values and scales inside
    its band (the round trip is monotone for a given scale, so the ends do)."""
    n, K = h.shape
    ref = o4.roundtrip_rows(h).reshape(n, -1, 32)
    hb, bb = h.reshape(n, -1, 32), band.reshape(n, -1, 32)
    amax, bmax = np.abs(hb).max(axis=2), bb.max(axis=2)
    D = np.zeros_like(hb)
    for am in (np.maximum(amax - bmax, 0.0), amax, amax + bmax):
        s = o4.scale_values(o4.scale_bytes(am))[:, :, None]
        for v in (hb - bb, hb + bb):
            D = np.maximum(D, np.abs(_round_trip_with(v, s) - ref))
    return D.reshape(n, K)


def _allowance(f, shape):
    allow = np.zeros(shape)
    for q in f["parts"]:
        ba = acc_band(q["a"], q["w1q"])
        I = q["h"].shape[1]
        sg = omoe.sigmoid(q["g"])
        slope = np.abs(sg * (1.0 + q["g"] * (1.0 - sg)))
        band = np.abs(q["p"]) * (slope * np.abs(q["u"]) * ba[:, :I] + np.abs(omoe.silu(q["g"])) * ba[:, I:]
                                 + ba[:, :I] * ba[:, I:]) + ACT * np.abs(q["h"])
        hq = o4.roundtrip_rows(q["h"])
        y = _h_ambiguity(q["h"], band) @ np.abs(q["w2q"]).T + acc_band(hq, q["w2q"]) + 2.0 ** -15 * np.abs(q["y"])
        np.add.at(allow, q["t"], y)
    return allow


def _problem(T, H, I, E, k, seed, idx=None):
    rng = np.random.default_rng(seed)
    x = bf16_bits_from_f32(rng.normal(size=(T, H)).astype(np.float32))
    w1 = bf16_bits_from_f32((rng.normal(size=(E, 2 * I, H)) / np.sqrt(H)).astype(np.float32))
    w2 = bf16_bits_from_f32((rng.normal(size=(E, H, I)) / np.sqrt(I)).astype(np.float32))
    if idx is None:
        idx = np.argsort(rng.random((T, E)), axis=1)[:, :k]
    prob = rng.random((T, k)).astype(np.float32)
    return x, w1, w2, np.ascontiguousarray(idx, np.int32), prob


def _layer(T, H, I, E, k, w1=None, w2=None):
    from mxfp8_grouped_gemm_x32_b200.layer import GroupedMLP
    layer = GroupedMLP(T, H, I, E, k, backward=False, mxfp8=False, guard=4096)
    if w1 is not None:
        layer.quantize_weights_mxfp4(_bf(w1), _bf(w2))
    return layer


def _check_out(out, x, w1, w2, idx, prob):
    f = o4.forward(bf16_bits_to_f32(x), bf16_bits_to_f32(w1), bf16_bits_to_f32(w2), idx, prob)
    allow = _allowance(f, f["out"].shape)
    got = out.float().cpu().numpy().astype(np.float64)
    bar = allow + 2.0 ** -8 * (np.abs(f["out"]) + allow) + 1e-37
    assert np.all(np.abs(got - f["out"]) <= bar), float(np.max(np.abs(got - f["out"]) / bar))
    # and as a whole: without the allowance only the roundings that are always there
    rms = np.sqrt(np.mean(f["out"] ** 2))
    if rms > 0:
        assert np.sqrt(np.mean((got - f["out"]) ** 2)) <= 1e-2 * rms


@pytest.mark.parametrize("T,H,I,E,k", [
    (1, 32, 64, 1, 1),          # one scale atom, one MMA, one row
    (1, 256, 512, 8, 8),        # a single token on every expert
    (3, 96, 64, 4, 4),          # K = 96: half an instruction past K
    (9, 160, 192, 3, 2),        # atoms and instructions cut on both sides
    (127, 288, 320, 1, 1), (128, 256, 128, 1, 1), (129, 256, 128, 1, 1),   # around one row tile
    (64, 416, 448, 5, 2),       # T k = 128: the A box's limit
    (63, 512, 256, 4, 2),
    (300, 544, 640, 6, 3),
    (40, 2880, 192, 3, 2), (40, 192, 2880, 3, 2),
    (700, 1024, 384, 16, 4),
])
def test_forward(T, H, I, E, k):
    import torch
    x, w1, w2, idx, prob = _problem(T, H, I, E, k, seed=T + H + I)
    layer = _layer(T, H, I, E, k, w1, w2)
    layer.permute_index(torch.from_numpy(idx).cuda(), torch.from_numpy(prob).cuda())
    out = layer.forward_mxfp4(_bf(x))
    torch.cuda.synchronize()
    assert _status() == 0 and layer.check_guards() == []
    _check_out(out, x, w1, w2, idx, prob)


@pytest.mark.parametrize("kind", ["one expert", "skewed", "one listed twice", "rejected ids"])
def test_routings(kind):
    import torch
    T, H, I, E, k = 333, 256, 192, 7, 3
    rng = np.random.default_rng(4)
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k]
    if kind == "one expert":
        idx[:] = 5
    elif kind == "skewed":
        idx[:, 0] = np.where(rng.random(T) < 0.9, 2, idx[:, 0])
        idx[idx == 6] = 0                                    # an empty expert
    elif kind == "one listed twice":
        idx[:, 1] = idx[:, 0]
    else:
        idx[::5, 1] = -1
        idx[1::7, 2] = E
    x, w1, w2, idx, prob = _problem(T, H, I, E, k, seed=5, idx=idx)
    layer = _layer(T, H, I, E, k, w1, w2)
    layer.permute_index(torch.from_numpy(idx).cuda(), torch.from_numpy(prob).cuda())
    out = layer.forward_mxfp4(_bf(x))
    torch.cuda.synchronize()
    assert _status() == (5 if kind == "rejected ids" else 0) and layer.check_guards() == []
    _check_out(out, x, w1, w2, idx, prob)


def test_loaded_weights_equal_quantised_ones():
    """Codes and plain scales as a checkpoint holds them give the same bits."""
    import torch
    T, H, I, E, k = 50, 288, 192, 4, 2
    x, w1, w2, idx, prob = _problem(T, H, I, E, k, seed=8)
    a, b = _layer(T, H, I, E, k, w1, w2), _layer(T, H, I, E, k)
    host = []
    for w in (w1, w2):
        c, s = o4.quantize_rows(bf16_bits_to_f32(w).astype(np.float64).reshape(-1, w.shape[2]))
        host += [o4.pack(c).reshape(*w.shape[:2], -1), s.reshape(*w.shape[:2], -1)]
    b.load_weights_mxfp4(*(torch.from_numpy(h).cuda() for h in host))
    outs = []
    for layer in (a, b):
        layer.permute_index(torch.from_numpy(idx).cuda(), torch.from_numpy(prob).cuda())
        outs.append(layer.forward_mxfp4(_bf(x)).clone())
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])
    assert b.check_guards() == []


def test_non_finite_tokens_stay_alone():
    """A NaN or infinity in a token reaches that token's output only."""
    import torch
    T, H, I, E, k = 150, 256, 192, 4, 2
    x, w1, w2, idx, prob = _problem(T, H, I, E, k, seed=9)
    clean = _layer(T, H, I, E, k, w1, w2)
    di, dp = torch.from_numpy(idx).cuda(), torch.from_numpy(prob).cuda()
    clean.permute_index(di, dp)
    ref = clean.forward_mxfp4(_bf(x)).clone()
    x[17, 3], x[90, 200] = 0x7FC0, 0x7F80
    clean.permute_index(di, dp)
    out = clean.forward_mxfp4(_bf(x))
    torch.cuda.synchronize()
    others = torch.ones(T, dtype=torch.bool, device="cuda")
    others[[17, 90]] = False
    assert torch.isnan(out[17]).all() and torch.isnan(out[90]).all()
    assert torch.equal(out[others], ref[others])


def test_zero_tokens_and_zero_values():
    import torch
    from mxfp8_grouped_gemm_x32_b200 import lib
    _, w1, w2, _, _ = _problem(1, 64, 64, 2, 1, seed=1)
    empty = _layer(0, 64, 64, 2, 1, w1, w2)
    empty.permute_index(torch.empty(0, 1, dtype=torch.int32, device="cuda"), torch.empty(0, 1, device="cuda"))
    assert empty.forward_mxfp4(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")).shape == (0, 64)
    layer = _layer(5, 64, 64, 2, 2, w1, w2)
    layer.permute_index(torch.tensor([[0, 1]] * 5, dtype=torch.int32, device="cuda"), torch.ones(5, 2, device="cuda"))
    layer.out.fill_(7.0)
    out = layer.forward_mxfp4(torch.zeros(5, 64, dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(out, torch.zeros_like(out)) and lib.moe_get_device_status(0) == 0


def test_refusals():
    import torch
    from mxfp8_grouped_gemm_x32_b200.layer import GroupedMLP
    _, w1, w2, _, _ = _problem(1, 64, 64, 2, 1, seed=1)
    layer = _layer(4, 64, 64, 2, 1)
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(RuntimeError):
        layer.forward_mxfp4(x)                               # no weights yet
    layer.quantize_weights_mxfp4(_bf(w1), _bf(w2))
    for bad, exc in ((x.float(), TypeError), (x[:3], ValueError), (x.cpu(), ValueError),
                     (torch.zeros(64, 4, dtype=torch.bfloat16, device="cuda").t(), ValueError)):
        with pytest.raises(exc):
            layer.forward_mxfp4(bad)
    with pytest.raises(TypeError):
        layer.quantize_weights_mxfp4(_bf(w1).float(), _bf(w2))
    for call in (lambda: layer.forward(), lambda: layer.quantize_weights(_bf(w1), _bf(w2)),
                 lambda: layer.permute(x, layer.topk_idx, layer.topk_prob)):
        with pytest.raises(RuntimeError):
            call()                                           # built without the MXFP8 buffers
    small = GroupedMLP(4, 64, 64, 2, 1, backward=False)
    with pytest.raises(RuntimeError):
        small.route_backward(torch.zeros(4, 2, device="cuda"))


def test_graphs_and_streams():
    """Two layers of one process, replayed from graphs in turn and called from a
    side stream, keep apart."""
    import torch
    T, H, I, E, k = 90, 256, 192, 4, 2
    probs = [_problem(T, H, I, E, k, seed=s) for s in (20, 21)]
    want, graphs, layers, ins = [], [], [], []
    for x, w1, w2, idx, prob in probs:
        layer = _layer(T, H, I, E, k, w1, w2)
        dx, di, dp = _bf(x), torch.from_numpy(idx).cuda(), torch.from_numpy(prob).cuda()
        layer.permute_index(di, dp)
        want.append(layer.forward_mxfp4(dx).clone())
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.permute_index(di, dp)
            layer.forward_mxfp4(dx)
        layers.append(layer)
        graphs.append(g)
        ins.append((dx, di, dp))
    for layer in layers:
        layer.out.zero_()
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(la.out, w) for la, w in zip(layers, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layers[0].out.zero_()
        layers[0].permute_index(*ins[0][1:])
        layers[0].forward_mxfp4(ins[0][0])
    side.synchronize()
    assert torch.equal(layers[0].out, want[0])


def test_router_then_mlp():
    """The serving sequence: router, permutation, MXFP4 experts."""
    import torch
    T, H, I, E, k = 37, 256, 192, 12, 3
    x, w1, w2, _, _ = _problem(T, H, I, E, k, seed=30)
    layer = _layer(T, H, I, E, k, w1, w2)
    logits = torch.from_numpy(np.random.default_rng(31).normal(size=(T, E)).astype(np.float32)).cuda()
    idx, prob, _ = layer.route_losses(logits)
    layer.permute_index(idx, prob)
    out = layer.forward_mxfp4(_bf(x))
    torch.cuda.synchronize()
    _check_out(out, x, w1, w2, idx.cpu().numpy(), prob.cpu().numpy())
