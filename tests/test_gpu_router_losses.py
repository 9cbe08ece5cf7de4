"""Router losses and gradient (moe_router_losses, moe_router_bwd) against the
oracle on the same logits.

Bars, for logits within 30 of their row's maximum.  ids, counts and tokens
exact; probabilities within 4e-6 relative (expf 2 ulp, its argument's rounding,
up to 31 additions, a division: (30 + 35) 2^-24).  lse = m + log(sum): the sum
carries at most (30 + 20) 2^-24 relative, which the logarithm turns into an
absolute error, plus one rounding of the result: 6e-6 + 2^-23 |lse|.  The sums
over tokens have only positive terms, each with (50) 2^-24 relative and at
most 40 additions after it: 1e-5 relative.  The z-loss: twice lse's error
times |lse| on the mean, and those additions.  Gradient: s = exp(z - lse)
carries lse's error, the difference's rounding and expf's, 1e-5 in all; it
enters each term at most twice, with four more roundings: 3e-5 of the sum of
the terms' magnitudes, element by element; a bf16 result is off by half a
step more (2^-8).
"""
import numpy as np
import pytest

from mxfp8_grouped_gemm_x32_b200.workloads import bf16_bits_from_f32, bf16_bits_to_f32, get_config, make_inputs
from oracle import router as orouter

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _layer(T, E, k):
    from mxfp8_grouped_gemm_x32_b200.layer import GroupedMLP
    return GroupedMLP(T, 32, 64, E, k, backward=False, mxfp8=False, guard=4096)


def _device(a, bf16=False):
    import torch
    if bf16:
        return torch.from_numpy(bf16_bits_from_f32(a).view(np.int16)).view(torch.bfloat16).cuda()
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()


def _status():
    from mxfp8_grouped_gemm_x32_b200 import lib
    return lib.moe_get_device_status(0)


def _check_forward(layer, idx, prob, losses, f):
    assert np.array_equal(idx.cpu().numpy(), f["idx"])
    gp = prob.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(gp), np.isnan(f["prob"]))
    ok = np.isfinite(f["prob"])
    assert np.all(np.abs(gp - f["prob"])[ok] <= 4e-6 * f["prob"][ok] + 1e-30)
    assert np.array_equal(layer.expert_counts.cpu().numpy(), f["counts"])
    assert int(layer.routed_tokens) == f["n"]
    lse = layer.router_lse.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(lse - f["lse"]) <= 6e-6 + 2.0 ** -23 * np.abs(f["lse"]))
    assert np.all(np.abs(layer.prob_sums.cpu().numpy() - f["sums"]) <= 1e-5 * f["sums"] + 1e-30)
    gl = losses.cpu().numpy().astype(np.float64)
    assert abs(gl[0] - f["losses"][0]) <= 2e-5 * abs(f["losses"][0])
    zl = 2 * np.mean(np.abs(f["lse"][f["live"]]) * (6e-6 + 2.0 ** -23 * np.abs(f["lse"][f["live"]]))) if f["n"] else 0.0
    assert abs(gl[1] - f["losses"][1]) <= zl + 1e-5 * f["losses"][1]


def _grad_bar(f, E, dprob, dlosses, bf16):
    """Reference gradient and what the device's may be off by."""
    T, k, n = f["s"].shape[0], f["k"], max(1, f["n"])
    ref = orouter.route_backward(f, dprob, dlosses)
    mag = np.zeros((T, E))
    if dlosses is not None:
        sh = f["counts"] / (n * k)
        fs = f["s"] @ sh
        mag += f["s"] * (abs(dlosses[0]) * E / n * (sh + fs[:, None]) + abs(dlosses[1]) * 2 / n * np.abs(f["lse"])[:, None])
    if dprob is not None:
        p, dp = f["prob"], np.abs(dprob)
        np.add.at(mag, (np.arange(T)[:, None], f["idx"]), p * (dp + np.sum(p * dp, axis=1, keepdims=True)))
    mag = np.where(f["live"][:, None], mag, 0.0)
    return ref, 3e-5 * mag + (2.0 ** -8 * np.abs(ref) if bf16 else 0.0) + 1e-30


def _run(z, k, mask=None, bf16=False, dprob=True, dlosses=(0.3, 0.1), seed=0):
    import torch
    T, E = z.shape
    rng = np.random.default_rng(seed)
    dz = _device(z, bf16)
    ref_in = bf16_bits_to_f32(bf16_bits_from_f32(z)) if bf16 else z.astype(np.float32)
    dm = None if mask is None else torch.from_numpy(mask).cuda()
    dp = rng.normal(size=(T, k)).astype(np.float32) if dprob else None
    layer = _layer(T, E, k)
    idx, prob, losses = layer.route_losses(dz, dm)
    dl = None if dlosses is None else torch.tensor(dlosses, dtype=torch.float32, device="cuda")
    g = layer.route_backward(dz, None if dp is None else torch.from_numpy(dp).cuda(), dl, dm)
    torch.cuda.synchronize()
    assert _status() == 0 and layer.check_guards() == []
    f = orouter.route_losses(ref_in, k, mask)
    _check_forward(layer, idx, prob, losses, f)
    dl32 = None if dlosses is None else np.array(dlosses, np.float32).astype(np.float64)
    ref, bar = _grad_bar(f, E, dp, dl32, bf16)
    assert g.dtype == dz.dtype
    got = g.float().cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - ref) <= bar), float(np.max(np.abs(got - ref) - bar))
    assert np.all(got[~f["live"]] == 0.0)
    return layer


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 8), (7, 2, 1), (33, 9, 3), (100, 16, 16), (257, 17, 2),
                                   (64, 33, 32), (500, 60, 6), (129, 100, 5), (1000, 128, 8), (77, 129, 4),
                                   (300, 200, 7), (900, 256, 32), (5000, 256, 1)])
@pytest.mark.parametrize("bf16", [False, True])
def test_shapes(T, E, k, bf16):
    rng = np.random.default_rng(T + E)
    _run(rng.normal(size=(T, E)) * 3, k, bf16=bf16)


@pytest.mark.parametrize("T,E,k", [(300, 5, 5), (300, 8, 3), (200, 16, 16), (200, 29, 20), (200, 32, 32), (200, 60, 31),
                                   (200, 128, 12), (200, 256, 32)])
def test_same_bits_as_the_plain_router(T, E, k):
    import torch
    z = _device(np.random.default_rng(E + k).normal(size=(T, E)) * 2)
    layer = _layer(T, E, k)
    idx, prob, _ = layer.route_losses(z)
    idx, prob = idx.clone(), prob.clone()
    i2, p2 = layer.route(z)
    assert torch.equal(idx, i2) and torch.equal(prob, p2)


@pytest.mark.parametrize("name", ["tiny", "gpt_oss_20b", "qwen3_30b_ragged"])
def test_workload_logits(name):
    cfg = get_config(name)
    z = make_inputs(cfg, seed=1, weights=False, grad=False)["router_logits"]
    mask = np.random.default_rng(2).random(cfg.T) < 0.7
    _run(z, cfg.k, mask=mask)


@pytest.mark.parametrize("E", [33, 40, 63, 64, 65, 72, 100, 128, 129, 136, 200, 256])
@pytest.mark.parametrize("k", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("bf16", [False, True])
def test_many_experts_with_few_kept(E, k, bf16):
    rng = np.random.default_rng(E * k)
    _run(rng.normal(size=(601, E)) * 2 + rng.normal(size=E), k, bf16=bf16, mask=rng.random(601) < 0.9)


@pytest.mark.parametrize("E", [62, 96, 250])
@pytest.mark.parametrize("kind", ["all equal", "two values", "five values", "rising", "falling", "one lane", "two lanes",
                                  "minus infinity", "zeros of both signs", "zero rows"])
def test_many_experts_with_ties(E, kind):
    rng = np.random.default_rng(E)
    T = 515
    z = {"all equal": lambda: np.full((T, E), 0.25),
         "two values": lambda: rng.integers(0, 2, (T, E)) * 1.0,
         "five values": lambda: rng.integers(0, 5, (T, E)) * 0.5,
         "rising": lambda: np.tile(np.arange(E) / 16.0, (T, 1)),
         "falling": lambda: np.tile(-np.arange(E) / 16.0, (T, 1)),
         "one lane": lambda: np.where(np.arange(E)[None, :] // 16 == rng.integers(0, E // 16, (T, 1)), 4.0, 0.0)
                             + np.round(rng.normal(size=(T, E)) * 4) / 4,
         "two lanes": lambda: np.where(np.arange(E)[None, :] // 16 % 2 == np.arange(T)[:, None] % 2, 9.0, 0.0)
                              + rng.normal(size=(T, E)),
         "zero rows": lambda: np.where(rng.random((T, 1)) < 0.5, 0.0, rng.normal(size=(T, E))),
         "minus infinity": lambda: np.where(rng.random((T, E)) < 0.97, -np.inf, rng.normal(size=(T, E))),
         "zeros of both signs": lambda: np.where(rng.random((T, E)) < 0.5, 0.0, -0.0)}[kind]()
    if kind == "minus infinity":
        z[:, 3] = 0.0  # no row without a finite logit
    _run(z, 7)


@pytest.mark.parametrize("k", [4, 8])
def test_many_experts_with_odd_logits_behind_the_mask(k):
    rng = np.random.default_rng(k)
    T, E = 700, 200
    z = rng.normal(size=(T, E))
    mask = rng.random(T) < 0.5
    bad = np.flatnonzero(~mask)
    z[bad[0::4]] = np.nan
    z[bad[1::4]] = np.inf
    z[bad[2::4]] = -np.inf
    z[bad[3::4], ::3] = np.nan
    _run(z, k, mask=mask)


@pytest.mark.parametrize("E,k", [(128, 8), (256, 8), (256, 3), (100, 4)])
def test_many_tokens_same_bits_as_the_plain_router(E, k):
    import torch
    T = 20011  # several tokens for every group of lanes
    z = _device(np.random.default_rng(E + k).normal(size=(T, E)) * 2)
    layer = _layer(T, E, k)
    idx, prob, losses = layer.route_losses(z)
    idx, prob, losses, counts = idx.clone(), prob.clone(), losses.clone(), layer.expert_counts.clone()
    i2, p2 = layer.route(z)
    assert torch.equal(idx, i2) and torch.equal(prob, p2)
    assert torch.equal(counts.long(), torch.bincount(idx.flatten().long(), minlength=E))
    _, _, again = layer.route_losses(z)
    assert torch.equal(losses, again)


def test_ties():
    rng = np.random.default_rng(5)
    z = np.round(rng.normal(size=(999, 40)) * 2) / 2
    z[::7] = 1.0
    _run(z, 6)


@pytest.mark.parametrize("kind", ["none", "all but one", "anything behind the mask"])
def test_masks(kind):
    rng = np.random.default_rng(9)
    T, E, k = 211, 24, 3
    z = rng.normal(size=(T, E))
    mask = np.zeros(T, bool)
    if kind == "all but one":
        mask[100] = True
    if kind == "anything behind the mask":
        mask = rng.random(T) < 0.5
        bad = np.flatnonzero(~mask)
        z[bad[0::4]] = np.nan
        z[bad[1::4]] = np.inf
        z[bad[2::4]] = -np.inf
        z[bad[3::4]] = -3.4e38
    _run(z, k, mask=mask)


def test_minus_infinity_logits():
    """Experts switched off by -inf: no probability, no gradient; kept all the
    same where fewer than k are left."""
    rng = np.random.default_rng(11)
    z = rng.normal(size=(130, 12))
    z[:, 5:10] = -np.inf
    z[::3, 2:] = -np.inf
    z[1::3] = np.where(z[1::3] == -np.inf, -3.4028235e38, z[1::3])      # the type's lowest value
    _run(z, 4)


@pytest.mark.parametrize("E,k", [(12, 4), (48, 6), (128, 2), (200, 8), (256, 20)])
def test_rows_of_the_lowest_value_and_huge_logits(E, k):
    """Rows whose experts are all switched off by the type's lowest value are
    rows of equal logits; the softmax holds at any magnitude."""
    import torch
    rng = np.random.default_rng(E)
    T = 700
    low = -3.4028234663852886e38
    z = rng.normal(size=(T, E)).astype(np.float32)
    z[0::7] = low
    z[1::7, E // 2:] = low
    z[2::7] *= np.float32(3e37)
    z[3::7] = np.float32(3.4e38)
    z[4::7] += np.float32(1e8)
    z[5::7] -= np.float32(3e5)
    layer = _layer(T, E, k)
    dz = _device(z)
    idx, prob, losses = layer.route_losses(dz)
    dp = rng.normal(size=(T, k)).astype(np.float32)
    g = layer.route_backward(dz, torch.from_numpy(dp).cuda(), torch.tensor([0.3, 0.0], device="cuda"))
    f = orouter.route_losses(z, k)
    assert np.array_equal(idx.cpu().numpy(), f["idx"])
    assert np.array_equal(layer.expert_counts.cpu().numpy(), f["counts"])
    gp = prob.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(gp - f["prob"]) <= 4e-6 * f["prob"] + 1e-30)
    lse = layer.router_lse.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(lse - f["lse"]) <= 6e-6 + 2.0 ** -23 * np.abs(f["lse"]))
    assert np.all(np.abs(layer.prob_sums.cpu().numpy() - f["sums"]) <= 1e-5 * f["sums"] + 1e-30)
    assert abs(float(losses[0]) - f["losses"][0]) <= 2e-5 * f["losses"][0]
    assert float(losses[1]) == np.inf                # the square passes fp32
    ref, bar = _grad_bar(f, E, dp, np.array([np.float32(0.3), 0.0], np.float64), False)
    got = g.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - ref) <= bar), float(np.max(np.abs(got - ref) - bar))


@pytest.mark.parametrize("E,k", [(48, 6), (100, 4), (200, 8)])
def test_nan_and_infinity_among_many_experts(E, k):
    import torch
    rng = np.random.default_rng(E)
    T = 640
    z = rng.normal(size=(T, E)).astype(np.float32)
    z[3, 4], z[9, 0], z[20], z[33, ::2] = np.nan, np.inf, -np.inf, np.nan
    layer = _layer(T, E, k)
    dz = _device(z)
    idx, prob, losses = layer.route_losses(dz)
    g = layer.route_backward(dz, torch.ones(T, k, device="cuda"), torch.ones(2, device="cuda"))
    idx, prob = idx.clone(), prob.clone()
    i2, p2 = layer.route(dz)
    f = orouter.route_losses(z, k)
    assert np.array_equal(idx.cpu().numpy(), f["idx"]) and torch.equal(idx, i2)
    assert torch.equal(prob.view(torch.int32)[~torch.isnan(prob)], p2.view(torch.int32)[~torch.isnan(p2)])
    assert torch.isnan(losses).all()
    clean = torch.ones(T, dtype=torch.bool, device="cuda")
    clean[[3, 9, 20, 33]] = False
    assert torch.isfinite(g[clean]).all() and torch.isnan(g[~clean]).any(1).all()


def test_nan_and_infinity_stay_in_their_tokens():
    import torch
    rng = np.random.default_rng(12)
    z = rng.normal(size=(64, 20)).astype(np.float32)
    z[3, 4], z[9, 0], z[20] = np.nan, np.inf, -np.inf
    layer = _layer(64, 20, 2)
    dz = _device(z)
    idx, prob, losses = layer.route_losses(dz)
    dp = torch.ones(64, 2, device="cuda")
    g = layer.route_backward(dz, dp, torch.ones(2, device="cuda"))
    torch.cuda.synchronize()
    f = orouter.route_losses(z, 2)
    assert np.array_equal(idx.cpu().numpy(), f["idx"])
    assert torch.isnan(losses).all()
    clean = np.setdiff1d(np.arange(64), [3, 9, 20])
    assert torch.isfinite(g[torch.from_numpy(clean).cuda()]).all()
    assert torch.isnan(g[3]).all() and torch.isnan(g[20]).any()


@pytest.mark.parametrize("dprob,dlosses", [(True, None), (False, (1.0, 0.0)), (False, (0.0, 1.0)), (False, None)])
def test_gradients_apart(dprob, dlosses):
    rng = np.random.default_rng(13)
    _run(rng.normal(size=(400, 48)), 5, dprob=dprob, dlosses=dlosses)


def test_ids_listed_twice_and_out_of_range():
    import torch
    rng = np.random.default_rng(14)
    T, E, k = 10, 12, 3
    z = rng.normal(size=(T, E))
    layer = _layer(T, E, k)
    dz = _device(z)
    layer.route_losses(dz)
    torch.cuda.synchronize()
    layer.topk_idx[2] = torch.tensor([7, 7, 1], dtype=torch.int32)
    layer.topk_idx[4, 1] = E
    layer.topk_idx[5, 2] = -1
    dp = rng.normal(size=(T, k)).astype(np.float32)
    g = layer.route_backward(dz, torch.from_numpy(dp).cuda())
    torch.cuda.synchronize()
    assert _status() == 5
    p = layer.topk_prob.cpu().numpy().astype(np.float64)
    inner = p * (dp - np.sum(p * dp, axis=1, keepdims=True))
    ref = np.zeros((T, E))
    idx = layer.topk_idx.cpu().numpy()
    for t in range(T):
        for j in range(k):
            if 0 <= idx[t, j] < E:
                ref[t, idx[t, j]] += inner[t, j]
    # p and dot carry 4e-6 of magnitudes below 4, then two roundings
    assert np.max(np.abs(g.cpu().numpy() - ref)) <= 5e-5


def test_out_of_range_id_is_recorded():
    import torch
    layer = _layer(4, 8, 2)
    dz = _device(np.zeros((4, 8)))
    layer.route_losses(dz)
    layer.topk_idx[1, 0] = 8
    layer.route_backward(dz, torch.zeros(4, 2, device="cuda"))
    assert _status() == 5
    assert _status() == 0


def test_empty_batch():
    import torch
    layer = _layer(0, 8, 2)
    z = torch.empty(0, 8, device="cuda")
    _, _, losses = layer.route_losses(z)
    layer.route_backward(z, None, torch.ones(2, device="cuda"))
    torch.cuda.synchronize()
    assert losses.tolist() == [0.0, 0.0] and int(layer.expert_counts.sum()) == 0 and int(layer.routed_tokens) == 0


def test_unaligned_rows_and_repeatable_bits():
    """A view that starts off a 16-byte boundary takes the element-wise loads
    and gives the same bits as an aligned copy; so does a second run."""
    import torch
    rng = np.random.default_rng(15)
    T, E, k = 300, 64, 4
    buf = torch.zeros(T * E + 1, device="cuda")
    buf[1:] = _device(rng.normal(size=(T * E,)))
    view, copy = buf[1:].view(T, E), buf[1:].clone().view(T, E)
    out = []
    for z in (view, copy, copy):
        layer = _layer(T, E, k)
        idx, prob, losses = layer.route_losses(z)
        g = layer.route_backward(z, torch.ones(T, k, device="cuda"), torch.ones(2, device="cuda"))
        out.append([t.clone() for t in (idx, prob, losses, layer.prob_sums, g)])
    for other in out[1:]:
        assert all(torch.equal(a, b) for a, b in zip(out[0], other))


def test_captured_graph_and_another_stream():
    import torch
    rng = np.random.default_rng(16)
    T, E, k = 700, 96, 4
    z = _device(rng.normal(size=(T, E)))
    dl = torch.tensor([0.5, 0.25], device="cuda")
    layer = _layer(T, E, k)
    layer.route_losses(z)
    layer.route_backward(z, None, dl)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, _, losses = layer.route_losses(z)
        g = layer.route_backward(z, None, dl)
    z.copy_(_device(rng.normal(size=(T, E))))
    graph.replay()
    torch.cuda.synchronize()
    f = orouter.route_losses(z.cpu().numpy(), k)
    _check_forward(layer, layer.topk_idx, layer.topk_prob, losses, f)
    ref, bar = _grad_bar(f, E, None, [0.5, 0.25], False)
    assert np.all(np.abs(g.cpu().numpy() - ref) <= bar)
    side = torch.cuda.Stream()
    other = _layer(T, E, k)
    with torch.cuda.stream(side):
        _, _, l2 = other.route_losses(z)
    side.synchronize()
    assert torch.equal(l2, losses)
