"""Pins of the oracle's MXFP4 codec: the format's values, codes by exhaustive
search over bf16 values, minimal scales, edge blocks, and the expert MLP on it
against a per-token loop."""
import math

import numpy as np
import pytest

from mxfp8_grouped_gemm_x32_b200.workloads import bf16_bits_to_f32
from oracle import mxfp4 as o4


def test_format_values():
    assert o4.MAGNITUDES.tolist() == [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def test_codes_of_ties_and_borders():
    ties = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6}   # to the even code
    for v, c in ties.items():
        assert o4.encode(np.array([v]))[0] == c
        assert o4.encode(np.array([-v]))[0] == (c | 8)
        up, down = np.nextafter(v, 9.0), np.nextafter(v, 0.0)
        lo = int(np.searchsorted(o4.MAGNITUDES, v)) - 1
        assert o4.encode(np.array([down]))[0] == lo and o4.encode(np.array([up]))[0] == lo + 1


def test_scale_is_the_smallest():
    rng = np.random.default_rng(0)
    amax = np.concatenate([np.exp(rng.uniform(-85, 85, 5000)), 6.0 * 2.0 ** np.arange(-120, 120),
                           np.nextafter(6.0 * 2.0 ** np.arange(-120, 120), np.inf)])
    s = o4.scale_bytes(amax).astype(np.int64) - 127
    assert np.all(amax <= 6.0 * 2.0 ** s.astype(np.float64))
    assert np.all((amax > 6.0 * 2.0 ** (s - 1.0)) | (s == -127))
    assert o4.scale_bytes(np.array([0.0, np.nan, np.inf])).tolist() == [0, 255, 255]


def test_round_trip_is_the_nearest():
    """Every finite bf16 value in a block with amax 6 * 2^s: no grid value is nearer."""
    bits = np.arange(0, 1 << 16, dtype=np.uint16)
    v = bf16_bits_to_f32(bits[(bits & 0x7F80) != 0x7F80]).astype(np.float64)
    v = v[np.abs(v) <= 6.0]
    v = v[: v.size // 31 * 31].reshape(-1, 31)
    x = np.concatenate([v, np.full((v.shape[0], 1), 6.0)], axis=1)
    r = o4.roundtrip_rows(x)
    grid = np.concatenate([o4.MAGNITUDES, -o4.MAGNITUDES])
    near = np.abs(x[:, :, None] - grid).min(axis=2)
    assert np.array_equal(np.abs(r - x), near)


def test_nan_and_zero_blocks_and_packing():
    x = np.ones((3, 64))
    x[0, 3], x[1, 40] = np.nan, -np.inf
    x[2, 32:] = 0.0
    r = o4.roundtrip_rows(x)
    assert np.isnan(r[0, :32]).all() and np.isfinite(r[0, 32:]).all()
    assert np.isnan(r[1, 32:]).all() and np.isfinite(r[1, :32]).all()
    assert np.all(r[2, 32:] == 0.0)
    c = np.arange(64, dtype=np.uint8).reshape(2, 32) % 16
    assert np.array_equal(o4.unpack(o4.pack(c)), c)
    assert o4.pack(np.array([[1, 2] * 16], np.uint8))[0, 0] == 0x21


@pytest.mark.parametrize("T,H,I,E,k", [(5, 32, 64, 3, 2), (4, 96, 64, 4, 4)])
def test_forward_is_the_per_token_loop(T, H, I, E, k):
    rng = np.random.default_rng(T)
    x, w1, w2 = rng.normal(size=(T, H)), rng.normal(size=(E, 2 * I, H)), rng.normal(size=(E, H, I))
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    idx[0] = idx[0, 0]                                       # one expert listed k times
    prob = rng.random((T, k))
    got = o4.forward(x, w1, w2, idx, prob)["out"]
    for t in range(T):
        row = np.zeros(H)
        for j in range(k):
            e = idx[t, j]
            a = o4.roundtrip_rows(w1[e]) @ o4.roundtrip_rows(x[t][None])[0]
            h = prob[t, j] * a[:I] / (1.0 + np.exp(-a[:I])) * a[I:]
            row += o4.roundtrip_rows(w2[e]) @ o4.roundtrip_rows(h[None])[0]
        assert np.allclose(got[t], row, rtol=1e-12, atol=1e-12)


def test_error_against_the_unquantised_layer():
    """E2M1's half step is at most 1/4 of the value above the smallest
    magnitudes: the layer stays within a third of the unquantised one."""
    rng = np.random.default_rng(3)
    T, H, I, E, k = 32, 256, 256, 4, 2
    x, w1, w2 = rng.normal(size=(T, H)), rng.normal(size=(E, 2 * I, H)) / 16, rng.normal(size=(E, H, I)) / 16
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    prob = np.full((T, k), 0.5)
    q = o4.forward(x, w1, w2, idx, prob)["out"]
    exact = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            a = w1[idx[t, j]] @ x[t]
            exact[t] += w2[idx[t, j]] @ (prob[t, j] * a[:I] / (1 + np.exp(-a[:I])) * a[I:])
    assert math.sqrt(np.mean((q - exact) ** 2) / np.mean(exact ** 2)) < 0.34
