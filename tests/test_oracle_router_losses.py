"""Pins of the oracle's router losses and gradient: closed forms, the balanced
and the collapsed router, masks, and central differences of a loss that uses
every output."""
import numpy as np
import pytest

from oracle import router as orouter


def test_balanced_and_collapsed():
    # token t prefers expert t mod E by far: every expert gets T / E tokens
    E, T = 4, 32
    z = np.zeros((T, E))
    z[np.arange(T), np.arange(T) % E] = 60.0
    r = orouter.route_losses(z, 1)
    assert r["counts"].tolist() == [8] * 4 and abs(r["losses"][0] - 1.0) < 1e-12
    z[:] = 0.0
    z[:, 2] = 60.0
    r = orouter.route_losses(z, 1)
    assert r["counts"].tolist() == [0, 0, 32, 0] and abs(r["losses"][0] - E) < 1e-12
    assert abs(r["losses"][1] - 3600.0) < 1e-9


def test_uniform_router_closed_form():
    r = orouter.route_losses(np.full((7, 5), 1.5), 2)
    assert np.allclose(r["losses"], [1.0, (1.5 + np.log(5.0)) ** 2])
    assert r["counts"].tolist() == [7, 7, 0, 0, 0]          # ties to the lower id


def test_mask_leaves_what_the_unmasked_tokens_give():
    rng = np.random.default_rng(0)
    z = rng.normal(size=(20, 6))
    mask = rng.random(20) < 0.5
    z2 = z.copy()
    z2[~mask] = np.nan
    r, s = orouter.route_losses(z2, 3, mask), orouter.route_losses(z[mask], 3)
    assert np.array_equal(r["counts"], s["counts"]) and np.allclose(r["losses"], s["losses"], rtol=1e-14)
    d = orouter.route_backward(r, rng.normal(size=(20, 3)), [1.0, 1.0])
    assert np.all(d[~mask] == 0.0) and np.isfinite(d).all()
    e = orouter.route_losses(z, 3, np.zeros(20, bool))
    assert e["losses"].tolist() == [0.0, 0.0] and np.all(orouter.route_backward(e, None, [1.0, 1.0]) == 0.0)


@pytest.mark.parametrize("T,E,k,masked", [(6, 5, 2, False), (5, 4, 4, True), (3, 9, 1, False)])
def test_gradient_against_differences(T, E, k, masked):
    """Central differences of sum(c * prob) + a * balance + b * z with the
    counts held (the selection does not move for steps this small)."""
    rng = np.random.default_rng(T * E + k)
    z = rng.normal(size=(T, E)) * 2
    mask = np.arange(T) % 3 != 1 if masked else None
    c, a, b = rng.normal(size=(T, k)), 0.7, 0.3

    def loss(v):
        r = orouter.route_losses(v, k, mask)
        return float(np.sum(c * r["prob"]) + a * r["losses"][0] + b * r["losses"][1])

    g = orouter.route_backward(orouter.route_losses(z, k, mask), c, [a, b])
    h = 1e-6
    num = np.zeros_like(z)
    for t in range(T):
        for e in range(E):
            zp, zm = z.copy(), z.copy()
            zp[t, e] += h
            zm[t, e] -= h
            num[t, e] = (loss(zp) - loss(zm)) / (2 * h)
    # truncation h^2 |f'''| and rounding 2^-52 |f| / h are both below 1e-8
    assert np.max(np.abs(num - g)) < 1e-7
