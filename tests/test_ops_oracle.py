"""Pins of the float64 oracle of the operators around the layer: closed forms,
equivariance, and gradients against central differences."""

import numpy as np
import pytest

from oracle import feql_ops_oracle as O

EPS = 1e-5


def rng(k):
    return np.random.default_rng(4200 + k)


def central(f, v, k, step=1e-5):
    """d f / d v[k] by central differences (f of the whole array)."""
    p, m = v.copy(), v.copy()
    p[k] += step
    m[k] -= step
    return (f(p) - f(m)) / (2 * step)


def test_norm_has_zero_mean_and_unit_variance():
    x = rng(0).standard_normal((5, 7, 4)) * 3 + 2
    y, mu, r = O.norm_forward(x, None, None, 1e-12)
    assert np.allclose(y.mean(axis=(1, 2)), 0, atol=1e-12)
    assert np.allclose((y * y).mean(axis=(1, 2)), 1, atol=1e-9)
    assert np.allclose(mu, x.reshape(5, -1).mean(1)) and np.allclose(r, 1 / x.reshape(5, -1).std(1))


def test_norm_commutes_with_the_group():
    r = rng(1)
    x, g, b = r.standard_normal((3, 5, 8)), r.standard_normal(5), r.standard_normal(5)
    perm = r.permutation(8)  # any permutation of the group axis, rotations among them
    y = O.norm_forward(x, g, b, EPS)[0]
    assert np.allclose(O.norm_forward(x[:, :, perm], g, b, EPS)[0], y[:, :, perm], atol=1e-12)


def test_norm_gradients_are_the_derivatives():
    r = rng(2)
    x, g, b, dy = (r.standard_normal(s) for s in ((2, 3, 4), 3, 3, (2, 3, 4)))
    dx, dg, db = O.norm_backward(x, dy, g, EPS)
    loss = lambda x_, g_, b_: (dy * O.norm_forward(x_, g_, b_, EPS)[0]).sum()
    for k in np.ndindex(x.shape):
        assert abs(central(lambda v: loss(v, g, b), x, k) - dx[k]) < 1e-7
    for k in range(3):
        assert abs(central(lambda v: loss(x, v, b), g, k) - dg[k]) < 1e-7
        assert abs(central(lambda v: loss(x, g, v), b, k) - db[k]) < 1e-7


@pytest.mark.parametrize("name", ["none", "relu", "gelu", "silu"])
def test_activation_slopes_are_the_derivatives(name):
    z = np.concatenate([np.linspace(-9, 9, 61), [1e-3, -1e-3, 30.0, -30.0]])
    z = z[np.abs(z) > 1e-4]  # not at relu's corner
    d = (O.act(name, z + 1e-5) - O.act(name, z - 1e-5)) / 2e-5
    assert np.allclose(d, O.act_slope(name, z), atol=1e-8)


def test_scan_closed_forms():
    r = rng(3)
    u, h0 = r.standard_normal((6, 2, 4)), r.standard_normal((1, 2, 4))
    off = [0, 6]
    # gates shut: the state passes through; wide open: the input does
    h, hN = O.scan_forward(u, np.full(u.shape, 800.0), h0, off)
    assert np.array_equal(h, np.broadcast_to(h0, h.shape)) and np.array_equal(hN, h0)
    h, hN = O.scan_forward(u, np.full(u.shape, -800.0), h0, off)
    assert np.array_equal(h, u) and np.array_equal(hN[0], u[-1])
    # one gate for all: a geometric average
    a = 1 / (1 + np.exp(-0.7))
    h, _ = O.scan_forward(u, np.full(u.shape, 0.7), h0, off)
    want = a ** 6 * h0[0] + (1 - a) * sum(a ** (5 - l) * u[l] for l in range(6))
    assert np.allclose(h[-1], want, atol=1e-13)


def test_scan_sequences_do_not_meet():
    r = rng(4)
    u, g, h0 = r.standard_normal((9, 2, 3)), r.standard_normal((9, 2)), r.standard_normal((4, 2, 3))
    off = [1, 4, 4, 8, 8]  # a row before, one behind, two empty sequences
    h, hN = O.scan_forward(u, g, h0, off)
    assert np.array_equal(h[0], np.zeros((2, 3))) and np.array_equal(h[8], np.zeros((2, 3)))
    assert np.array_equal(hN[1], h0[1]) and np.array_equal(hN[3], h0[3])
    alone, last = O.scan_forward(u[4:8], g[4:8], h0[2:3], [0, 4])
    assert np.array_equal(h[4:8], alone) and np.array_equal(hN[2], last[0])


@pytest.mark.parametrize("shared", [False, True])
def test_scan_gradients_are_the_derivatives(shared):
    r = rng(5)
    N, C, T = 7, 2, 3
    off = [0, 3, 3, 6]
    u, dh = r.standard_normal((N, C, T)), r.standard_normal((N, C, T))
    g = r.standard_normal((N, C) if shared else (N, C, T))
    h0, dhN = r.standard_normal((3, C, T)), r.standard_normal((3, C, T))

    def loss(u_, g_, h0_):
        h, hN = O.scan_forward(u_, g_, h0_, off)
        return (dh * h).sum() + (dhN * hN).sum()

    du, dg, dh0 = O.scan_backward(dh, u, g, h0, dhN, off)
    for k in np.ndindex(u.shape):
        assert abs(central(lambda v: loss(v, g, h0), u, k) - du[k]) < 1e-8
    for k in np.ndindex(g.shape):
        assert abs(central(lambda v: loss(u, v, h0), g, k) - dg[k]) < 1e-8
    for k in np.ndindex(h0.shape):
        assert abs(central(lambda v: loss(u, g, v), h0, k) - dh0[k]) < 1e-8
