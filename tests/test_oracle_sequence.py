"""The sequence operators' oracle: closed forms, and its gradients against
central differences of its forward functions."""

import numpy as np
import pytest

import oracle as orc


def _rng(seed):
    return np.random.default_rng(seed)


def test_gated_scan_closed_forms():
    rng = _rng(0)
    x = rng.normal(size=(2, 3, 9, 4))
    h0 = rng.normal(size=(2, 3, 4))
    # no decay: a prefix sum on top of the state
    h, last = orc.gated_scan(x, np.zeros_like(x), h0)
    assert np.allclose(h, h0[:, :, None] + np.cumsum(x, 2))
    assert np.array_equal(last, h[:, :, -1])
    # a constant decay: powers
    h, _ = orc.gated_scan(x, np.full_like(x, np.log(0.5)), h0)
    t = 6
    want = h0 * 0.5 ** (t + 1) + sum(x[:, :, s] * 0.5 ** (t - s) for s in range(t + 1))
    assert np.allclose(h[:, :, t], want)
    # a closed gate starts over, whatever the state was
    g = np.zeros_like(x)
    g[:, :, 5] = -np.inf
    bad = x.copy()
    bad[:, :, 2] = np.inf
    bad[:, 1, 3] = np.nan
    with np.errstate(invalid="ignore"):
        h, _ = orc.gated_scan(bad, g, h0)
    assert np.allclose(h[:, :, 5:], np.cumsum(x[:, :, 5:], 2))


def _difference(f, x, where, eps=1e-6):
    a, b = x.copy(), x.copy()
    a[where] += eps
    b[where] -= eps
    return (f(a) - f(b)) / (2 * eps)


def test_gated_scan_gradients_against_differences():
    rng = _rng(1)
    B, H, L, d = 2, 2, 7, 3
    x, g, dh = (rng.normal(size=(B, H, L, d)) for _ in range(3))
    g = -np.abs(g)
    h0, dhT = rng.normal(size=(B, H, d)), rng.normal(size=(B, H, d))

    def loss(x, g, h0):
        h, last = orc.gated_scan(x, g, h0)
        return (h * dh).sum() + (last * dhT).sum()

    dx, dg, dh0 = orc.gated_scan_grad(g, orc.gated_scan(x, g, h0)[0], dh, h0, dhT)
    for w in [(0, 0, 0, 0), (1, 1, 3, 2), (0, 1, 6, 1)]:
        assert np.isclose(dx[w], _difference(lambda v: loss(v, g, h0), x, w), rtol=1e-6, atol=1e-8)
        assert np.isclose(dg[w], _difference(lambda v: loss(x, v, h0), g, w), rtol=1e-6, atol=1e-8)
    for w in [(0, 0, 0), (1, 1, 2)]:
        assert np.isclose(dh0[w], _difference(lambda v: loss(x, g, v), h0, w), rtol=1e-6, atol=1e-8)


def test_layer_norm_rows_and_gradients():
    rng = _rng(2)
    x = rng.normal(size=(2, 2, 3, 5)) * 3 + 1
    y = orc.layer_norm(x, eps=1e-12)
    assert np.allclose(y.mean(-1), 0) and np.allclose(y.std(-1), 1)
    assert np.allclose(orc.layer_norm(np.full((1, 1, 1, 4), 7.0)), 0)          # a constant row
    gamma, beta, dy = rng.normal(size=5), rng.normal(size=5), rng.normal(size=x.shape)

    def loss(x, gamma, beta):
        return (orc.layer_norm(x, gamma, beta, 1e-3) * dy).sum()

    dx, dgamma, dbeta = orc.layer_norm_grad(x, dy, gamma, 1e-3)
    for w in [(0, 0, 0, 0), (1, 1, 2, 4), (0, 1, 1, 3)]:
        assert np.isclose(dx[w], _difference(lambda v: loss(v, gamma, beta), x, w), rtol=1e-6, atol=1e-8)
    for w in range(5):
        assert np.isclose(dgamma[w], _difference(lambda v: loss(x, v, beta), gamma, w), rtol=1e-6, atol=1e-8)
        assert np.isclose(dbeta[w], _difference(lambda v: loss(x, gamma, v), beta, w), rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("halves", [False, True])
def test_rotary_is_a_rotation_by_relative_positions(halves):
    rng = _rng(3)
    sections = (2, 1)
    freq, axis = orc.rotary_frequencies(sections)
    assert np.allclose(freq, [1.0, 1e-2, 1.0]) and axis.tolist() == [0, 0, 1]
    x, y = rng.normal(size=(2, 1, 2, 4, 8))
    pos = rng.integers(0, 50, size=(2, 1, 4))
    r = orc.rotary(x, pos, freq, axis, halves)
    assert np.allclose((r ** 2).sum(-1), (x ** 2).sum(-1))
    assert np.array_equal(r[..., 6:], x[..., 6:])                              # channels behind the pairs
    assert np.allclose(orc.rotary(r, pos, freq, axis, halves, inverse=True), x)
    # q.k depends on the difference of the positions alone
    a = (orc.rotary(x, pos, freq, axis, halves) * orc.rotary(y, pos + 9, freq, axis, halves)).sum(-1)
    b = (orc.rotary(x, pos + 31, freq, axis, halves) * orc.rotary(y, pos + 40, freq, axis, halves)).sum(-1)
    assert np.allclose(a, b)
    # one pair by a quarter turn
    z = orc.rotary(np.array([[[[1.0, 2.0]]]]), np.array([[[1]]]), np.array([np.pi / 2]), np.array([0]), halves)
    assert np.allclose(z, [[[[-2.0, 1.0]]]])
