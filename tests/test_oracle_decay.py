"""The oracle of the decayed attention and of the norms with rotation: closed
forms, and its gradients against central differences of its forward functions."""

import numpy as np
import pytest

import oracle as orc


def _rng(seed):
    return np.random.default_rng(seed)


def _difference(f, x, where, eps=1e-6):
    a, b = x.copy(), x.copy()
    a[where] += eps
    b[where] -= eps
    return (f(a) - f(b)) / (2 * eps)


def test_decay_attention_closed_forms():
    rng = _rng(0)
    B, H, L, d = 2, 3, 9, 4
    q, k, v = (rng.normal(size=(B, H, L, d)) for _ in range(3))
    S0 = rng.normal(size=(B, H, d, d))
    g = np.array([0.0, np.log(0.5), -np.inf])
    o, ST = orc.decay_attention(q, k, v, g, 0.3, S0)
    # head 0: no decay, a prefix sum of outer products on top of the state
    S = S0[:, 0, None] + np.cumsum(k[:, 0, :, :, None] * v[:, 0, :, None, :], 1)
    assert np.allclose(o[:, 0], 0.3 * np.einsum("bli,blij->blj", q[:, 0], S))
    assert np.allclose(ST[:, 0], S[:, -1])
    # head 1: powers of one half
    t = 6
    want = 0.5 ** (t + 1) * np.einsum("bi,bij->bj", q[:, 1, t], S0[:, 1])
    want = want + sum(0.5 ** (t - s) * (q[:, 1, t] * k[:, 1, s]).sum(-1)[:, None] * v[:, 1, s] for s in range(t + 1))
    assert np.allclose(o[:, 1, t], 0.3 * want)
    # head 2: a token sees itself alone
    assert np.allclose(o[:, 2], 0.3 * (q[:, 2] * k[:, 2]).sum(-1, keepdims=True) * v[:, 2])
    # lengths: nothing behind them is used, and a sequence without tokens keeps its state
    for x in (q, k, v):
        x[0, :, 4:] = np.nan
        x[1] = np.nan
    o2, ST2 = orc.decay_attention(q, k, v, g, 0.3, S0, [4, 0])
    assert np.allclose(o2[0, :, :4], o[0, :, :4]) and (o2[0, :, 4:] == 0).all() and (o2[1] == 0).all()
    assert np.array_equal(ST2[1], S0[1])
    assert np.allclose(ST2[0, 0], S[0, 3])


@pytest.mark.parametrize("lengths", [None, [5, 2]])
def test_decay_attention_gradients_against_differences(lengths):
    rng = _rng(1)
    B, H, L, d = 2, 2, 6, 3
    q, k, v, do = (rng.normal(size=(B, H, L, d)) for _ in range(4))
    S0, dST = rng.normal(size=(B, H, d, d)), rng.normal(size=(B, H, d, d))
    g = np.array([-0.1, -1.3])

    def loss(q, k, v, S0):
        o, ST = orc.decay_attention(q, k, v, g, 0.7, S0, lengths)
        return (o * do).sum() + (ST * dST).sum()

    grads = orc.decay_attention_grad(q, k, v, g, do, 0.7, S0, dST, lengths)
    args = [q, k, v, S0]
    for i, got in enumerate(grads):
        for _ in range(12):
            w = tuple(int(rng.integers(n)) for n in got.shape)
            num = _difference(lambda x: loss(*args[:i], x, *args[i + 1:]), args[i], w)
            assert np.isclose(got[w], num, rtol=1e-6, atol=1e-8), (i, w)


def test_decay_attention_bounds_cover_fp32():
    # the recurrence in 32 bits, one rounding an operation, stays inside the bounds
    rng = _rng(2)
    B, H, L, d = 1, 2, 200, 8
    f = np.float32
    q, k, v = (rng.normal(size=(B, H, L, d)).astype(f) for _ in range(3))
    g = np.array([-0.01, -0.7], f)
    o, ST = orc.decay_attention(*(x.astype(np.float64) for x in (q, k, v)), g.astype(np.float64))
    bo, bs = orc.decay_attention_bound(q, k, v, g.astype(np.float64))
    C = 64
    S = np.zeros((B, H, d, d), f)
    for t0 in range(0, L, C):
        n = min(C, L - t0)
        a, b, c = (x[:, :, t0:t0 + n] for x in (q, k, v))
        i = np.arange(n)
        w = np.where(i[:, None] >= i, np.exp(g[:, None, None] * np.maximum(i[:, None] - i, 0).astype(f)), f(0))
        out = np.matmul(np.matmul(a, b.swapaxes(-1, -2)) * w[None], c)
        out = out + np.exp(g[:, None] * (i + 1).astype(f))[None, :, :, None] * np.matmul(a, S)
        assert (np.abs(out - o[:, :, t0:t0 + n]) <= bo[:, :, t0:t0 + n]).all()
        u = np.exp(g[:, None] * (n - 1 - i).astype(f))[None, :, :, None]
        S = np.exp(g * f(n))[None, :, None, None] * S + np.matmul((b * u).swapaxes(-1, -2), c)
    assert (np.abs(S - ST) <= bs).all()
    assert np.median(bo / np.abs(o)) < 1e-3                       # and says something


@pytest.mark.parametrize("halves", [False, True])
def test_qk_norm_rotary_against_parts_and_differences(halves):
    rng = _rng(3)
    B, H, L, d = 2, 2, 3, 10
    x, dy, w = rng.normal(size=(B, H, L, d)), rng.normal(size=(B, H, L, d)), rng.normal(size=d)
    pos = rng.integers(-50, 50, size=(2, 1, L))
    freq, axis = orc.rotary_frequencies((1, 3))
    y = orc.qk_norm_rotary(x, w, 1e-3, pos, freq, axis, halves)
    # with a weight of 1 the rotation leaves the length: mean y^2 = mean x^2 / (mean x^2 + eps)
    m = (x * x).mean(-1)
    y1 = orc.qk_norm_rotary(x, None, 1e-3, pos, freq, axis, halves)
    assert np.allclose((y1 * y1).mean(-1), m / (m + 1e-3))
    assert np.allclose(orc.rotary(y, pos, freq, axis, halves, inverse=True), x / np.sqrt(m + 1e-3)[..., None] * w)

    def loss(x, w):
        return (orc.qk_norm_rotary(x, w, 1e-3, pos, freq, axis, halves) * dy).sum()

    dx, dw = orc.qk_norm_rotary_grad(x, dy, w, 1e-3, pos, freq, axis, halves)
    for _ in range(20):
        i = tuple(int(rng.integers(n)) for n in x.shape)
        assert np.isclose(dx[i], _difference(lambda a: loss(a, w), x, i), rtol=1e-6, atol=1e-8)
    for i in range(d):
        assert np.isclose(dw[i], _difference(lambda a: loss(x, a), w, (i,)), rtol=1e-6, atol=1e-8)
