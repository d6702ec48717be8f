"""fp64 NumPy oracle of the sequence operators: the gated linear recurrence,
layer norm and rotary positions, forward and backward.

TEST INFRASTRUCTURE ONLY, like the FAVOR+ oracle beside it.  Arrays are
[B, H, L, d].  Every function evaluates its formula token by token or row by
row, with no regrouping.  ``*_bound`` functions give how far an fp32
evaluation in any order of summation may be off (first order): a product or
sum of n terms carries n roundings of 2^-24, an exponential or sine of the
device's library twice 2^-23 (2 ulp).
"""

from __future__ import annotations

import math

import numpy as np

__all__ = ["gated_scan", "gated_scan_grad", "gated_scan_bound", "gated_scan_grad_bound", "layer_norm",
           "layer_norm_grad", "layer_norm_bound", "layer_norm_grad_bound", "rotary", "rotary_bound",
           "rotary_frequencies", "ROUND_F32"]

ROUND_F32 = 2.0 ** -24
ULP2 = 2.0 ** -22                    # two units in the last place, relative
SUM_DEPTH = 96                       # additions that a term of a row's sum passes through, at most


def gated_scan(x, g, h0=None):
    """(h, hT): h_t = exp(g_t) h_{t-1} + x_t; a gate of 0 drops the state."""
    h = np.zeros(x.shape[:2] + x.shape[3:]) if h0 is None else h0.astype(np.float64)
    out = np.empty(x.shape)
    for t in range(x.shape[2]):
        a = np.exp(g[:, :, t])
        h = np.where(a == 0, 0.0, a * np.where(a == 0, 0.0, h)) + x[:, :, t]
        out[:, :, t] = h
    return out, h


def gated_scan_grad(g, h, dh, h0=None, dhT=None):
    """(dx, dg, dh0) of sum(dh h) + sum(dhT hT)."""
    shape = g.shape[:2] + g.shape[3:]
    first = np.zeros(shape) if h0 is None else h0
    c = np.zeros(shape) if dhT is None else dhT.astype(np.float64)
    dx, dg = np.empty(g.shape), np.empty(g.shape)
    for t in reversed(range(g.shape[2])):
        a = np.exp(g[:, :, t])
        before = h[:, :, t - 1] if t > 0 else first
        dx[:, :, t] = dh[:, :, t] + c
        c = np.where(a == 0, 0.0, a * np.where(a == 0, 0.0, dx[:, :, t]))
        dg[:, :, t] = c * np.where(a == 0, 0.0, before)
    return dx, dg, c


def gated_scan_bound(x, g, h0=None):
    """Absolute error bounds of h (every token; the last is hT's)."""
    mag = np.zeros(x.shape[:2] + x.shape[3:]) if h0 is None else np.abs(h0)     # the sum of the terms' sizes
    err = np.zeros_like(mag)
    out = np.empty(x.shape)
    for t in range(x.shape[2]):
        a = np.exp(g[:, :, t])
        err = a * err + (ULP2 + 2 * ROUND_F32) * a * mag
        mag = a * mag + np.abs(x[:, :, t])
        err = err + 2 * ROUND_F32 * mag
        out[:, :, t] = err
    return out


def gated_scan_grad_bound(g, h, dh, h0=None, dhT=None):
    """Absolute error bounds of (dx, dg, dh0)."""
    shape = g.shape[:2] + g.shape[3:]
    first = np.zeros(shape) if h0 is None else np.abs(h0)
    mag = np.zeros(shape) if dhT is None else np.abs(dhT)
    err = np.zeros(shape)
    dx, dg = np.empty(g.shape), np.empty(g.shape)
    for t in reversed(range(g.shape[2])):
        a = np.exp(g[:, :, t])
        before = np.abs(h[:, :, t - 1]) if t > 0 else first
        mag = mag + np.abs(dh[:, :, t])
        err = err + 2 * ROUND_F32 * mag
        dx[:, :, t] = err
        err = a * err + (ULP2 + 2 * ROUND_F32) * a * mag
        mag = a * mag
        dg[:, :, t] = np.where(a == 0, 0.0, err * before + ROUND_F32 * mag * before)
    return dx, dg, err


def _stats(x, eps):
    mu = x.mean(-1, keepdims=True)
    var = ((x - mu) ** 2).mean(-1, keepdims=True)
    return mu, 1.0 / np.sqrt(var + eps)


def layer_norm(x, gamma=None, beta=None, eps=1e-5):
    mu, r = _stats(x, eps)
    return (x - mu) * r * (1.0 if gamma is None else gamma) + (0.0 if beta is None else beta)


def layer_norm_grad(x, dy, gamma=None, eps=1e-5):
    """(dx, dgamma, dbeta) of sum(dy y)."""
    mu, r = _stats(x, eps)
    xh = (x - mu) * r
    n = dy * (1.0 if gamma is None else gamma)
    dx = r * (n - n.mean(-1, keepdims=True) - xh * (n * xh).mean(-1, keepdims=True))
    axes = tuple(range(x.ndim - 1))
    return dx, (dy * xh).sum(axes), dy.sum(axes)


def _normed_bound(x, eps):
    """xh, the relative error of r and the absolute one of xh."""
    u = ROUND_F32
    mu, r = _stats(x, eps)
    off = (SUM_DEPTH + 1) * u * np.abs(x).mean(-1, keepdims=True)             # of the mean
    xh = (x - mu) * r
    rel = 0.5 * ((SUM_DEPTH + 4) * u + (off * r) ** 2) + 4 * u
    return xh, r, rel, r * off + r * u * np.abs(x - mu) + np.abs(xh) * (rel + u)


def layer_norm_bound(x, gamma=None, beta=None, eps=1e-5):
    xh, _, _, e = _normed_bound(x, eps)
    w = np.abs(np.ones(x.shape[-1]) if gamma is None else gamma)
    z = np.abs(np.zeros(x.shape[-1]) if beta is None else beta)
    return e * w + 2 * ROUND_F32 * (np.abs(xh) * w + z)


def layer_norm_grad_bound(x, dy, gamma=None, eps=1e-5):
    """Absolute error bounds of (dx, dgamma, dbeta)."""
    u = ROUND_F32
    xh, r, rel, e = _normed_bound(x, eps)
    n = np.abs(dy * (1.0 if gamma is None else gamma))
    signed = dy * (1.0 if gamma is None else gamma)
    m1, m2 = np.abs(signed.mean(-1, keepdims=True)), np.abs((signed * xh).mean(-1, keepdims=True))
    e1 = (SUM_DEPTH + 2) * u * n.mean(-1, keepdims=True)
    e2 = (SUM_DEPTH + 3) * u * (n * np.abs(xh)).mean(-1, keepdims=True) + (n * e).mean(-1, keepdims=True)
    mag = n + m1 + np.abs(xh) * m2
    dx = r * (e1 + np.abs(xh) * e2 + e * m2 + 5 * u * mag) + r * mag * rel
    axes = tuple(range(x.ndim - 1))
    # additions that a row passes through: those of its thread's rows (with one row to a CTA and 64 CTAs; the
    # kernels run more) and the joins; the exact sums of many rows are tested with whole numbers
    depth = 128 + x[..., 0].size // 64
    dgamma = (depth * u * np.abs(dy * xh) + np.abs(dy) * e).sum(axes)
    return dx, dgamma, depth * u * np.abs(dy).sum(axes)


def rotary_frequencies(sections, base=10000.0):
    """Radians per unit of position of each pair, and each pair's axis."""
    freq = [base ** (-j / n) for n in sections for j in range(n)]
    return np.array(freq), np.array([a for a, n in enumerate(sections) for _ in range(n)], dtype=int)


def rotary(x, pos, freq, axis, halves, inverse=False):
    """x [B, H, L, d] rotated by pos [axes, B or 1, L]."""
    P = len(freq)
    out = x.astype(np.float64).copy()
    for p in range(P):
        t = pos[axis[p]].astype(np.float64) * freq[p]                          # [B or 1, L]
        c, s = np.cos(t)[:, None, :], np.sin(t)[:, None, :] * (-1.0 if inverse else 1.0)
        iu, iv = (p, p + P) if halves else (2 * p, 2 * p + 1)
        u, v = x[..., iu], x[..., iv]
        out[..., iu], out[..., iv] = u * c - v * s, u * s + v * c
    return out


def rotary_bound(x, P, halves):
    """Absolute error bounds: the angle to half a rounding of pi and 2^-31 of a
    turn, sine and cosine to 2 ulp, two products and a sum."""
    e = math.pi * ROUND_F32 + 2 * math.pi * 2.0 ** -31 + ULP2 + 2 * ROUND_F32
    out = np.zeros(x.shape)
    for p in range(P):
        iu, iv = (p, p + P) if halves else (2 * p, 2 * p + 1)
        out[..., iu] = out[..., iv] = e * (np.abs(x[..., iu]) + np.abs(x[..., iv]))
    return out
