"""fp64 NumPy oracle of the causal linear attention with a decay per head and
of the norms of queries and keys with their rotation, forward and backward.

TEST INFRASTRUCTURE ONLY, like the oracles beside it.  Arrays are
[B, H, L, d], states [B, H, d, d].  Every function evaluates its formula token
by token or row by row.  ``*_bound`` functions give how far an evaluation may
be off (first order, element by element):

fp32 (``u`` = 2^-24): an exponential is off by 2 ulp and its argument n g by
3 u n |g|; a term passes a chunk's border (a product with such a power and an
addition) at most once per 64 tokens and twice more, and at most ``depth``
additions besides (a row's d products, a chunk's tokens, a state's rows).

bf16 tensors may be taken through tensor cores: ``half`` = 2^-8 is the most that
one rounding to bf16 moves a value by.  A score (with its decay) is rounded
once; of the state, which other tokens of the row meet, the factors of its
outer products are rounded once and it itself once, so that a term of o is off
by 2 half of its size.  What is returned in fp32 keeps three bf16 parts of a
factor: half^3.
"""

from __future__ import annotations

import numpy as np

from .sequence import ROUND_F32, SUM_DEPTH, ULP2, rotary, rotary_bound

__all__ = ["decay_attention", "decay_attention_grad", "decay_attention_bound", "decay_attention_grad_bound",
           "qk_norm_rotary", "qk_norm_rotary_grad", "qk_norm_rotary_bound", "qk_norm_rotary_grad_bound", "HALF_BF16"]

HALF_BF16 = 2.0 ** -8
CHUNK = 64                           # the fewest tokens of a whole chunk


def _lengths(lengths, q):
    return np.full(q.shape[0], q.shape[2]) if lengths is None else np.asarray(lengths)


def _walk(b, c, g, first, lengths, reverse=False, late=False):
    """Yields (t, state): the state l state + b_t c_t^T with t taken in, of the
    sequences that have a token t; `late`: the factor comes after the read
    (a gradient's state)."""
    B, H, L, d = b.shape
    s = np.zeros((B, H, d, d)) if first is None else first.astype(np.float64).copy()
    lam = np.exp(g)[None, :, None, None]
    for t in (reversed(range(L)) if reverse else range(L)):
        live = (t < lengths)[:, None, None, None]
        add = b[:, :, t, :, None] * c[:, :, t, None, :]
        if late:
            s = np.where(live, s + add, s)
            yield t, s
            s = np.where(live, lam * s, s)
        else:
            s = np.where(live, lam * s + add, s)
            yield t, s
    yield None, s


def _zero_behind(x, lengths):
    for i, n in enumerate(lengths):
        x[i, :, n:] = 0.0
    return x


def _clean(lengths, *arrays):
    """Copies whose rows behind the sequences' ends are 0: nothing of them is used."""
    return [_zero_behind(a.astype(np.float64).copy(), lengths) for a in arrays]


def decay_attention(q, k, v, g, scale=1.0, S0=None, lengths=None):
    """(o, ST)"""
    n = _lengths(lengths, q)
    q, k, v = _clean(n, q, k, v)
    o = np.zeros(q.shape)
    for t, s in _walk(k, v, g, S0, n):
        if t is None:
            return _zero_behind(o, n), s
        o[:, :, t] = scale * np.einsum("bhi,bhij->bhj", q[:, :, t], s)


def decay_attention_grad(q, k, v, g, do, scale=1.0, S0=None, dST=None, lengths=None):
    """(dq, dk, dv, dS0) of sum(do o) + sum(dST ST)."""
    n = _lengths(lengths, q)
    q, k, v, do = _clean(n, q, k, v, do)
    dq, dk, dv = (np.zeros(q.shape) for _ in range(3))
    for t, s in _walk(k, v, g, S0, n):
        if t is not None:
            dq[:, :, t] = scale * np.einsum("bhij,bhj->bhi", s, do[:, :, t])
    for t, r in _walk(scale * q, do, g, dST, n, reverse=True, late=True):
        if t is None:
            return tuple(_zero_behind(x, n) for x in (dq, dk, dv)) + (r,)
        dk[:, :, t] = np.einsum("bhij,bhj->bhi", r, v[:, :, t])
        dv[:, :, t] = np.einsum("bhij,bhi->bhj", r, k[:, :, t])


def _form_bound(a, b, c, g, scale_u, scale_r, first, lengths, half, reverse=False):
    """Bounds of out_t = scale_r M_t^T a_t and of the last state, where M_t is the
    state of scale_u b c^T (decay.cuh's one form of every pass)."""
    u, d = ROUND_F32, a.shape[-1]
    a, b, c = _clean(lengths, np.abs(a), np.abs(b), np.abs(c))
    b = b * abs(scale_u)
    lam = np.exp(g)
    # per token that passes; where a decay is 0 in fp64 its terms are exact zeros
    rate = np.where(lam == 0, 0.0, (ULP2 + 4 * u) / CHUNK + 3 * u * np.where(lam == 0, 0.0, np.abs(g)))
    base = 2 * (ULP2 + 4 * u) + (2 * d + 2 * CHUNK + 16) * u
    out = np.zeros(a.shape)
    lam, rate = lam[None, :, None, None], rate[None, :, None, None]
    mag = np.zeros(a.shape[:2] + (d, d)) if first is None else np.abs(first).astype(np.float64)
    err = np.zeros_like(mag)
    for t in (reversed(range(a.shape[2])) if reverse else range(a.shape[2])):
        live = (t < lengths)[:, None, None, None]
        add = b[:, :, t, :, None] * c[:, :, t, None, :]
        if reverse:
            mag = np.where(live, mag + add, mag)
        else:
            err = np.where(live, lam * (err + rate * mag), err)
            mag = np.where(live, lam * mag + add, mag)
        out[:, :, t] = abs(scale_r) * np.einsum("bhi,bhij->bhj", a[:, :, t], err + (base + 2 * half) * mag)
        if reverse:
            err = np.where(live, lam * (err + rate * mag), err)
            mag = np.where(live, lam * mag, mag)
    return _zero_behind(out, lengths), err + (base + half ** 3) * mag


def decay_attention_bound(q, k, v, g, scale=1.0, S0=None, lengths=None, half=0.0):
    """Absolute error bounds of (o, ST); half: HALF_BF16 where tensor cores may be used."""
    return _form_bound(q, k, v, g, 1.0, scale, S0, _lengths(lengths, q), half)


def decay_attention_grad_bound(q, k, v, g, do, scale=1.0, S0=None, dST=None, lengths=None, half=0.0):
    """Absolute error bounds of (dq, dk, dv, dS0)."""
    n = _lengths(lengths, q)

    def turned(s):
        return None if s is None else np.swapaxes(s, -1, -2)

    dq, _ = _form_bound(do, v, k, g, 1.0, scale, turned(S0), n, half)
    dk, _ = _form_bound(v, do, q, g, scale, 1.0, turned(dST), n, half, reverse=True)
    dv, ds0 = _form_bound(k, q, do, g, scale, 1.0, dST, n, half, reverse=True)
    return dq, dk, dv, ds0


# ---- norms of queries and keys with their rotation ------------------------------

def _root(x, eps):
    return 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def qk_norm_rotary(x, w, eps, pos, freq, axis, halves):
    return rotary(x * _root(x, eps) * (1.0 if w is None else w), pos, freq, axis, halves)


def qk_norm_rotary_grad(x, dy, w, eps, pos, freq, axis, halves):
    """(dx, dw) of sum(dy y)."""
    w = np.ones(x.shape[-1]) if w is None else w
    r = _root(x, eps)
    z, xh = rotary(dy, pos, freq, axis, halves, inverse=True), x * r
    dx = r * (z * w - xh * (z * w * xh).mean(-1, keepdims=True))
    return dx, (z * xh).sum((0, 1, 2))


ROOT_REL = 0.5 * (SUM_DEPTH + 4) * ROUND_F32 + 4 * ROUND_F32     # of 1 / sqrt(mean x^2 + eps)


def qk_norm_rotary_bound(x, w, eps, pos, freq, axis, halves):
    y = np.abs(x * _root(x, eps) * (1.0 if w is None else w))
    e = ROOT_REL + 3 * ROUND_F32                                   # of the normed row
    both = rotary_bound(y, len(freq), halves)                      # the rotation's own
    out = y * e
    for p in range(len(freq)):
        iu, iv = (p, p + len(freq)) if halves else (2 * p, 2 * p + 1)
        out[..., iu] = out[..., iv] = e * (y[..., iu] + y[..., iv])
    return out + both


def qk_norm_rotary_grad_bound(x, dy, w, eps, pos, freq, axis, halves):
    """Absolute error bounds of (dx, dw)."""
    u = ROUND_F32
    w = np.ones(x.shape[-1]) if w is None else w
    r = _root(x, eps)
    z = rotary(dy, pos, freq, axis, halves, inverse=True)
    ez = rotary_bound(np.abs(dy), len(freq), halves)
    xh = x * r
    zw, ezw = np.abs(z * w), ez * np.abs(w) + u * np.abs(z * w)
    m = np.abs((z * w * xh).mean(-1, keepdims=True))
    em = ((ezw + (SUM_DEPTH + 4) * u * zw) * np.abs(xh)).mean(-1, keepdims=True) + 4 * ROOT_REL * m
    dx = r * (ezw + np.abs(xh) * em + (2 * ROOT_REL + 6 * u) * (zw + np.abs(xh) * m))
    # additions that a row passes through: those of its thread's rows and the joins
    depth = 128 + x[..., 0].size // 16
    dw = ((ez + (ROOT_REL + 3 * u + depth * u) * np.abs(z)) * np.abs(xh)).sum((0, 1, 2))
    return dx, dw
