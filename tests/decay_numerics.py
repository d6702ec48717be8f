"""How far the decayed attention's tensor-core path may be off in the norm, and a
model of its roundings in NumPy that shows what each of them costs.

Element by element bounds (oracle/decay.py) have to cover the worst case of every
sum, thousands of terms whose errors do not add up in earnest; a part of a factor
that went missing would stay inside them.  Norms of all elements see it.

A rounding to bf16 is off by up to half a step, evenly spread: 2^(e-7) / sqrt(12) in the
mean square for values of [2^e, 2^(e+1)).  Over normally distributed values that is R =
0.00166 of their norm, whatever their size.  Independent roundings add up by their squares:
  o, dq, dk, dv   each term rounded once, and the output: sqrt(2) R = 0.00235; a third
                  rounding of the terms across chunks would bring it towards sqrt(3) R = 0.00288
  o of a state    (products of other tokens small beside it) the output alone: R; a
                  state in one bf16 part would make it sqrt(2) R
The limits lie halfway between, in the squares.

States in fp32: a factor that is off by 2 ulp and the rounding of its product, 2^-22 +
2^-24; its argument 3 2^-24 n |g|, n |g| about 1 where terms matter; a chunk's eight sums
of 16 tokens, each cut off by less than 2^-23 of what they have reached, half on average
and half of the final sum on average: 2^-23 8 / 4.  Together 7.2e-7 where all have one
sign (the factor of a segment's border is off the same way, but passed by old, faded
terms alone): 1e-6.  Two bf16 parts of a factor (16 or 17 bits) are more than twice that
off, and so are hundreds of cut sums in one accumulator.
"""

import math

import numpy as np

R = math.sqrt(sum(4.0 ** (e - 7) / 12 * (math.erf(2.0 ** (e + 0.5)) - math.erf(2.0 ** (e - 0.5))) for e in range(-20, 4)))
LIMIT_OUT = math.sqrt(2.5) * R
LIMIT_OUT_OF_STATE = math.sqrt(1.5) * R
LIMIT_STATE = 1e-6

CHUNK = 128
F = np.float32


def bf16(x):
    """x (fp32) to the nearest bf16, ties to even"""
    i = np.ascontiguousarray(x, F).view(np.uint32)
    return ((i + 0x7fff + (i >> 16 & 1)) & np.uint32(0xffff0000)).view(F)


def cut(x):
    """x (fp64) to fp32 towards zero"""
    f = x.astype(F)
    return np.where(np.abs(f.astype(np.float64)) > np.abs(x), np.nextafter(f, F(0)), f)


def powers(g, n):
    """l^n in fp32, one head"""
    return np.exp2((F(g) * F(1.4426950408889634)) * np.asarray(n, F)).astype(F)


def gain(b, c, g, parts=3, whole=False):
    """sum_t l^(n-1-t) b_t c_t^T of one head's n tokens [n, d] by the tensor cores'
    sums: b's faded rows in bf16 parts, a chunk's products in accumulators of their
    own (whole: in the same ones throughout)."""
    n, d = b.shape
    u = powers(g, n - 1 - np.arange(n))[:, None]
    rest, split = (b * u).astype(F), []
    for _ in range(parts):
        split.append(bf16(rest))
        rest = rest - split[-1]
    c = c.astype(np.float64)
    total, acc = np.zeros((d, d), F), [np.zeros((d, d), F) for _ in range(parts)]
    for t0 in range(0, n, CHUNK):
        if not whole:
            acc = [np.zeros((d, d), F) for _ in range(parts)]
        for t in range(t0, min(t0 + CHUNK, n), 16):
            for k in range(parts):
                acc[k] = cut(acc[k] + split[k][t:t + 16].T.astype(np.float64) @ c[t:t + 16])
        if not whole:
            total = total + sum(acc[::-1], np.zeros((d, d), F))
    return sum(acc[::-1], np.zeros((d, d), F)) if whole else total


def outputs(q, k, v, g, S0=None, rest=True, key=True, weight=True):
    """o of one head's tokens [L, d] chunk by chunk as the passes form it: the weights rounded to bf16, the faded keys
    that the state takes in, the state itself in two parts; rest=False: in one; key, weight=False: those kept as they are."""
    L, d = q.shape
    state = np.zeros((d, d)) if S0 is None else S0.astype(np.float64)
    o = np.zeros((L, d))
    for t0 in range(0, L, CHUNK):
        a, b, c = (x[t0:t0 + CHUNK].astype(np.float64) for x in (q, k, v))
        n = len(a)
        i = np.arange(n)
        w = np.where(i[:, None] >= i, (a @ b.T) * powers(g, np.abs(i[:, None] - i)), 0.0)
        m = state.astype(F)
        hi = bf16(m)
        m = hi.astype(np.float64) + (bf16(m - hi) if rest else 0.0)
        o[t0:t0 + n] = (bf16(w.astype(F)) if weight else w) @ c + powers(g, i + 1)[:, None] * (a @ m)
        f = (b * powers(g, n - 1 - i)[:, None]).astype(F)
        state = float(powers(g, n)) * state + (bf16(f) if key else f).astype(np.float64).T @ c
    return bf16(o.astype(F))


def off(got, want):
    """by norm"""
    return float(np.linalg.norm(np.asarray(got, np.float64) - want) / np.linalg.norm(want))
