"""The limits of the norm-wise tests on the GPU, on a model of the kernels'
roundings: the model keeps them, and each is left when a part goes missing."""

import numpy as np
import pytest

import oracle as orc
from decay_numerics import LIMIT_OUT, LIMIT_OUT_OF_STATE, LIMIT_STATE, R, bf16, cut, gain, off, outputs


def rows(rng, *shape):
    return bf16(rng.normal(size=shape).astype(np.float32))


def exact(q, k, v, g, S0=None):
    o, s = orc.decay_attention(*(x[None, None].astype(np.float64) for x in (q, k, v)), np.array([float(np.float32(g))]),
                               1.0, None if S0 is None else S0[None, None])
    return o[0, 0], s[0, 0]


def test_roundings():
    x = np.array([1.0, 1.00390625, 1.01171875, -1.005, 3.0e38], np.float32)
    assert bf16(x).tolist()[:3] == [1.0, 1.0, 1.015625]              # ties to even
    rng = np.random.default_rng(0)
    for size in (1.0, 1.3, 1.7):
        y = (rng.normal(size=200000) * size).astype(np.float32)
        assert abs(off(bf16(y), y) / R - 1) < 0.02
    z = np.array([1 + 2.0 ** -24, -1 - 2.0 ** -23 - 2.0 ** -25, 2.0 ** 24 + 1.0])
    assert cut(z).tolist() == [1.0, -1 - 2.0 ** -23, 2.0 ** 24]


@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("g", [-0.05, -0.002])
def test_two_parts_of_a_factor_are_not_enough(d, g):
    rng = np.random.default_rng(d)
    k, v = rows(rng, 1024, d), rows(rng, 1024, d)
    want = exact(k, k, v, g)[1]
    assert off(gain(k, v, g), want) < LIMIT_STATE
    assert off(gain(k, v, g, parts=2), want) > 1.3 * LIMIT_STATE
    assert off(gain(k, v, g, parts=1), want) > 100 * LIMIT_STATE


@pytest.mark.parametrize("d", [16, 64])
def test_one_accumulator_for_many_chunks_cuts_off_too_much(d):
    rng = np.random.default_rng(d)
    k, v = np.abs(rows(rng, 1536, d)), np.abs(rows(rng, 1536, d))
    want = exact(k, k, v, -1e-5)[1]
    assert off(gain(k, v, -1e-5), want) < LIMIT_STATE
    assert off(gain(k, v, -1e-5, whole=True), want) > 1.3 * LIMIT_STATE


@pytest.mark.parametrize("d", [64, 128])
def test_a_third_rounding_of_a_term_is_seen(d):
    rng = np.random.default_rng(d)
    q, k, v = (rows(rng, 2048, d) for _ in range(3))
    want = exact(q, k, v, -1e-4)[0]
    assert off(outputs(q, k, v, -1e-4), want) < LIMIT_OUT
    assert off(outputs(q, k, v, -1e-4, rest=False), want) > LIMIT_OUT
    # a term's one rounding is all that the output has beside its own
    assert off(outputs(q, k, v, -1e-4, key=False, weight=False), want) < LIMIT_OUT_OF_STATE


@pytest.mark.parametrize("d", [64, 128])
def test_a_state_in_one_part_is_seen(d):
    rng = np.random.default_rng(d)
    q, k, v = rows(rng, 512, d), rows(rng, 512, d) / 1024, rows(rng, 512, d)
    S0 = rng.normal(size=(d, d)).astype(np.float32)
    want = exact(q, k, v, -1e-3, S0.astype(np.float64))[0]
    assert off(outputs(q, k, v, -1e-3, S0), want) < LIMIT_OUT_OF_STATE
    assert off(outputs(q, k, v, -1e-3, S0, rest=False), want) > LIMIT_OUT_OF_STATE
