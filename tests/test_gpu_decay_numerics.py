"""The decayed attention against the fp64 oracle at sizes of many chunks in a
segment and in a CTA's share of the gains, by norms (decay_numerics has the
limits and where they come from).

fp32 calls (CUDA cores) are held to the oracle's first-order bounds, element by
element, as in test_gpu_decay: there a term passes a power of l at each chunk's
border, which may be off by 2 ulp, the same way each time, beside a product's and a
sum's rounding: 23 borders of 1500 tokens in one segment allow 23 (2^-22 + 4 2^-24) =
1.1e-5 of a norm.  (The tensor cores' path takes a token to its segment's end by one
power.)
"""

import pytest
import torch

import oracle as orc
from decay_numerics import CHUNK, LIMIT_OUT, LIMIT_OUT_OF_STATE, LIMIT_STATE, off
from helpers import to_np
from test_gpu_sequence import close

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def gpu_inputs(shape, dtype, seed):
    """q, k, v, do (bf16 values), S0, dST on the GPU"""
    B, H, L, d = shape
    r = torch.Generator("cuda").manual_seed(seed)
    tokens = [torch.randn(shape, generator=r, device="cuda").to(BF16).to(dtype) for _ in range(4)]
    return (*tokens, *(torch.randn((B, H, d, d), generator=r, device="cuda") for _ in range(2)))


def check(cuda_lib, q, k, v, do, g, S0, dST, scale, limit=LIMIT_OUT, lengths=None, sequences=None, heads=None):
    """Both directions; of `sequences` and `heads` (None: all) every state by itself and every chunk of the outputs."""
    pick = torch.tensor(list(range(q.shape[0])) if sequences is None else sequences)
    some = torch.tensor(list(range(q.shape[1])) if heads is None else heads)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    o, ST = cuda_lib.fwd_decay_attention(q, k, v, g, scale, S0, n, dev_status=status)
    grads = cuda_lib.bwd_decay_attention(q, k, v, g, do, scale, S0, dST, n, dev_status=status)
    assert int(status.item()) == 0

    def taken(x):
        return x[pick.cuda()][:, some.cuda()]

    Q, K, V, D, S, E = (to_np(taken(x)) for x in (q, k, v, do, S0, dST))
    G, m = to_np(g)[some], None if lengths is None else [lengths[i] for i in pick]
    got = [taken(x) for x in (o, ST, *grads)]
    want = (*orc.decay_attention(Q, K, V, G, scale, S, m), *orc.decay_attention_grad(Q, K, V, G, D, scale, S, E, m))
    if q.dtype is F32:
        bounds = (*orc.decay_attention_bound(Q, K, V, G, scale, S, m),
                  *orc.decay_attention_grad_bound(Q, K, V, G, D, scale, S, E, m))
        for x, ref, bound in zip(got, want, bounds):
            close(x, ref, bound)
        return
    for name, x, ref in zip(("o", "ST", "dq", "dk", "dv", "dS0"), got, want):
        x = to_np(x)
        for i in range(ref.shape[0]):
            for h in range(ref.shape[1]):
                if name in ("ST", "dS0"):
                    assert off(x[i, h], ref[i, h]) < LIMIT_STATE, (name, i, h, off(x[i, h], ref[i, h]))
                    continue
                end = ref.shape[2] if m is None else m[i]
                assert (x[i, h, end:] == 0).all()
                for t in range(0, end, CHUNK):
                    a, b = x[i, h, t:min(t + CHUNK, end)], ref[i, h, t:min(t + CHUNK, end)]
                    # the few rows of a last chunk by their worst case: two roundings of half a step
                    assert off(a, b) < (limit if len(a) >= 32 else 2 * 2.0 ** -8), (name, i, h, t, off(a, b))


# segments of several chunks (8 and 11; 5 and 10; 12 and 12; 2 and 5), shares of the gains of up to 27 chunks that begin and
# end inside segments, rings that wrap
LONG = [((8, 8, 4096, 64), [0, 7], [0, 1, 7], None), ((2, 16, 4096, 128), [1], [0, 1, 15], None),
        ((30, 10, 1500, 64), [0, 29], [0, 1, 9], None), ((3, 5, 9001, 40), None, None, [9001, 4000, 8960])]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape,sequences,heads,lengths", LONG)
def test_many_chunks(cuda_lib, dtype, shape, sequences, heads, lengths):
    q, k, v, do, S0, dST = gpu_inputs(shape, dtype, sum(shape))
    g = -torch.exp(torch.linspace(-9, -2, shape[1], device="cuda"))     # memories of 7 to 8000 tokens
    check(cuda_lib, q, k, v, do, g, S0, dST, shape[-1] ** -0.5, LIMIT_OUT, lengths, sequences, heads)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(30, 10, 1500, 64), (15, 10, 1500, 128), (8, 8, 4096, 64)])
def test_sums_of_one_sign(cuda_lib, dtype, shape):
    # whatever is cut off adds up
    q, k, v, do, S0, dST = (x.abs() for x in gpu_inputs(shape, dtype, 3))
    g = torch.full((shape[1],), -1e-5, device="cuda")
    check(cuda_lib, q, k, v, do, g, S0, dST, 0.1, sequences=[0, shape[0] - 1], heads=[0, shape[1] - 1])


@pytest.mark.parametrize("shape", [(2, 4, 400, 64), (2, 4, 700, 64), (1, 4, 700, 128), (2, 2, 300, 24)])
def test_states_that_outweigh_the_tokens(cuda_lib, shape):
    # outputs made of the state alone are rounded once
    q, k, v, do, S0, dST = gpu_inputs(shape, BF16, 4)
    g = torch.full((shape[1],), -1e-3, device="cuda")
    check(cuda_lib, q / 1024, k / 1024, v, do, g, S0, dST, 1.0, LIMIT_OUT_OF_STATE)
