"""GPU parity of the causal linear attention with a decay per head against the
fp64 oracle, element by element.

Tolerance of each element: the oracle's first-order bound (``*_bound``; with
the roundings to bf16 where bf16 tensors may go through tensor cores) plus half
a step of the storage type.
"""

import concurrent.futures

import numpy as np
import pytest
import torch

import oracle as orc
from helpers import to_np
from test_gpu_sequence import LAYOUTS, close, gen, view

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF, NAN = float("inf"), float("nan")


def half(dtype):
    return orc.HALF_BF16 if dtype is BF16 else 0.0


def inputs(shape, dtype, seed, g=None):
    """q, k, v, do, g, S0, dST on the CPU"""
    B, H, L, d = shape
    r = gen(seed)
    q, k, v, do = (torch.randn(shape, generator=r).to(dtype) for _ in range(4))
    S0, dST = (torch.randn((B, H, d, d), generator=r) for _ in range(2))
    if g is None:
        g = -torch.exp(torch.rand(H, generator=r) * 7 - 7)         # memories of one token to a thousand
    return q, k, v, do, torch.as_tensor(g, dtype=F32), S0, dST


def check(lib, case, got, want, bounds, names, status=None):
    if status is not None:
        assert int(status.item()) == 0
    for name, a, ref, b in zip(names, got, want, bounds):
        close(a, ref, b, (case, name))


def both(lib, t, scale, lengths=None, states=True, layout="plain", **out):
    """fwd and bwd of the CPU tensors t against the oracle; returns the outputs."""
    q, k, v, do, g, S0, dST = t
    hf = half(q.dtype)
    Q, K, V, D, G, S, E = (to_np(x) for x in t)
    if not states:
        S = E = S0 = dST = None
    on = [view(x, layout) for x in (q, k, v, do)]
    dev = [None if x is None else x.cuda() for x in (g, S0, dST)]
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fwd = lib.fwd_decay_attention(*on[:3], dev[0], scale=scale, S0=dev[1], lengths=n, dev_status=status)
    args = (Q, K, V, G)
    check(lib, "fwd", fwd, orc.decay_attention(*args, scale, S, lengths),
          orc.decay_attention_bound(*args, scale, S, lengths, hf), ("o", "ST"), status)
    bwd = lib.bwd_decay_attention(*on[:3], dev[0], on[3], scale=scale, S0=dev[1], dST=dev[2], lengths=n,
                                  dev_status=status)
    check(lib, "bwd", bwd, orc.decay_attention_grad(*args, D, scale, S, E, lengths),
          orc.decay_attention_grad_bound(*args, D, scale, S, E, lengths, hf), ("dq", "dk", "dv", "dS0"), status)
    return fwd, bwd


SHAPES = [(1, 1, 1, 1), (2, 3, 2, 5), (1, 2, 63, 16), (1, 1, 64, 64), (2, 1, 65, 64), (1, 2, 127, 128), (1, 1, 128, 64),
          (2, 2, 129, 40), (1, 3, 200, 33), (1, 2, 257, 96), (3, 1, 400, 128), (2, 5, 333, 64), (1, 2, 640, 80),
          (1, 1, 1100, 32), (1, 40, 70, 8), (20, 10, 130, 64), (1, 1, 900, 128)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_matches_oracle(cuda_lib, dtype, shape):
    both(cuda_lib, inputs(shape, dtype, sum(shape)), shape[-1] ** -0.5, states=shape[0] != 3)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape,lengths", [((4, 2, 300, 64), [300, 0, 129, 1]), ((3, 1, 200, 24), [128, 64, 199]),
                                           ((2, 2, 520, 128), [511, 7]), ((2, 1, 130, 64), [0, 0]),
                                           ((3, 2, 65, 33), [-5, 70, 64]), ((2, 1, 2600, 64), [2593, 3]),
                                           ((3, 1, 1500, 128), [0, 1500, 700])])
def test_lengths_and_what_lies_behind_them(cuda_lib, dtype, shape, lengths):
    t = inputs(shape, dtype, 11)
    for b, n in enumerate(lengths):
        for x in t[:4]:
            x[b, :, max(0, n):] = NAN if b % 2 else INF
    clipped = [min(max(n, 0), shape[2]) for n in lengths]
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    fwd, bwd = both(cuda_lib, t, 0.2, clipped)
    on = [x.cuda() for x in t]
    again = cuda_lib.fwd_decay_attention(*on[:3], on[4], 0.2, on[5], n)
    assert all(torch.equal(a, b) for a, b in zip(again, fwd))
    for b, m in enumerate(clipped):
        for x in (fwd[0], *bwd[:3]):
            assert (x[b, :, m:] == 0).all()
        if m == 0:
            assert torch.equal(fwd[1][b], on[5][b]) and torch.equal(bwd[3][b], on[6][b])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128, 24])
def test_decays_of_every_size(cuda_lib, dtype, d):
    # none, slow, one half a token, strong, and a memory of nothing
    g = [0.0, -1e-4, -0.6931, -20.0, -INF, -1e30]
    both(cuda_lib, inputs((1, 6, 270, d), dtype, 3, g), 0.1)
    both(cuda_lib, inputs((1, 6, 1400, d), dtype, 4, g), 0.1)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("shape", [(2, 3, 77, 24), (1, 4, 300, 64), (2, 2, 1, 8), (1, 2, 140, 128), (2, 2, 150, 72)])
def test_layouts(cuda_lib, dtype, layout, shape):
    t = inputs(shape, dtype, 7)
    fwd, bwd = both(cuda_lib, t, 0.3, layout=layout)
    assert fwd[0].is_contiguous()
    q, k, v, do = (view(x, layout) for x in t[:4])
    g, S0, dST = (x.cuda() for x in t[4:])
    outs = [view(torch.zeros_like(t[0]), layout) for _ in range(4)]
    o, _ = cuda_lib.fwd_decay_attention(q, k, v, g, 0.3, S0, O=outs[0])
    got = cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.3, S0, dST, dQ=outs[1], dK=outs[2], dV=outs[3])
    assert o is outs[0]
    for a, b in zip((o, *got), (fwd[0], *bwd)):
        assert torch.equal(a, b)
    if layout in ("joint", "even", "odd"):
        for x in (*outs, q, k, v, do):
            assert int(torch.isnan(x._base).sum()) == x._base.numel() - x.numel()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_broadcast_heads(cuda_lib, dtype):
    # one head of keys and values for all query heads: a stride of 0
    t = inputs((2, 4, 150, 64), dtype, 5)
    q, do, g, S0 = (t[i].cuda() for i in (0, 3, 4, 5))
    k1, v1 = t[1][:, :1].cuda(), t[2][:, :1].cuda()
    kb, vb = k1.expand(-1, 4, -1, -1), v1.expand(-1, 4, -1, -1)
    a = cuda_lib.fwd_decay_attention(q, kb, vb, g, 0.2, S0)
    b = cuda_lib.fwd_decay_attention(q, kb.contiguous(), vb.contiguous(), g, 0.2, S0)
    Q, K, V, G, S, D = (to_np(x) for x in (q, kb, vb, g, S0, do))
    for got in (a, b):
        check(cuda_lib, "broadcast", got, orc.decay_attention(Q, K, V, G, 0.2, S),
              orc.decay_attention_bound(Q, K, V, G, 0.2, S, None, half(dtype)), ("o", "ST"))
    got = cuda_lib.bwd_decay_attention(q, kb, vb, g, do, 0.2, S0)
    check(cuda_lib, "broadcast", got, orc.decay_attention_grad(Q, K, V, G, D, 0.2, S),
          orc.decay_attention_grad_bound(Q, K, V, G, D, 0.2, S, None, None, half(dtype)), ("dq", "dk", "dv", "dS0"))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(2, 3, 5, 64), (3, 2, 4, 128), (1, 1, 3, 1), (2, 2, 3, 33), (300, 8, 1, 64), (1, 2, 2, 100)])
def test_steps_continue_a_sequence(cuda_lib, dtype, shape):
    B, H, L, d = shape
    t = inputs(shape, dtype, 21)
    q, k, v = (x.cuda() for x in t[:3])
    g, state = t[4].cuda(), t[5].cuda()
    Q, K, V, G, S = (to_np(t[i]) for i in (0, 1, 2, 4, 5))
    want, last = orc.decay_attention(Q, K, V, G, 0.4, S)
    bo, bs = orc.decay_attention_bound(Q, K, V, G, 0.4, S)
    kept = state.clone()
    for i in range(L):
        # views of the token inside the sequences; every other step to a new state
        o, new = cuda_lib.decay_attention_step(q[:, :, i], k[:, :, i], v[:, :, i], g, state, 0.4,
                                               new_state=torch.empty_like(state) if i % 2 == 0 else None)
        assert (new is state) == (i % 2 == 1)
        close(o, want[:, :, i], bo[:, :, i], i)
        state = new
    close(state, last, bs, "state")
    assert torch.equal(kept, t[5].cuda())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128, 48])
def test_a_prompt_in_pieces_and_then_tokens(cuda_lib, dtype, d):
    shape = (2, 3, 400, d)
    t = inputs(shape, dtype, 31)
    q, k, v = (x.cuda() for x in t[:3])
    g = t[4].cuda()
    Q, K, V, G = (to_np(t[i]) for i in (0, 1, 2, 4))
    want, last = orc.decay_attention(Q, K, V, G, 0.2)
    bo, bs = orc.decay_attention_bound(Q, K, V, G, 0.2, half=half(dtype))
    state = cuda_lib.new_decay_state(2, 3, d)
    for a, b in ((0, 150), (150, 151), (151, 395)):
        o, out = cuda_lib.fwd_decay_attention(q[:, :, a:b], k[:, :, a:b], v[:, :, a:b], g, 0.2, state, ST=state)
        assert out is state
        close(o, want[:, :, a:b], bo[:, :, a:b], (a, b))
    for i in range(395, 400):
        o, _ = cuda_lib.decay_attention_step(q[:, :, i], k[:, :, i], v[:, :, i], g, state, 0.2)
        close(o, want[:, :, i], bo[:, :, i], i)
    close(state, last, bs, "state")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128, 24])
def test_infinities_and_nan_reach_no_earlier_row(cuda_lib, dtype, d):
    t = inputs((1, 4, 300, d), dtype, 41)
    q, k, v, do = (x.cuda() for x in t[:4])
    g, S0, dST = (x.cuda() for x in t[4:])
    clean = cuda_lib.fwd_decay_attention(q, k, v, g, 0.2, S0)[0]
    grads = cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.2, S0, dST)
    at = 170
    for i, value in ((0, NAN), (1, INF), (2, NAN), (2, INF)):
        ins = [q.clone(), k.clone(), v.clone()]
        ins[i][0, 1, at, d // 2] = value
        o = cuda_lib.fwd_decay_attention(*ins, g, 0.2, S0)[0]
        assert torch.equal(o[:, :, :at], clean[:, :, :at])            # no earlier row
        assert torch.equal(o[:, [0, 2, 3]], clean[:, [0, 2, 3]])      # no other head
        assert not torch.isfinite(o[0, 1, at]).all()
        if i == 0:
            assert torch.equal(o[0, 1, at + 1:], clean[0, 1, at + 1:])
        dq, dk, dv, _ = cuda_lib.bwd_decay_attention(*ins, g, do, 0.2, S0, dST)
        assert torch.equal(dq[0, 1, :at], grads[0][0, 1, :at])        # dq sees earlier tokens
        if i == 0:                                                     # dk and dv see later queries
            assert torch.equal(dk[0, 1, at + 1:], grads[1][0, 1, at + 1:])
            assert torch.equal(dv[0, 1, at + 1:], grads[2][0, 1, at + 1:])
    bad = do.clone()
    bad[0, 2, at, 0] = NAN
    dq, dk, dv, _ = cuda_lib.bwd_decay_attention(q, k, v, g, bad, 0.2, S0, dST)
    for a, b in zip((dk, dv), grads[1:3]):
        assert torch.equal(a[0, 2, at + 1:], b[0, 2, at + 1:]) and torch.equal(a[:, [0, 1, 3]], b[:, [0, 1, 3]])
    keep = [i for i in range(300) if i != at]
    assert torch.equal(dq[0, 2, keep], grads[0][0, 2, keep])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [1, 4, 16, 31, 32, 40, 44, 64, 65, 72, 96, 100, 127, 128])
def test_few_tokens(cuda_lib, dtype, d):
    # fp32 arithmetic, whatever the tensors' type; neighbours of the states stay as they are
    for L in (1, 3, 4, 5, 16, 17):
        B, H = 3, 2
        t = inputs((B, H, L, d), dtype, 300 + L)
        n = [L, 0, L // 2]
        for b in range(B):
            for x in t[:3]:
                x[b, :, n[b]:] = NAN
        args = [to_np(x) for x in (t[0], t[1], t[2], t[4])]
        want, last = orc.decay_attention(*args, 0.3, to_np(t[5]), n)
        bo, bs = orc.decay_attention_bound(*args, 0.3, to_np(t[5]), n, half(dtype) if L > 16 else 0.0)
        lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
        for layout in LAYOUTS:
            for off in (0, 1):
                buf = torch.full((B * H * d * d + 2,), NAN, device="cuda")
                state = buf[off:off + B * H * d * d].view(B, H, d, d)
                state.copy_(t[5])
                o, ST = cuda_lib.fwd_decay_attention(*(view(x, layout) for x in t[:3]), t[4].cuda(), 0.3, state, lengths,
                                                     O=view(torch.zeros_like(t[0]), layout), ST=state)
                assert ST is state
                close(o, want, bo, (L, layout, off, "o"))
                close(ST, last, bs, (L, layout, off, "ST"))
                assert torch.equal(ST[1], t[5][1].cuda()) and int(torch.isnan(buf).sum()) == 2
                assert all((o[b, :, n[b]:] == 0).all() for b in range(B))
        none = cuda_lib.fwd_decay_attention(*(x.cuda() for x in t[:3]), t[4].cuda(), 0.3, None, lengths)
        zero = cuda_lib.fwd_decay_attention(*(x.cuda() for x in t[:3]), t[4].cuda(), 0.3, torch.zeros_like(ST), lengths)
        assert all(torch.equal(a, b) for a, b in zip(none, zero))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [33, 64])
def test_few_tokens_with_infinities(cuda_lib, dtype, d):
    t = inputs((1, 3, 12, d), dtype, 91)
    q, k, v = (x.cuda() for x in t[:3])
    g, S0 = t[4].cuda(), t[5].cuda()
    clean, last = cuda_lib.fwd_decay_attention(q, k, v, g, 0.2, S0)
    for i, value in ((0, NAN), (1, INF), (2, NAN), (2, -INF)):
        ins = [q.clone(), k.clone(), v.clone()]
        ins[i][0, 1, 7, d // 2] = value
        o, ST = cuda_lib.fwd_decay_attention(*ins, g, 0.2, S0)
        assert torch.equal(o[:, :, :7], clean[:, :, :7]) and torch.equal(o[:, ::2], clean[:, ::2])
        assert torch.equal(ST[:, ::2], last[:, ::2]) and not torch.isfinite(o[0, 1, 7]).all()
        if i == 0:
            assert torch.equal(o[0, 1, 8:], clean[0, 1, 8:]) and torch.equal(ST, last)
        elif i == 2:                                                   # only its column
            keep = [j for j in range(d) if j != d // 2]
            assert torch.equal(o[..., keep], clean[..., keep]) and torch.equal(ST[..., keep], last[..., keep])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(2, 2, 50, 64), (2, 2, 200, 64), (1, 2, 2500, 64), (1, 1, 2100, 128), (2, 2, 300, 128),
                                   (1, 3, 900, 24)])
def test_states_in_place(cuda_lib, dtype, shape):
    t = inputs(shape, dtype, 45)
    q, k, v, do, g, S0, dST = (x.cuda() for x in t)
    for lengths in (None, torch.tensor([shape[2] - 30, 0][:shape[0]], dtype=torch.int32, device="cuda")):
        o, ST = cuda_lib.fwd_decay_attention(q, k, v, g, 0.2, S0, lengths)
        grads = cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.2, S0, dST, lengths)
        state, grad = S0.clone(), dST.clone()
        got = (*cuda_lib.fwd_decay_attention(q, k, v, g, 0.2, state, lengths, ST=state),
               *cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.2, S0, grad, lengths, dS0=grad))
        assert got[1] is state and got[5] is grad
        assert all(torch.equal(a, b) for a, b in zip(got, (o, ST, *grads)))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 2, 200, 64), (1, 2, 1500, 64), (1, 1, 700, 128)])
def test_states_off_16_bytes(cuda_lib, dtype, shape):
    B, H, L, d = shape
    t = inputs(shape, dtype, 47)
    q, k, v, do, g = (x.cuda() for x in t[:5])
    n = B * H * d * d
    buf = torch.full((4, n + 4), NAN, device="cuda")
    S0, dST, ST, dS0 = (buf[i, 1 + i % 3:][:n].view(B, H, d, d) for i in range(4))
    S0.copy_(t[5])
    dST.copy_(t[6])
    args = [to_np(x) for x in (t[0], t[1], t[2], t[4])]
    D, S, E = (to_np(t[i]) for i in (3, 5, 6))
    for first, grad in ((S0, dST), (t[5].cuda(), t[6].cuda())):
        fwd = cuda_lib.fwd_decay_attention(q, k, v, g, 0.2, first, ST=ST)
        check(cuda_lib, "fwd", fwd, orc.decay_attention(*args, 0.2, S),
              orc.decay_attention_bound(*args, 0.2, S, None, half(dtype)), ("o", "ST"))
        bwd = cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.2, first, grad, dS0=dS0)
        check(cuda_lib, "bwd", bwd, orc.decay_attention_grad(*args, D, 0.2, S, E),
              orc.decay_attention_grad_bound(*args, D, 0.2, S, E, None, half(dtype)), ("dq", "dk", "dv", "dS0"))
    assert int(torch.isnan(buf).sum()) == 4 * 4                     # nothing beside them is written


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L", [2, 17])
def test_states_beyond_32_bits(cuda_lib, dtype, L):
    # 131080 heads of 128 x 128: the last ones' states lie behind 2^31 elements
    B, H, d = 16385, 8, 128
    r = torch.Generator("cuda").manual_seed(9)
    q, k, v, do = (torch.randn((B, H, L, d), generator=r, device="cuda").to(dtype) for _ in range(4))
    g = torch.linspace(-0.5, -0.01, H, device="cuda")
    S0 = torch.empty((B, H, d, d), device="cuda")
    S0.normal_(generator=r)
    last = slice(B - 2, B)
    small = [x[last].clone() for x in (q, k, v, do, S0)]
    want = cuda_lib.fwd_decay_attention(*small[:3], g, 0.1, small[4])
    o, ST = cuda_lib.fwd_decay_attention(q, k, v, g, 0.1, S0)
    assert torch.equal(o[last], want[0]) and torch.equal(ST[last], want[1])
    step = cuda_lib.decay_attention_step(q[last, :, 0], k[last, :, 0], v[last, :, 0], g, want[1], 0.1)
    ot, _ = cuda_lib.decay_attention_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], g, ST, 0.1)
    assert torch.equal(ot[last], step[0]) and torch.equal(ST[last], step[1])
    want = cuda_lib.bwd_decay_attention(*small[:3], g, small[3], 0.1, small[4], small[4])
    got = cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.1, S0, S0, dS0=ST)
    assert all(torch.equal(a[last], b) for a, b in zip(got, want))


def test_short_sequences_in_graphs_and_on_streams(cuda_lib):
    # the states that run beside the passes: what follows waits for both
    t = inputs((4, 8, 333, 64), BF16, 73)
    q, k, v, do, g, S0, dST = (x.cuda() for x in t)
    want = (*cuda_lib.fwd_decay_attention(q, k, v, g, 0.1, S0),
            *cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.1, S0, dST))
    two = cuda_lib.fwd_decay_attention(q, k, v, g, 0.1, want[1])
    outs, state = [torch.empty_like(x) for x in want], torch.empty_like(S0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        state.copy_(S0)
        cuda_lib.fwd_decay_attention(q, k, v, g, 0.1, state, O=outs[0], ST=state)
        outs[1].copy_(state)
        o2, _ = cuda_lib.fwd_decay_attention(q, k, v, g, 0.1, state, ST=state)
        cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.1, S0, dST, dQ=outs[2], dK=outs[3], dV=outs[4], dS0=outs[5])
    for _ in range(20):
        for x in outs:
            x.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*outs, o2, state), (*want, *two)))
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for stream in streams:
        stream.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for stream in streams:
            got.append((stream, *cuda_lib.fwd_decay_attention(q, k, v, g, 0.1, S0, stream=stream),
                        *cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.1, S0, dST, stream=stream)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for _, *x in got for a, b in zip(x, want))


def test_gradients_against_differences(cuda_lib):
    # of the kernels' own forward, in directions
    t = inputs((2, 2, 150, 32), F32, 51, [-0.02, -0.3])
    q, k, v, do, g, S0, dST = (x.cuda() for x in t)
    lengths = torch.tensor([150, 97], dtype=torch.int32, device="cuda")

    def loss(q, k, v, S0):
        o, ST = cuda_lib.fwd_decay_attention(q, k, v, g, 0.2, S0, lengths)
        return float((o.double() * do.double()).sum() + (ST.double() * dST.double()).sum())

    args = [q, k, v, S0]
    grads = cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.2, S0, dST, lengths)
    r = torch.Generator("cuda").manual_seed(1)
    for i, got in enumerate(grads):
        way = torch.randn(got.shape, generator=r, device="cuda")
        eps = 1e-2                     # the loss is linear in each input by itself: no curvature
        up, down = (loss(*args[:i], args[i] + s * eps * way, *args[i + 1:]) for s in (1, -1))
        want = float((got.double() * way.double()).sum())
        # the outputs' fp32 roundings over the step
        o, ST = cuda_lib.fwd_decay_attention(*args[:3], g, 0.2, S0, lengths)
        noise = 400 * 2.0 ** -24 * float((o.abs() * do.abs()).sum() + (ST.abs() * dST.abs()).sum()) / eps
        assert abs((up - down) / (2 * eps) - want) < noise, i


def test_same_results_every_time_and_on_any_workspace(cuda_lib):
    t = inputs((1, 2, 3000, 64), BF16, 61)
    q, k, v, do, g, S0, dST = (x.cuda() for x in t)
    n = [cuda_lib.decay_attention_workspace_bytes(1, 2, 3000, 64, BF16, back) for back in (False, True)]
    first = None
    for fill in (0, 255, 127):
        ws = [torch.full((m + 256,), fill, dtype=torch.uint8, device="cuda") for m in n]
        got = (*cuda_lib.fwd_decay_attention(q, k, v, g, 0.1, S0, workspace=ws[0][:n[0]]),
               *cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.1, S0, dST, workspace=ws[1][:n[1]]))
        if first is None:
            first = got
        assert all(torch.equal(a, b) for a, b in zip(got, first))
        for w, m in zip(ws, n):
            assert (w[m:] == fill).all()
    with pytest.raises(cuda_lib.FavorError):
        cuda_lib.fwd_decay_attention(q, k, v, g, 0.1, S0, workspace=torch.empty(n[0] - 1, dtype=torch.uint8, device="cuda"))


def test_graphs_streams_and_threads(cuda_lib):
    t = inputs((2, 2, 700, 64), BF16, 71)
    q, k, v, do, g, S0, dST = (x.cuda() for x in t)
    want = (*cuda_lib.fwd_decay_attention(q, k, v, g, 0.1, S0),
            *cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.1, S0, dST))
    # two graphs that share a workspace, replayed in order
    ws = torch.empty(cuda_lib.decay_attention_workspace_bytes(2, 2, 700, 64, BF16, True), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(x) for x in want]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        cuda_lib.fwd_decay_attention(q, k, v, g, 0.1, S0, O=outs[0], ST=outs[1], workspace=ws)
    with torch.cuda.graph(graphs[1]):
        cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.1, S0, dST, dQ=outs[2], dK=outs[3], dV=outs[4], dS0=outs[5],
                                     workspace=ws)
    for _ in range(3):
        for x in outs:
            x.fill_(NAN)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (*cuda_lib.fwd_decay_attention(q, k, v, g, 0.1, S0, stream=side),
           *cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.1, S0, dST, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    def work(_):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                o = cuda_lib.fwd_decay_attention(q, k, v, g, 0.1, S0)
                d = cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.1, S0, dST)
            torch.cuda.current_stream().synchronize()
            return all(torch.equal(a, b) for a, b in zip((*o, *d), want))

    torch.cuda.synchronize()
    with concurrent.futures.ThreadPoolExecutor(2) as pool:
        assert all(pool.map(work, range(2)))


@pytest.mark.parametrize("shape", [(8, 8, 4096, 64), (2, 8, 6144, 128), (1, 1, 30000, 64)])
def test_many_calls_end_in_time(cuda_lib, shape):
    # one by one on an idle GPU, and one behind the other: no wait runs out, and the results are the first call's
    B, H, L, d = shape
    r = torch.Generator("cuda").manual_seed(5)
    q, k, v, do = (torch.randn(shape, generator=r, device="cuda").to(BF16) for _ in range(4))
    g = -torch.exp(torch.rand(H, generator=r, device="cuda") * 7 - 7)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        return (*cuda_lib.fwd_decay_attention(q, k, v, g, 0.1, dev_status=status),
                *cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.1, dev_status=status))

    first = call()
    for n in range(60):
        got = call()
        if n % 2 == 0:
            torch.cuda.synchronize()
            assert int(status.item()) == 0
        assert all(torch.equal(a, b) for a, b in zip(got, first))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_offsets_beyond_32_bits(cuda_lib, dtype):
    # tokens 2^26 elements apart: the last ones lie behind 2^31 elements
    L, d, far = 40, 64, 1 << 26
    t = inputs((1, 2, L, d), dtype, 81)
    buf = torch.empty(far * L, dtype=dtype, device="cuda")
    views = []
    for i, x in enumerate(t[:4]):
        v = buf.as_strided((1, 2, L, d), (0, d, far, 1), i * 4 * d)
        v.copy_(x)
        views.append(v)
    out = buf.as_strided((1, 2, L, d), (0, d, far, 1), 20 * d)
    q, k, v, do = (x.cuda() for x in t[:4])
    g, S0, dST = (x.cuda() for x in t[4:])
    o, ST = cuda_lib.fwd_decay_attention(*views[:3], g, 0.2, S0, O=out)
    want = cuda_lib.fwd_decay_attention(q, k, v, g, 0.2, S0)
    assert torch.equal(o, want[0]) and torch.equal(ST, want[1])
    got = cuda_lib.bwd_decay_attention(*views[:3], g, views[3], 0.2, S0, dST, dQ=out)
    for a, b in zip(got, cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.2, S0, dST)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_layer_of_them(cuda_lib, dtype):
    # a joint projection's output -> norms and positions of q and k -> decayed attention -> layer norm of its heads,
    # forward, backward and token by token
    B, H, L, d = 2, 3, 200, 64
    r = gen(91)
    joint = torch.randn((B, L, 3, H, d), generator=r).to(dtype).cuda()
    q, k, v = (joint[:, :, i].transpose(1, 2) for i in range(3))
    wq, wk = (1 + 0.2 * torch.randn(d, generator=r)).cuda(), (1 + 0.2 * torch.randn(d, generator=r)).cuda()
    g = torch.tensor([-0.01, -0.1, -0.5], device="cuda")
    dy = torch.randn((B, H, L, d), generator=r).to(dtype).cuda()
    sections = (d // 2,)
    table = cuda_lib.new_rotary_table(sections)
    pos = torch.arange(L, dtype=torch.int32, device="cuda").view(1, 1, L)
    turn = (pos, table, sections, "halves")
    qn, kn = cuda_lib.fwd_qk_norm_rotary(q, k, wq, wk, *turn)
    o, ST = cuda_lib.fwd_decay_attention(qn, kn, v, g, d ** -0.5)
    y = cuda_lib.fwd_layer_norm(o)
    do, _, _ = cuda_lib.bwd_layer_norm(o, dy, weight_grads=False)
    dqn, dkn, dv, _ = cuda_lib.bwd_decay_attention(qn, kn, v, g, do, d ** -0.5)
    dq, dk, dwq, dwk = cuda_lib.bwd_qk_norm_rotary(q, k, dqn, dkn, wq, wk, *turn)
    # every stage against the oracle on what the stage before has given
    freq, axis = orc.rotary_frequencies(sections)
    P = pos.cpu().numpy()
    ang = (P, freq, axis, True)
    for x, w, out, grad, dx, dw in ((q, wq, qn, dqn, dq, dwq), (k, wk, kn, dkn, dk, dwk)):
        X, W, D = to_np(x), to_np(w), to_np(grad)
        close(out, orc.qk_norm_rotary(X, W, 1e-5, *ang), orc.qk_norm_rotary_bound(X, W, 1e-5, *ang))
        for a, ref, b in zip((dx, dw), orc.qk_norm_rotary_grad(X, D, W, 1e-5, *ang),
                             orc.qk_norm_rotary_grad_bound(X, D, W, 1e-5, *ang)):
            close(a, ref, b)
    args = tuple(to_np(x) for x in (qn, kn, v, g))
    for a, ref, b in zip((o, ST), orc.decay_attention(*args, d ** -0.5),
                         orc.decay_attention_bound(*args, d ** -0.5, half=half(dtype))):
        close(a, ref, b)
    for a, ref, b in zip((dqn, dkn, dv), orc.decay_attention_grad(*args, to_np(do), d ** -0.5),
                         orc.decay_attention_grad_bound(*args, to_np(do), d ** -0.5, half=half(dtype))):
        close(a, ref, b)
    close(y, orc.layer_norm(to_np(o)), orc.layer_norm_bound(to_np(o)))
    # token by token: the norms of one row are the rows' own, bit by bit
    state = cuda_lib.new_decay_state(B, H, d)
    bo = orc.decay_attention_bound(*args, d ** -0.5)[0]
    want = orc.decay_attention(*args, d ** -0.5)[0]
    for i in range(L):
        qt, kt = cuda_lib.fwd_qk_norm_rotary(q[:, :, i:i + 1], k[:, :, i:i + 1], wq, wk, pos[:, :, i:i + 1].contiguous(),
                                             table, sections, "halves")
        assert torch.equal(qt[:, :, 0], qn[:, :, i]) and torch.equal(kt[:, :, 0], kn[:, :, i])
        ot, _ = cuda_lib.decay_attention_step(qt[:, :, 0], kt[:, :, 0], v[:, :, i], g, state, d ** -0.5)
        close(ot, want[:, :, i], bo[:, :, i], i)
