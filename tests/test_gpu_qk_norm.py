"""GPU parity of the norms of queries and keys with their rotation against the
fp64 oracle, element by element.

Tolerance of each element: the oracle's first-order bound of an fp32
evaluation, plus half a step of the storage type.
"""

import numpy as np
import pytest
import torch

import oracle as orc
from helpers import to_np
from test_gpu_sequence import LAYOUTS, ROTARY, close, gen, rotary_inputs, view

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-5
CASES = [c for c in ROTARY if c[4] <= 512] + [
    (1, 2, 1, 6, 512, (256,), True),
    (1, 1, 2, 5, 512, (8,), True),
    (2, 1, 1, 7, 500, (125, 125), False),
    (1, 2, 2, 5, 257, (3, 90), True),
    (1, 3, 1, 4, 510, (1, 254), True),
    (1, 4, 4, 3000, 32, (16,), True),
]


def inputs(case, dtype, seed):
    q, k, pos = rotary_inputs(case, dtype, seed)
    r = gen(seed + 1)
    q, k = (x * (0.25 + 4 * torch.rand(x.shape[:3] + (1,), generator=r)).to(dtype) for x in (q, k))
    d = case[4]
    wq, wk = 1 + 0.3 * torch.randn(d, generator=r), 1 + 0.3 * torch.randn(d, generator=r)
    dq, dk = torch.randn(q.shape, generator=r).to(dtype), torch.randn(k.shape, generator=r).to(dtype)
    return q, k, dq, dk, wq, wk, pos


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", CASES)
def test_matches_oracle(cuda_lib, case, dtype, halves):
    t = inputs(case, dtype, sum(case[:5]))
    q, k, dq, dk, wq, wk, pos = (x.cuda() for x in t)
    sections = case[5]
    table = cuda_lib.new_rotary_table(sections)
    turn = dict(pairing="halves" if halves else "adjacent", eps=EPS)
    out = cuda_lib.fwd_qk_norm_rotary(q, k, wq, wk, pos, table, sections, **turn)
    back = cuda_lib.bwd_qk_norm_rotary(q, k, dq, dk, wq, wk, pos, table, sections, **turn)
    freq, axis = orc.rotary_frequencies(sections)
    ang = (EPS, pos.cpu().numpy(), freq, axis, halves)
    for i, (x, w, dy) in enumerate(((q, wq, dq), (k, wk, dk))):
        X, W, D = to_np(x), to_np(w), to_np(dy)
        close(out[i], orc.qk_norm_rotary(X, W, *ang), orc.qk_norm_rotary_bound(X, W, *ang), i)
        for a, ref, b in zip((back[i], back[i + 2]), orc.qk_norm_rotary_grad(X, D, W, *ang),
                             orc.qk_norm_rotary_grad_bound(X, D, W, *ang)):
            close(a, ref, b, i)
    # without weights, without keys, without the weights' gradients
    Q, D = to_np(q), to_np(dq)
    alone, none = cuda_lib.fwd_qk_norm_rotary(q, None, None, None, pos, table, sections, **turn)
    assert none is None
    close(alone, orc.qk_norm_rotary(Q, None, *ang), orc.qk_norm_rotary_bound(Q, None, *ang))
    dx, dk_, dw, dwk_ = cuda_lib.bwd_qk_norm_rotary(q, None, dq, None, None, None, pos, table, sections, **turn)
    assert dk_ is None and dwk_ is None
    for a, ref, b in zip((dx, dw), orc.qk_norm_rotary_grad(Q, D, None, *ang),
                         orc.qk_norm_rotary_grad_bound(Q, D, None, *ang)):
        close(a, ref, b)
    only = cuda_lib.bwd_qk_norm_rotary(q, k, dq, dk, wq, wk, pos, table, sections, weight_grads=False, **turn)
    assert only[2] is None and only[3] is None
    assert torch.equal(only[0], back[0]) and torch.equal(only[1], back[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("case", [(2, 3, 2, 41, 64, (32,), True), (1, 4, 1, 30, 128, (20, 24), False),
                                  (2, 2, 2, 9, 33, (5, 8), True)])
@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
def test_layouts_and_in_place(cuda_lib, dtype, layout, case, pairing):
    t = inputs(case, dtype, 3)
    q, k, dq, dk, wq, wk, pos = (x.cuda() for x in t)
    sections = case[5]
    rest = (wq, wk, pos, cuda_lib.new_rotary_table(sections), sections, pairing)
    freq, axis = orc.rotary_frequencies(sections)
    ang = (EPS, pos.cpu().numpy(), freq, axis, pairing == "halves")
    qv, kv, dqv, dkv = (view(x, layout) for x in t[:4])
    out = cuda_lib.fwd_qk_norm_rotary(qv, kv, *rest)
    back = cuda_lib.bwd_qk_norm_rotary(qv, kv, dqv, dkv, *rest)
    for i, (x, w, dy) in enumerate(((q, wq, dq), (k, wk, dk))):
        X, W, D = to_np(x), to_np(w), to_np(dy)
        assert out[i].is_contiguous()
        close(out[i], orc.qk_norm_rotary(X, W, *ang), orc.qk_norm_rotary_bound(X, W, *ang))
        for a, ref, b in zip((back[i], back[i + 2]), orc.qk_norm_rotary_grad(X, D, W, *ang),
                             orc.qk_norm_rotary_grad_bound(X, D, W, *ang)):
            close(a, ref, b)
    # outputs in the inputs' layout, then in the inputs' places
    outs = [view(torch.zeros_like(x), layout) for x in t[:4]]
    cuda_lib.fwd_qk_norm_rotary(qv, kv, *rest, Qo=outs[0], Ko=outs[1])
    cuda_lib.bwd_qk_norm_rotary(qv, kv, dqv, dkv, *rest, dQ=outs[2], dK=outs[3])
    for a, b in zip(outs, (*out, *back[:2])):
        assert torch.equal(a, b)
    xs = [view(x, layout) for x in t[:4]]
    again = cuda_lib.bwd_qk_norm_rotary(*xs, *rest, dQ=xs[0], dK=xs[1])        # in the places of q and k
    assert again[0] is xs[0] and all(torch.equal(a, b) for a, b in zip(again, back))
    cuda_lib.bwd_qk_norm_rotary(qv, kv, dqv, dkv, *rest, dQ=dqv, dK=dkv)       # of the outputs' gradients
    cuda_lib.fwd_qk_norm_rotary(qv, kv, *rest, Qo=qv, Ko=kv)
    for a, b in zip((qv, kv, dqv, dkv), (*out, *back[:2])):
        assert torch.equal(a, b)
    if layout in ("joint", "even", "odd"):
        for x in (*outs, qv, kv, dqv, dkv):
            assert int(torch.isnan(x._base).sum()) == x._base.numel() - x.numel()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_bad_rows_and_zero_rows(cuda_lib, dtype):
    case = (1, 2, 2, 50, 64, (32,), True)
    t = inputs(case, dtype, 5)
    q, k, dq, dk, wq, wk, pos = (x.cuda() for x in t)
    rest = (wq, wk, pos, cuda_lib.new_rotary_table(case[5]), case[5])
    clean = cuda_lib.fwd_qk_norm_rotary(q, k, *rest)[0]
    grads = cuda_lib.bwd_qk_norm_rotary(q, k, dq, dk, *rest)
    bad = q.clone()
    bad[0, 0, 7, 3] = float("nan")
    bad[0, 0, 8, 5] = float("inf")
    bad[0, 0, 9] = 1e25                       # its squares leave fp32
    bad[0, 1, 9] = 0
    y = cuda_lib.fwd_qk_norm_rotary(bad, k, *rest)[0]
    dx = cuda_lib.bwd_qk_norm_rotary(bad, k, dq, dk, *rest, weight_grads=False)[0]
    assert torch.isnan(y[0, 0, 7:10]).all() and torch.isnan(dx[0, 0, 7:10]).all()
    assert (y[0, 1, 9] == 0).all() and torch.isfinite(dx[0, 1, 9]).all()
    keep = [i for i in range(50) if i not in (7, 8, 9)]
    assert torch.equal(y[:, :, keep], clean[:, :, keep]) and torch.equal(dx[:, :, keep], grads[0][:, :, keep])


def test_many_rows_are_all_summed(cuda_lib):
    # sums that are exact in any order: x = +-1 (mean x^2 = 1, eps chosen so that r = 1/2), whole gradients at position 0
    B, H, L, d = 3, 5, 70001, 32
    r = torch.Generator("cuda").manual_seed(1)
    x = (torch.randint(0, 2, (B, H, L, d), generator=r, device="cuda") * 2 - 1).to(BF16)
    dy = torch.randint(-2, 3, (B, H, L, d), generator=r, device="cuda").to(BF16)
    pos = torch.zeros((1, 1, L), dtype=torch.int32, device="cuda")
    table = cuda_lib.new_rotary_table((d // 2,))
    got = cuda_lib.bwd_qk_norm_rotary(x, x[:, :2], dy, dy[:, :2], None, None, pos, table, (d // 2,), eps=3.0)
    for dw, n in ((got[2], H), (got[3], 2)):
        want = (x[:, :n].double() * dy[:, :n].double()).sum((0, 1, 2)) / 2
        assert torch.equal(dw.double(), want)


def test_offsets_beyond_32_bits_and_streams(cuda_lib):
    case = (1, 2, 2, 40, 64, (32,), True)
    t = inputs(case, BF16, 9)
    q, k, dq, dk, wq, wk, pos = (x.cuda() for x in t)
    rest = (wq, wk, pos, cuda_lib.new_rotary_table(case[5]), case[5], "halves")
    far = 1 << 26
    buf = torch.empty(far * 40, dtype=BF16, device="cuda")
    views = []
    for i, x in enumerate(t[:4]):
        v = buf.as_strided((1, 2, 40, 64), (0, 64, far, 1), i * 256)
        v.copy_(x)
        views.append(v)
    want = (*cuda_lib.fwd_qk_norm_rotary(q, k, *rest), *cuda_lib.bwd_qk_norm_rotary(q, k, dq, dk, *rest))
    got = (*cuda_lib.fwd_qk_norm_rotary(*views[:2], *rest), *cuda_lib.bwd_qk_norm_rotary(*views, *rest))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (*cuda_lib.fwd_qk_norm_rotary(q, k, *rest, stream=side),
           *cuda_lib.bwd_qk_norm_rotary(q, k, dq, dk, *rest, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs = [torch.empty_like(x) for x in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.fwd_qk_norm_rotary(q, k, *rest, Qo=outs[0], Ko=outs[1])
        cuda_lib.bwd_qk_norm_rotary(q, k, dq, dk, *rest, dQ=outs[2], dK=outs[3], dq_weight=outs[4], dk_weight=outs[5])
    for _ in range(2):
        for x in outs:
            x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
