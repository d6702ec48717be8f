"""GPU parity of the sequence operators (layer norm, rotary positions, gated
scan) against the fp64 oracle, element by element.

Tolerance of each element: the oracle's first-order bound of an fp32
evaluation (``*_bound``), plus half a step of the storage type (2^-24 of the
value for fp32, 2^-8 for bf16), plus the smallest normal number of the type.
"""

import concurrent.futures
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle as orc
from helpers import to_np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def close(got, want, bound, what=""):
    """|got - want| within the bound and the rounding to got's type."""
    step = torch.finfo(got.dtype).eps / 2
    got = to_np(got)
    tol = (np.abs(want) + bound) * step + bound + 2.0 ** -126
    off = np.abs(got - want)
    assert got.shape == want.shape
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    with np.errstate(invalid="ignore"):
        bad = ~(off <= tol) & ~np.isnan(want) & ~(got == want)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), float(off[bad].max()),
                           float(tol[bad].min()))


def gen(seed):
    return torch.Generator(device="cpu").manual_seed(seed)


def view(t, layout, g=None):
    """The values of t [B, H, L, d] on the GPU in a memory layout: "plain";
    "tokens", a view of [B, L, H, d]; "joint", one of three parts of
    [B, L, 3, H, d]; "even", rows of d + 2 starting two elements in; "odd",
    rows of d + 3 starting one element in."""
    t = t.cuda()
    B, H, L, d = t.shape
    if layout == "plain":
        return t.contiguous()
    if layout == "tokens":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "joint":
        buf = torch.full((B, L, 3, H, d), float("nan"), dtype=t.dtype, device="cuda")
        out = buf[:, :, 1].transpose(1, 2)
    else:
        more, at = (2, 2) if layout == "even" else (3, 1)
        buf = torch.full((B, H, L, d + more), float("nan"), dtype=t.dtype, device="cuda")
        out = buf[..., at:] if layout == "even" else buf[..., at:d + at]
    out.copy_(t)
    return out


LAYOUTS = ["plain", "tokens", "joint", "even", "odd"]


# ---- gated scan -----------------------------------------------------------------

SCAN_SHAPES = [(1, 1, 1, 1), (2, 3, 2, 5), (1, 2, 17, 40), (2, 1, 129, 64), (3, 1, 1000, 33), (2, 2, 2500, 64),
               (1, 1, 6000, 130), (1, 40, 300, 16), (1, 150, 513, 64), (2, 300, 40, 32), (1, 1, 4096, 2)]


def scan_inputs(shape, dtype, seed, reset=()):
    B, H, L, d = shape
    r = gen(seed)
    slow = torch.exp(torch.rand((1, H, 1, d), generator=r) * 6 - 6)
    g = -2 * slow * torch.rand(shape, generator=r)
    for t in reset:
        if t < L:
            g[:, :, t] = -float("inf")
    x, dh = torch.randn(shape, generator=r), torch.randn(shape, generator=r)
    h0, dhT = torch.randn((B, H, d), generator=r), torch.randn((B, H, d), generator=r)
    return [t.to(dtype) for t in (x, g, dh)] + [h0, dhT]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SCAN_SHAPES)
def test_gated_scan_matches_oracle(cuda_lib, dtype, shape):
    x, g, dh, h0, dhT = scan_inputs(shape, dtype, sum(shape))
    xg, gg, dg_, sg, eg = x.cuda(), g.cuda(), dh.cuda(), h0.cuda(), dhT.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    h, hT = cuda_lib.fwd_gated_scan(xg, gg, h0=sg, dev_status=status)
    X, G, D, S, E = to_np(x), to_np(g), to_np(dh), to_np(h0), to_np(dhT)
    want, last = orc.gated_scan(X, G, S)
    bound = orc.gated_scan_bound(X, G, S)
    close(h, want, bound, "h")
    close(hT, last, bound[:, :, -1], "hT")
    dx, dg, dh0 = cuda_lib.bwd_gated_scan(gg, h, dg_, h0=sg, dhT=eg, dev_status=status)
    assert int(status.item()) == 0
    refs, bounds = orc.gated_scan_grad(G, to_np(h), D, S, E), orc.gated_scan_grad_bound(G, to_np(h), D, S, E)
    for name, got, ref, b in zip(("dx", "dg", "dh0"), (dx, dg, dh0), refs, bounds):
        close(got, ref, b, name)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("shape", [(2, 3, 77, 24), (1, 4, 700, 64), (2, 2, 1, 8)])
def test_gated_scan_layouts(cuda_lib, dtype, layout, shape):
    # no states, closed gates at a few tokens, and outputs in the inputs' layout
    x, g, dh, _, _ = scan_inputs(shape, dtype, 7, reset=(0, 5, 63, 64, 300))
    X, G, D = to_np(x), to_np(g), to_np(dh)
    xv, gv, dv = (view(t, layout) for t in (x, g, dh))
    out, dxo, dgo = (view(torch.zeros_like(t), layout) for t in (x, x, x))
    h, hT = cuda_lib.fwd_gated_scan(xv, gv, O=out)
    assert h is out
    want, last = orc.gated_scan(X, G)
    bound = orc.gated_scan_bound(X, G)
    close(h, want, bound, "h")
    close(hT, last, bound[:, :, -1], "hT")
    dx, dg, dh0 = cuda_lib.bwd_gated_scan(gv, h, dv, dX=dxo, dG=dgo)
    hn = to_np(h)
    for name, got, ref, b in zip(("dx", "dg", "dh0"), (dx, dg, dh0), orc.gated_scan_grad(G, hn, D),
                                 orc.gated_scan_grad_bound(G, hn, D)):
        close(got, ref, b, name)
    if layout in ("joint", "even", "odd"):                                # what lies between the rows is left as it was
        for t in (out, dxo, dgo):
            whole = t._base
            assert int(torch.isnan(whole).sum()) == whole.numel() - t.numel()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gated_scan_closed_gates_stop_infinities_and_nan(cuda_lib, dtype):
    shape = (2, 2, 900, 20)
    for low in (-float("inf"), torch.finfo(dtype).min):
        x, g, dh, h0, dhT = scan_inputs(shape, dtype, 11)
        g[:, :, 400] = low
        x[:, 0, 100] = float("inf")
        x[:, 1, 399] = float("nan")
        dh[:, :, 700] = float("nan")
        dh[:, 1, 401] = float("inf")
        X, G, S = to_np(x), to_np(g), to_np(h0)
        h, hT = cuda_lib.fwd_gated_scan(x.cuda(), g.cuda(), h0=h0.cuda())
        want, last = orc.gated_scan(X[:, :, 400:], G[:, :, 400:])
        bound = orc.gated_scan_bound(X[:, :, 400:], G[:, :, 400:])
        close(h[:, :, 400:], want, bound, "behind the gate")
        close(hT, last, bound[:, :, -1], "hT")
        assert torch.isinf(h[:, 0, 100:400]).all() and torch.isnan(h[:, 1, 399]).all()
        close(h[:, :, :100], *[f(X[:, :, :100], G[:, :, :100], S) for f in
                               (lambda *a: orc.gated_scan(*a)[0], orc.gated_scan_bound)], "before")
        dx, dg, dh0 = cuda_lib.bwd_gated_scan(g.cuda(), h, dh.cuda(), h0=h0.cuda(), dhT=dhT.cuda())
        assert (dg[:, :, 400] == 0).all()                         # NaN and infinity on both sides of it
        assert torch.isnan(dx[:, :, 400:701]).all()
        hn = to_np(h)[:, :, :400]
        hn[~np.isfinite(hn)] = 0                                  # dg there is checked below
        D = to_np(dh)[:, :, :400]
        refs, bounds = orc.gated_scan_grad(G[:, :, :400], hn, D, S), orc.gated_scan_grad_bound(G[:, :, :400], hn, D, S)
        close(dx[:, :, :400], refs[0], bounds[0], "dx before")
        close(dg[:, :, :100], refs[1][:, :, :100], bounds[1][:, :, :100], "dg before")
        close(dh0, refs[2], bounds[2], "dh0")
        assert not torch.isfinite(dg[:, 0, 101:400]).any()        # an infinite state's gates


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 7])
def test_gated_scan_closed_gates_stop_an_overflow(cuda_lib, dtype, d):
    """Finite inputs whose sum leaves fp32 inside a run: infinite as far as the next closed gate."""
    shape, top = (1, 2, 2100, d), 3e38
    x, g = torch.ones(shape, dtype=dtype, device="cuda"), torch.zeros(shape, dtype=dtype, device="cuda")
    x[:, :, :102] = 0
    x[:, :, 100] = top
    g[:, :, 102] = -float("inf")
    h0 = torch.full((1, 2, d), top, device="cuda")
    h, hT = cuda_lib.fwd_gated_scan(x, g, h0=h0)
    count = torch.arange(1, 2100 - 102 + 1, device="cuda", dtype=F32)
    assert torch.equal(h[:, :, 102:], count.to(dtype)[:, None].expand(1, 2, -1, d))     # whole numbers: exact
    assert torch.equal(hT, torch.full_like(h0, 2100 - 102))
    assert torch.isinf(h[:, :, 100:102]).all() and (h[:, :, :100] == torch.tensor(top, dtype=dtype)).all()
    # against time: the gradients behind token 102 grow too large at 104 and count from 101 down again
    dh = torch.ones(shape, dtype=dtype, device="cuda")
    dh[:, :, 103:] = 0
    dh[:, :, 104] = top
    h = torch.zeros_like(x)
    dx, dg, dh0 = cuda_lib.bwd_gated_scan(g, h, dh, dhT=h0)
    count = torch.arange(102, 0, -1, device="cuda", dtype=F32)
    assert torch.equal(dx[:, :, :102], count.to(dtype)[:, None].expand(1, 2, -1, d))
    assert torch.equal(dh0, torch.full_like(dh0, 102))
    assert torch.isinf(dx[:, :, 102:105]).all() and (dx[:, :, 105:] == torch.tensor(top, dtype=dtype)).all()
    assert (dg[:, :, :103] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gated_scan_padding_in_place_and_broadcast_gate(cuda_lib, dtype):
    shape = (2, 3, 333, 16)
    x, g, dh, h0, _ = scan_inputs(shape, dtype, 3)
    x[:, :, 200:] = 0
    g[:, :, 200:] = 0
    h, hT = cuda_lib.fwd_gated_scan(x.cuda(), g.cuda(), h0=h0.cuda())
    short = cuda_lib.fwd_gated_scan(x[:, :, :200].cuda(), g[:, :, :200].cuda(), h0=h0.cuda())
    close(hT, to_np(short[1]), orc.gated_scan_bound(to_np(x), to_np(g), to_np(h0))[:, :, -1])
    # in place: the same bits
    xi, si = x.cuda(), h0.cuda()
    o, s = cuda_lib.fwd_gated_scan(xi, g.cuda(), h0=si, O=xi, hT=si)
    assert o is xi and s is si and torch.equal(xi, h) and torch.equal(si, hT)
    gi = g.cuda()
    cuda_lib.fwd_gated_scan(x.cuda(), gi, h0=h0.cuda(), O=gi)
    assert torch.equal(gi, h)
    dx, dg, dh0 = cuda_lib.bwd_gated_scan(g.cuda(), h, dh.cuda(), h0=h0.cuda(), dhT=h0.cuda())
    di, gi, ei = dh.cuda(), g.cuda(), h0.cuda()
    cuda_lib.bwd_gated_scan(gi, h, di, h0=h0.cuda(), dhT=ei, dX=di, dG=gi, dh0=ei)
    assert torch.equal(di, dx) and torch.equal(gi, dg) and torch.equal(ei, dh0)
    # one gate for all heads; one for all channels has no unit stride and is refused
    with pytest.raises(cuda_lib.FavorError, match="unit stride"):
        cuda_lib.fwd_gated_scan(x.cuda(), g[:, :1, :, :1].cuda().expand(shape))
    gb = g[:, :1].cuda().expand(shape)
    hb, _ = cuda_lib.fwd_gated_scan(x.cuda(), gb)
    close(hb, orc.gated_scan(to_np(x), to_np(gb))[0], orc.gated_scan_bound(to_np(x), to_np(gb)))


def test_gated_scan_three_axes(cuda_lib):
    x, g, dh, h0, dhT = scan_inputs((2, 1, 100, 48), BF16, 5)
    a = cuda_lib.fwd_gated_scan(x.cuda(), g.cuda(), h0=h0.cuda())
    b = cuda_lib.fwd_gated_scan(x[:, 0].cuda(), g[:, 0].cuda(), h0=h0[:, 0].cuda())
    assert b[0].shape == (2, 100, 48) and b[1].shape == (2, 48)
    assert torch.equal(a[0][:, 0], b[0]) and torch.equal(a[1][:, 0], b[1])
    ga = cuda_lib.bwd_gated_scan(g.cuda(), a[0], dh.cuda(), h0.cuda(), dhT.cuda())
    gb = cuda_lib.bwd_gated_scan(g[:, 0].cuda(), b[0], dh[:, 0].cuda(), h0[:, 0].cuda(), dhT[:, 0].cuda())
    for u, v in zip(ga, gb):
        assert torch.equal(u[:, 0], v)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,d", [(1, 1, 1), (3, 5, 7), (4, 8, 64), (256, 8, 64), (2, 3, 1001)])
def test_gated_scan_steps_continue_a_prompt(cuda_lib, dtype, B, H, d):
    L, L0 = 24, 17
    x, g, _, h0, _ = scan_inputs((B, H, L, d), dtype, B + d, reset=(20,))
    X, G, S = to_np(x), to_np(g), to_np(h0)
    want, bound = orc.gated_scan(X, G, S)[0], orc.gated_scan_bound(X, G, S)
    _, state = cuda_lib.fwd_gated_scan(x[:, :, :L0].contiguous().cuda(), g[:, :, :L0].contiguous().cuda(),
                                       h0=h0.cuda())
    for t in range(L0, L):
        xt, gt = x[:, :, t].contiguous().cuda(), g[:, :, t].contiguous().cuda()
        apart, new = cuda_lib.gated_scan_step(xt, gt, state, new_state=torch.empty_like(state))
        o, same = cuda_lib.gated_scan_step(xt, gt, state)                     # in place
        assert same is state and torch.equal(new, state) and torch.equal(o, apart)
        close(o, want[:, :, t], bound[:, :, t], t)
        close(state, want[:, :, t], bound[:, :, t], t)


def test_gated_scan_offsets_beyond_32_bits(cuda_lib):
    # 2^31 + elements: the last channels and tokens against a run of them alone
    L, d = 262151, 8200
    free, _ = torch.cuda.mem_get_info()
    assert L * d > 1 << 31 and free > 40 << 30
    x = torch.empty((1, 1, L, d), dtype=BF16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    g = torch.empty_like(x).uniform_(-1, -0.5, generator=torch.Generator("cuda").manual_seed(2))
    h, hT = cuda_lib.fwd_gated_scan(x, g)
    # 60 tokens decay by e^-30 at least: what came before is below fp32
    tail, tailT = cuda_lib.fwd_gated_scan(x[:, :, -260:, -72:], g[:, :, -260:, -72:])
    X, G = to_np(x[:, :, -260:, -72:]), to_np(g[:, :, -260:, -72:])
    bound = orc.gated_scan_bound(X, G)[:, :, 60:] + 1e-10
    want = orc.gated_scan(X, G)[0]
    close(h[:, :, -200:, -72:], want[:, :, 60:], bound)
    close(hT[..., -72:], want[:, :, -1], bound[:, :, -1])
    dx, dg, dh0 = cuda_lib.bwd_gated_scan(g, h, x, dX=torch.empty_like(x))
    hn, D = to_np(h[:, :, -200:, -72:]), to_np(x[:, :, -200:, -72:])
    refs = orc.gated_scan_grad(G[:, :, 60:], hn, D, h0=to_np(h[:, :, -201, -72:]))
    bounds = orc.gated_scan_grad_bound(G[:, :, 60:], hn, D, h0=to_np(h[:, :, -201, -72:]))
    close(dx[:, :, -200:, -72:], refs[0], bounds[0])
    close(dg[:, :, -200:, -72:], refs[1], bounds[1])


# ---- layer norm ------------------------------------------------------------------

NORM_SHAPES = [(1, 1, 1, 1), (2, 1, 3, 2), (1, 3, 5, 7), (2, 3, 17, 40), (1, 16, 50, 64), (2, 8, 33, 128), (3, 1, 9, 96),
               (8, 1, 1, 512), (2, 1, 700, 512), (1, 1, 37, 771), (1, 1, 20, 1000), (1, 1, 5, 2048), (2, 1, 9, 4100),
               (1, 1, 3, 8192), (1, 1, 2, 16384), (1, 1, 2, 16383), (1, 1, 4500, 24)]


def norm_inputs(shape, dtype, seed):
    r = gen(seed)
    d = shape[-1]
    x = torch.randn(shape, generator=r) * (0.1 + 3 * torch.rand(shape[:3] + (1,), generator=r))
    x = x + 2 * torch.randn(shape[:3] + (1,), generator=r)
    x[0, 0, 0] = 1.5                                                          # a constant row
    gamma, beta = 1 + 0.3 * torch.randn(d, generator=r), 0.3 * torch.randn(d, generator=r)
    return x.to(dtype), torch.randn(shape, generator=r).to(dtype), gamma, beta


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", NORM_SHAPES)
def test_layer_norm_matches_oracle(cuda_lib, dtype, shape):
    x, dy, gamma, beta = norm_inputs(shape, dtype, sum(shape))
    X, D, W, Z = to_np(x), to_np(dy), to_np(gamma), to_np(beta)
    for w, z in ((W, Z), (None, None), (W, None), (None, Z)):
        dev = [None if t is None else torch.from_numpy(t).float().cuda() for t in (w, z)]
        close(cuda_lib.fwd_layer_norm(x.cuda(), *dev, 1e-3), orc.layer_norm(X, w, z, 1e-3),
              orc.layer_norm_bound(X, w, z, 1e-3), "y")
    for w in (W, None):
        wd = None if w is None else gamma.cuda()
        got = cuda_lib.bwd_layer_norm(x.cuda(), dy.cuda(), wd, 1e-3)
        for name, a, ref, b in zip(("dx", "dgamma", "dbeta"), got, orc.layer_norm_grad(X, D, w, 1e-3),
                                   orc.layer_norm_grad_bound(X, D, w, 1e-3)):
            close(a, ref, b, name)
        dx, none, nothing = cuda_lib.bwd_layer_norm(x.cuda(), dy.cuda(), wd, 1e-3, weight_grads=False)
        assert none is None and nothing is None and torch.equal(dx, got[0])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("shape", [(2, 3, 41, 64), (1, 2, 30, 128), (2, 2, 9, 33)])
def test_layer_norm_layouts_and_in_place(cuda_lib, dtype, layout, shape):
    x, dy, gamma, beta = norm_inputs(shape, dtype, 5)
    X, D, W, Z = to_np(x), to_np(dy), to_np(gamma), to_np(beta)
    xv, dv = view(x, layout), view(dy, layout)
    wd, zd = gamma.cuda(), beta.cuda()
    y = cuda_lib.fwd_layer_norm(xv, wd, zd)
    assert y.is_contiguous()
    close(y, orc.layer_norm(X, W, Z), orc.layer_norm_bound(X, W, Z))
    out = view(torch.zeros_like(x), layout)
    assert torch.equal(cuda_lib.fwd_layer_norm(xv, wd, zd, Y=out), y)
    got = cuda_lib.bwd_layer_norm(xv, dv, wd)
    for a, ref, b in zip(got, orc.layer_norm_grad(X, D, W), orc.layer_norm_grad_bound(X, D, W)):
        close(a, ref, b)
    for place in (0, 1):                                                       # dX in the place of X, of dY
        xs, ds = view(x, layout), view(dy, layout)
        again = cuda_lib.bwd_layer_norm(xs, ds, wd, dX=(xs, ds)[place])
        for a, b in zip(again, got):
            assert torch.equal(a, b)
    cuda_lib.fwd_layer_norm(xv, wd, zd, Y=xv)
    assert torch.equal(xv, y)
    if layout in ("joint", "even", "odd"):
        for t in (out, xv):
            assert int(torch.isnan(t._base).sum()) == t._base.numel() - t.numel()


def test_layer_norm_one_gradient_and_bad_rows(cuda_lib):
    lib = cuda_lib.load()
    x, dy, gamma, _ = (t.cuda() for t in norm_inputs((1, 1, 300, 96), F32, 9))
    dx, dgamma, dbeta = cuda_lib.bwd_layer_norm(x, dy, gamma)
    n = cuda_lib.bwd_layer_norm_workspace_bytes(1, 1, 300, 96, F32)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")              # NaN in every word
    for which in (0, 1):
        out = torch.full((96,), float("nan"), device="cuda")
        ptrs = [out.data_ptr(), None] if which == 0 else [None, out.data_ptr()]
        dxi = torch.empty_like(x)
        code = lib.favor_bwd_layer_norm(x.data_ptr(), None, dy.data_ptr(), None, dxi.data_ptr(), None,
                                        gamma.data_ptr(), *ptrs, 1e-5, 1, 1, 300, 96, 0, ws.data_ptr(), n,
                                        torch.cuda.current_stream().cuda_stream)
        assert code == 0 and torch.equal(out, (dgamma, dbeta)[which]) and torch.equal(dxi, dx)
    # a row of NaN or infinities stays in its row
    bad = x.clone()
    bad[0, 0, 7, 3] = float("nan")
    bad[0, 0, 8, 5] = float("inf")
    y, yb = cuda_lib.fwd_layer_norm(x, gamma), cuda_lib.fwd_layer_norm(bad, gamma)
    assert torch.isnan(yb[0, 0, 7:9]).all()
    keep = [i for i in range(300) if i not in (7, 8)]
    assert torch.equal(yb[0, 0, keep], y[0, 0, keep])


def test_layer_norm_many_rows(cuda_lib):
    # more rows than a grid's first wave, and offsets beyond 2^31 elements
    rows, d = (1 << 24) + 5, 136
    r = torch.Generator("cuda").manual_seed(3)
    x = torch.empty((1, 1, rows, d), dtype=BF16, device="cuda").normal_(generator=r)
    y = cuda_lib.fwd_layer_norm(x)
    for a, b in ((0, 40), (rows - 40, rows)):
        X = to_np(x[:, :, a:b])
        close(y[:, :, a:b], orc.layer_norm(X), orc.layer_norm_bound(X))
    dx, dgamma, dbeta = cuda_lib.bwd_layer_norm(x, y, dX=torch.empty_like(x))
    X, D = to_np(x[:, :, -40:]), to_np(y[:, :, -40:])
    close(dx[:, :, -40:], orc.layer_norm_grad(X, D)[0], orc.layer_norm_grad_bound(X, D)[0])
    # sum of y xh: y is xh but for its rounding; dbeta: sums of 2^24 values of mean 0
    xd = torch.zeros(d, dtype=torch.float64, device="cuda")
    bd = torch.zeros_like(xd)
    for c in x.view(rows, d).split(1 << 20):
        xc = c.double()
        xh = (xc - xc.mean(-1, keepdim=True)) / (xc.var(-1, correction=0, keepdim=True) + 1e-5).sqrt()
        yc = xh.to(BF16).double()
        xd += (xh * yc).sum(0)
        bd += yc.sum(0)
    # the kernel's y may round one step otherwise in few places: 1e-4 of the sum's terms by 2^-8
    depth = (128 + rows // 64) * orc.ROUND_F32
    assert float(((dgamma.double() - xd).abs() / xd).max()) < depth + 1e-4
    assert float((dbeta.double() - bd).abs().max()) < (depth + 1e-4) * rows


# ---- rotary positions ---------------------------------------------------------------

ROTARY = [
    # B, Hq, Hk, L, d, sections, one row of positions for all
    (1, 1, 1, 1, 2, (1,), True),
    (2, 3, 1, 5, 8, (1, 2), False),
    (2, 8, 8, 33, 64, (32,), True),
    (1, 4, 2, 100, 64, (16, 16), False),
    (1, 16, 4, 257, 128, (16, 24, 24), True),
    (3, 2, 2, 19, 80, (8, 0, 9, 3), False),
    (2, 5, 1, 7, 37, (3, 4), True),
    (64, 8, 8, 1, 64, (32,), False),
    (1, 40, 1, 600, 96, (24, 24), True),
    (1, 1, 1, 3, 1000, (500,), True),
    (1, 2, 2, 9, 64, (8,), True),
    (1, 3, 2, 11, 128, (20, 12), False),
]


def rotary_inputs(case, dtype, seed):
    B, Hq, Hk, L, d, sections, shared = case
    r = gen(seed)
    q, k = torch.randn((B, Hq, L, d), generator=r).to(dtype), torch.randn((B, Hk, L, d), generator=r).to(dtype)
    # near, far and negative positions
    pos = torch.randint(-200, 200, (len(sections), 1 if shared else B, L), generator=r)
    far = torch.rand(pos.shape, generator=r) < 0.3
    pos = torch.where(far, torch.randint(-(1 << 20), 1 << 20, pos.shape, generator=r), pos)
    return q, k, pos.to(torch.int32)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("case", ROTARY)
def test_rotary_matches_oracle(cuda_lib, dtype, halves, case):
    B, Hq, Hk, L, d, sections, _ = case
    q, k, pos = rotary_inputs(case, dtype, d + L)
    freq, axis = orc.rotary_frequencies(sections)
    table = cuda_lib.new_rotary_table(sections)
    pairing = "halves" if halves else "adjacent"
    P = len(freq)
    for back, call in ((False, cuda_lib.fwd_rotary), (True, cuda_lib.bwd_rotary)):
        qo, ko = call(q.cuda(), k.cuda(), pos.cuda(), table, sections, pairing)
        alone, none = call(q.cuda(), None, pos.cuda(), table, sections, pairing)
        assert none is None and torch.equal(alone, qo)
        for got, x in ((qo, q), (ko, k)):
            X = to_np(x)
            close(got, orc.rotary(X, pos.numpy(), freq, axis, halves, back), orc.rotary_bound(X, P, halves))
            assert torch.equal(got[..., 2 * P:].cpu(), x[..., 2 * P:])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("case", [ROTARY[3], ROTARY[5], ROTARY[11]])
def test_rotary_layouts_and_in_place(cuda_lib, dtype, halves, layout, case):
    B, Hq, Hk, L, d, sections, _ = case
    q, k, pos = rotary_inputs(case, dtype, 2)
    table = cuda_lib.new_rotary_table(sections)
    pairing = "halves" if halves else "adjacent"
    want = cuda_lib.fwd_rotary(q.cuda(), k.cuda(), pos.cuda(), table, sections, pairing)
    qv, kv = view(q, layout), view(k, layout)
    qo, ko = view(torch.zeros_like(q), layout), view(torch.zeros_like(k), layout)
    got = cuda_lib.fwd_rotary(qv, kv, pos.cuda(), table, sections, pairing, Qo=qo, Ko=ko)
    plain = cuda_lib.fwd_rotary(qv, kv, pos.cuda(), table, sections, pairing)
    cuda_lib.fwd_rotary(qv, kv, pos.cuda(), table, sections, pairing, Qo=qv, Ko=kv)
    # the angle's sine and cosine are the same in every kernel; products may be
    # contracted otherwise: two fp32 roundings, then one of the type
    for i, x in enumerate((q, k)):
        b = 4 * orc.ROUND_F32 * (1 + np.abs(to_np(x)).max()) + torch.finfo(dtype).eps * np.abs(to_np(want[i]))
        for t in (got[i], plain[i], (qv, kv)[i]):
            close(t, to_np(want[i]), b)
    assert plain[0].is_contiguous() and plain[1].is_contiguous()
    if layout in ("joint", "even", "odd"):
        for t in (qo, ko, qv, kv):
            assert int(torch.isnan(t._base).sum()) == t._base.numel() - t.numel()


def test_rotary_of_a_joint_buffer_and_extreme_positions(cuda_lib):
    # queries and keys of one buffer, both in place; the values beside them stay
    B, L, H, d = 2, 50, 4, 64
    r = gen(8)
    buf = torch.randn((B, L, 3, H, d), generator=r).cuda()
    was = buf.clone()
    sections = (16, 16)
    table = cuda_lib.new_rotary_table(sections)
    pos = torch.randint(0, 90, (2, 1, L), generator=r).int().cuda()
    q, k = (buf[:, :, i].transpose(1, 2) for i in (0, 1))
    want = cuda_lib.fwd_rotary(was[:, :, 0].transpose(1, 2), was[:, :, 1].transpose(1, 2), pos, table, sections)
    cuda_lib.fwd_rotary(q, k, pos, table, sections, Qo=q, Ko=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(buf[:, :, 2], was[:, :, 2])
    # position 0 is the identity; the largest 32-bit positions against whole-number arithmetic
    zero = torch.zeros((2, 1, L), dtype=torch.int32, device="cuda")
    assert torch.equal(cuda_lib.fwd_rotary(want[0], None, zero, table, sections)[0], want[0])
    words = [int(w) % (1 << 64) for w in table.tolist()]
    for p in (2 ** 31 - 1, -2 ** 31, 123456789):
        x = torch.ones((1, 1, 1, 2 * len(words)), device="cuda")
        at = torch.full((2, 1, 1), p, dtype=torch.int64).int().cuda()
        got = to_np(cuda_lib.fwd_rotary(x, None, at, table, sections)[0])[0, 0, 0]
        turns = np.array([float((p * w) % (1 << 64)) / 2.0 ** 64 for w in words]) * 2 * np.pi
        tol = orc.rotary_bound(np.ones((1, 1, 1, 2)), 1, False).max() + 2 * orc.ROUND_F32
        assert np.abs(got[0::2] - (np.cos(turns) - np.sin(turns))).max() < tol
        assert np.abs(got[1::2] - (np.cos(turns) + np.sin(turns))).max() < tol


def test_rotary_offsets_beyond_32_bits(cuda_lib):
    B, H, L, d = 1, 4, 1 << 22, 136
    x = torch.empty((B, H, L, d), dtype=BF16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(5))
    assert x.numel() > 1 << 31
    sections = (30, 38)
    pos = torch.stack([torch.arange(L), torch.arange(L) // 7]).int().view(2, 1, L).cuda()
    y, _ = cuda_lib.fwd_rotary(x, None, pos, cuda_lib.new_rotary_table(sections), sections, "halves")
    freq, axis = orc.rotary_frequencies(sections)
    for h in (0, H - 1):
        X = to_np(x[:, h:h + 1, -30:])
        close(y[:, h:h + 1, -30:], orc.rotary(X, pos[:, :, -30:].cpu().numpy(), freq, axis, True),
              orc.rotary_bound(X, 68, True))


# ---- streams, graphs, repeats ------------------------------------------------------------

def _all_calls(favor, t, workspace=None):
    """Every operator once on the tensors of t; the outputs."""
    h, hT = favor.fwd_gated_scan(t["x"], t["g"], h0=t["h0"], stream=t.get("stream"))
    grads = favor.bwd_gated_scan(t["g"], h, t["dh"], h0=t["h0"], dhT=t["dhT"], stream=t.get("stream"))
    step = favor.gated_scan_step(t["h0"], t["dhT"], t["h0"], new_state=t["next"], stream=t.get("stream"))
    y = favor.fwd_layer_norm(t["x"], t["gamma"], t["beta"], stream=t.get("stream"))
    norms = favor.bwd_layer_norm(t["x"], t["dh"], t["gamma"], workspace=workspace, stream=t.get("stream"))
    q, k = favor.fwd_rotary(t["x"], t["dh"], t["pos"], t["table"], (16, 16), stream=t.get("stream"))
    dq, dk = favor.bwd_rotary(q, k, t["pos"], t["table"], (16, 16), "halves", stream=t.get("stream"))
    return [h, hT, *grads, *step, y, *norms, q, k, dq, dk]


def _tensors(favor, seed, shape=(2, 4, 1500, 64)):
    x, g, dh, h0, dhT = (t.cuda() for t in scan_inputs(shape, F32, seed, reset=(700,)))
    r = gen(seed)
    d = shape[-1]
    return dict(x=x, g=g, dh=dh, h0=h0, dhT=dhT, next=torch.empty_like(h0), gamma=torch.randn(d, generator=r).cuda(),
                beta=torch.randn(d, generator=r).cuda(), table=favor.new_rotary_table((16, 16)),
                pos=torch.randint(0, 999, (2, 1, shape[2]), generator=r).int().cuda())


def test_repeats_give_the_same_bits(cuda_lib):
    t = _tensors(cuda_lib, 1)
    first = [o.clone() for o in _all_calls(cuda_lib, t)]
    for _ in range(3):
        for a, b in zip(first, _all_calls(cuda_lib, t)):
            assert torch.equal(a, b)


def test_calls_on_another_stream(cuda_lib):
    t = _tensors(cuda_lib, 2)
    want = [o.clone() for o in _all_calls(cuda_lib, t)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for given in (False, True):
        for _ in range(3):
            if given:
                outs = _all_calls(cuda_lib, dict(t, stream=side))
                # new tensors of the current stream must not take the workspace's place meanwhile
                junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(4)]
            else:
                with torch.cuda.stream(side):
                    outs = _all_calls(cuda_lib, t)
                junk = []
            torch.cuda.current_stream().wait_stream(side)
            for a, b in zip(want, outs):
                assert torch.equal(a, b)
            del junk


def test_outputs_on_another_stream_keep_off_the_current_ones_memory(cuda_lib):
    # a tensor of the current stream is freed while that stream has yet to read
    # it: what a call on another stream allocates must not take its place
    f = cuda_lib
    shape = (1, 4, 4096, 64)
    x, g, dh, h0, _ = (t.cuda() for t in scan_inputs(shape, F32, 1))
    w = torch.ones(64, device="cuda")
    pos = torch.arange(4096, device="cuda", dtype=torch.int32).view(1, 1, -1)
    table, new = f.new_rotary_table((32,)), torch.empty_like(h0)
    side = torch.cuda.Stream()
    calls = [lambda: f.fwd_gated_scan(x, g, stream=side), lambda: f.bwd_gated_scan(g, x, dh, stream=side),
             lambda: f.fwd_layer_norm(x, w, stream=side), lambda: f.bwd_layer_norm(x, dh, w, stream=side),
             lambda: f.fwd_rotary(x, dh, pos, table, (32,), stream=side),
             lambda: f.gated_scan_step(h0, h0, h0, new_state=new, stream=side)]
    for call in calls:
        for _ in range(2):
            torch.cuda.synchronize()
            olds = [torch.full(shape, 3.0, device="cuda") for _ in range(4)]
            olds += [torch.full((1, 4, 64), 3.0, device="cuda") for _ in range(3)]
            kept = [torch.empty_like(o) for o in olds]
            torch.cuda.synchronize()
            torch.cuda._sleep(20_000_000)                        # about 10 ms before the copies
            for a, b in zip(kept, olds):
                a.copy_(b)
            del olds, a, b
            call()
            torch.cuda.synchronize()
            assert all((k == 3.0).all() for k in kept)


def test_two_host_threads_at_once(cuda_lib):
    # each with its own stream and tensors
    ts = [_tensors(cuda_lib, seed) for seed in (7, 8)]
    want = [[o.clone() for o in _all_calls(cuda_lib, t)] for t in ts]
    streams = [torch.cuda.Stream() for _ in ts]
    torch.cuda.synchronize()

    def work(i):
        with torch.cuda.stream(streams[i]):
            outs = [_all_calls(cuda_lib, ts[i]) for _ in range(10)]
            streams[i].synchronize()
        return all(torch.equal(a, b) for o in outs for a, b in zip(want[i], o))

    with concurrent.futures.ThreadPoolExecutor(2) as ex:
        assert list(ex.map(work, (0, 1))) == [True, True]


def test_two_graphs_share_a_workspace(cuda_lib):
    a, b = _tensors(cuda_lib, 3), _tensors(cuda_lib, 4)
    ws = torch.empty(cuda_lib.bwd_layer_norm_workspace_bytes(2, 4, 1500, 64, F32), dtype=torch.uint8, device="cuda")
    want = [[o.clone() for o in _all_calls(cuda_lib, t)] for t in (a, b)]
    graphs, outs = [], []
    for t in (a, b):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_all_calls(cuda_lib, t, ws))
        graphs.append(g)
    ws.fill_(255)
    for which in (0, 1, 1, 0, 1):
        for o in outs[which]:
            o.zero_()
        graphs[which].replay()
        for x, y in zip(want[which], outs[which]):
            assert torch.equal(x, y)
    # new inputs in the captured places
    for key in ("x", "g", "dh", "h0", "dhT", "gamma", "beta", "pos"):
        a[key].copy_(b[key])
    graphs[0].replay()
    for x, y in zip(want[1], outs[0]):
        assert torch.equal(x, y)


def test_first_calls_under_capture(cuda_lib):
    # a process whose first call of each operator is made while a graph is captured
    code = """
import sys
import torch
sys.path.insert(0, sys.argv[1])
import linear_softmax_attention_gb300 as f
x = torch.randn((2, 4, 1500, 64), device="cuda").to(torch.bfloat16)
g = -x.abs()
w = torch.ones(64, device="cuda")
pos = torch.arange(1500, device="cuda", dtype=torch.int32).view(1, 1, -1)
table = f.new_rotary_table((32,))
def calls():
    h, hT = f.fwd_gated_scan(x, g)
    return [h, hT, *f.bwd_gated_scan(g, x, x), f.fwd_layer_norm(x, w), *f.bwd_layer_norm(x, x, w),
            *f.fwd_rotary(x, x, pos, table, (32,))]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    outs = calls()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(outs, calls()))
print("same")
"""
    r = subprocess.run([sys.executable, "-c", code, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_refusals_of_the_binding(cuda_lib):
    f, E = cuda_lib, cuda_lib.FavorError
    t = _tensors(f, 6, (2, 2, 8, 64))
    x, g, h0 = t["x"], t["g"], t["h0"]
    bad = [
        lambda: f.fwd_gated_scan(x, g.to(BF16)), lambda: f.fwd_gated_scan(x, g[:, :, :7]),
        lambda: f.fwd_gated_scan(x, g.cpu()), lambda: f.fwd_gated_scan(x, g, h0=h0.to(BF16)),
        lambda: f.fwd_gated_scan(x, g, h0=h0[:, :1]), lambda: f.fwd_gated_scan(x.half(), g.half()),
        lambda: f.fwd_gated_scan(x, g, O=x[:, :, 1:]), lambda: f.fwd_gated_scan(x[:, :, :0], g[:, :, :0]),
        lambda: f.fwd_gated_scan(x.transpose(2, 3), g.transpose(2, 3)), lambda: f.fwd_gated_scan(x[0, 0], g[0, 0]),
        lambda: f.bwd_gated_scan(g, x, x, dX=x), lambda: f.bwd_gated_scan(g, x, x, dX=g),
        lambda: f.gated_scan_step(x[:, :, 0], g[:, :, 0].contiguous(), h0),
        lambda: f.gated_scan_step(h0, h0, h0.to(BF16)), lambda: f.gated_scan_step(h0, h0, h0[:1]),
        lambda: f.fwd_layer_norm(x, t["gamma"][:5]), lambda: f.fwd_layer_norm(x, t["gamma"].double()),
        lambda: f.fwd_layer_norm(x, eps=0.0), lambda: f.fwd_layer_norm(x, eps=float("nan")),
        lambda: f.fwd_layer_norm(torch.zeros((1, 1, 1, 16385), device="cuda")),
        lambda: f.bwd_layer_norm(x, x[:, :, :3]), lambda: f.bwd_layer_norm(x, x, weight_grads=False, dbeta=t["beta"]),
        lambda: f.bwd_layer_norm(x, x, workspace=torch.empty(8, dtype=torch.uint8, device="cuda")),
        lambda: f.fwd_rotary(x, x, t["pos"], t["table"], (16, 16)),          # positions of 8 tokens are wanted
    ]
    pos = t["pos"][:, :, :8].contiguous()
    bad[-1] = lambda: f.fwd_rotary(x, x, t["pos"].repeat(1, 1, 2), t["table"], (16, 16))
    bad += [
        lambda: f.fwd_rotary(x, x, pos.long(), t["table"], (16, 16)), lambda: f.fwd_rotary(x, x, pos, t["table"], (16,)),
        lambda: f.fwd_rotary(x, x, pos[:1], t["table"], (16, 16)), lambda: f.fwd_rotary(x, x, pos, t["table"], (20, 20)),
        lambda: f.fwd_rotary(x, x, pos, t["table"].double(), (16, 16)),
        lambda: f.fwd_rotary(x, x, pos, t["table"], (16, 16), pairing="other"),
        lambda: f.fwd_rotary(x, x[:1], pos, t["table"], (16, 16)),
        lambda: f.fwd_rotary(x, x[0], pos, t["table"], (16, 16)),
        lambda: f.fwd_rotary(x, None, pos, t["table"], (16, 16), Ko=x),
        lambda: f.fwd_rotary(x, g, pos, t["table"], (16, 16), Qo=g),
        lambda: f.fwd_rotary(x, x, pos.expand(2, 2, 8)[:, :, ::2], t["table"], (16, 16)),
    ]
    before = {k: v.clone() for k, v in t.items() if isinstance(v, torch.Tensor)}
    for i, call in enumerate(bad):
        with pytest.raises(E):
            call()
            pytest.fail(f"call {i} was let through")
    torch.cuda.synchronize()
    for k, v in before.items():
        if k != "next":
            assert torch.equal(v, t[k]), k


# ---- together, as a model's layer uses them -------------------------------------------------

def _layer(favor, t, om, ws, s, causal=True):
    """Layer norm of the queries and keys inside the joint projection's
    output, rotation by row and column, the causal attention, then a gated
    scan over its outputs."""
    q, k = (favor.fwd_layer_norm(t["joint"][:, :, i].transpose(1, 2), t["wq"], None) for i in (0, 1))
    favor.fwd_rotary(q, k, t["pos"], t["table"], t["sections"], "halves", Qo=q, Ko=k)
    v = t["joint"][:, :, 2].transpose(1, 2).contiguous()
    a = favor.fwd_causal(q, k, v, om, s, ws)
    h, hT = favor.fwd_gated_scan(a, t["g"], h0=t["h0"])
    return q, k, v, a, h, hT


@pytest.mark.parametrize("dtype,d,m", [(F32, 32, 64), (BF16, 64, 256)])
def test_a_layer_forward_backward_and_by_tokens(cuda_lib, dtype, d, m):
    favor = cuda_lib
    B, H, L = 1, 2, 200
    r = gen(d)
    joint = torch.randn((B, L, 3, H, d), generator=r).to(dtype)
    g = (-torch.rand((B, H, L, d), generator=r)).to(dtype)
    h0, dh = torch.randn((B, H, d), generator=r), torch.randn((B, H, L, d), generator=r).to(dtype)
    wq = 1 + 0.1 * torch.randn(d, generator=r)
    sections = (d // 4, d // 4)
    pos = torch.stack([torch.arange(L) // 20, torch.arange(L) % 20]).int().view(2, 1, L)
    t = dict(joint=joint.cuda(), g=g.cuda(), h0=h0.cuda(), wq=wq.cuda(), pos=pos.cuda(), sections=sections,
             table=favor.new_rotary_table(sections))
    om = favor.new_omega(3, m, d)
    s = 0.5 * d ** -0.25
    ws = favor.new_workspace(True, B, H, L, d, m, dtype)
    q, k, v, a, h, hT = _layer(favor, t, om, ws, s)
    # the same in 64 bits
    J, G, S, W, OM = to_np(joint), to_np(g), to_np(h0), to_np(wq), to_np(om)
    freq, axis = orc.rotary_frequencies(sections)
    parts = [J[:, :, i].transpose(0, 2, 1, 3) for i in range(3)]
    N = [orc.layer_norm(p, W) for p in parts[:2]]
    Q, K = (orc.rotary(n, pos.numpy(), freq, axis, True) for n in N)
    A = orc.favor_causal(Q, K, parts[2], OM, s)
    Hh, _ = orc.gated_scan(A, G, S)
    tol = 1e-4 if dtype == F32 else 2e-2              # the attention's own bars; the operators' are far below
    assert orc.rowwise_rel_err(to_np(a), A) < tol
    assert orc.rowwise_rel_err(to_np(h), Hh) < tol
    # backward through all four
    da, dg, dh0 = favor.bwd_gated_scan(t["g"], h, dh.cuda(), h0=t["h0"])
    dq, dk, dv = favor.bwd_causal(q, k, v, da, om, s)
    favor.bwd_rotary(dq, dk, t["pos"], t["table"], sections, "halves", dQ=dq, dK=dk)
    grads, dw = [], []
    for i, dn in enumerate((dq, dk)):
        dx, dgamma, _ = favor.bwd_layer_norm(t["joint"][:, :, i].transpose(1, 2), dn, t["wq"])
        grads.append(dx)
        dw.append(dgamma)
    DA, DG, DH0 = orc.gated_scan_grad(G, Hh, to_np(dh), S)
    DQ, DK, DV = orc.favor_causal_grad(Q, K, parts[2], OM, s, DA)
    refs, rw = [], []
    for p, D in zip(parts, (DQ, DK)):
        dx, dgamma, _ = orc.layer_norm_grad(p, orc.rotary(D, pos.numpy(), freq, axis, True, True), W)
        refs.append(dx)
        rw.append(dgamma)

    def per_head(got, ref):
        got, ref = (v.reshape(B * H, -1) for v in (to_np(got), ref))
        return float((np.abs(got - ref).max(1) / np.abs(ref).max(1)).max())

    for got, ref in ((da, DA), (dg, DG), (dv, DV), (grads[0], refs[0]), (grads[1], refs[1]), (dh0, DH0)):
        assert per_head(got, ref) < 2 * tol           # two bf16 tensors are handed on between the calls
    for got, ref in zip(dw, rw):
        assert np.abs(to_np(got) - ref).max() < 2 * tol * np.abs(ref).max()
    # token by token: the same rows, from the state of the first 150
    n = 150
    state = favor.decode_prefill(k[:, :, :n].contiguous(), v[:, :, :n].contiguous(), om, s,
                                 favor.new_decode_state(B, H, m, d))
    _, mem = favor.fwd_gated_scan(a[:, :, :n], t["g"][:, :, :n], h0=t["h0"])
    for i in range(n, L):
        row = t["joint"][:, i:i + 1]
        qi, ki = (favor.fwd_layer_norm(row[:, :, j].transpose(1, 2), t["wq"], None) for j in (0, 1))
        favor.fwd_rotary(qi, ki, t["pos"][:, :, i:i + 1].contiguous(), t["table"], sections, "halves", Qo=qi, Ko=ki)
        ai = favor.decode_step(qi[:, :, 0], ki[:, :, 0], v[:, :, i].contiguous(), om, s, state)
        hi, _ = favor.gated_scan_step(ai, t["g"][:, :, i].contiguous(), mem)
        assert orc.rowwise_rel_err(to_np(hi), Hh[:, :, i]) < tol
