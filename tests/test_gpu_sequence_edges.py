"""The sequence operators where their inputs leave the ordinary range, against
the fp64 oracle, with the tolerances of ``test_gpu_sequence``."""

import numpy as np
import pytest
import torch

import oracle as orc
from helpers import to_np
from test_gpu_sequence import BF16, F32, close, gen, norm_inputs, scan_inputs, view

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("low", [-0.5, -2.0, -6.0, -14.0])
@pytest.mark.parametrize("L,d", [(7, 5), (20, 64), (3000, 8), (3000, 7), (60, 64)])
def test_open_gates_pass_infinities_and_nan_on(cuda_lib, dtype, low, L, d):
    """Gates whose products over a few tokens are below fp32 and which are
    open all the same: an infinity or NaN ends at a closed gate alone."""
    shape = (1, 3, L, d)
    x, g, dh, h0, dhT = scan_inputs(shape, dtype, L)
    g[:] = low
    at, shut = L // 3, L - L // 4
    g[:, :, shut] = -float("inf")
    x[:, 0, at], x[:, 1, at], h0[:, 2] = float("inf"), float("nan"), -float("inf")
    X, G, S = to_np(x), to_np(g), to_np(h0)
    h, hT = cuda_lib.fwd_gated_scan(x.cuda(), g.cuda(), h0=h0.cuda())
    with np.errstate(invalid="ignore"):
        want, last = orc.gated_scan(X, G, S)
        bound = orc.gated_scan_bound(X, G, S)
        assert np.isposinf(want[:, 0, at:shut]).all() and np.isfinite(want[:, :, shut:]).all()
        # behind the closed gate what came before does not count
        bound[:, :, shut:] = orc.gated_scan_bound(X[:, :, shut:], G[:, :, shut:])
        close(h, want, bound, "h")
        close(hT, last, bound[:, :, -1], "hT")
    # against time: from a late token to the closed gate, and from in front of it to the first token
    g[:, :, shut], g[:, :, at] = low, -float("inf")
    dh[:, 0, shut], dh[:, 1, shut], dhT[:, 2] = -float("inf"), float("nan"), float("inf")
    dh[:, 0, at // 2] = float("inf")
    G, D, E = to_np(g), to_np(dh), to_np(dhT)
    hn = torch.ones_like(x)
    dx, dg, dh0 = cuda_lib.bwd_gated_scan(g.cuda(), hn.cuda(), dh.cuda(), dhT=dhT.cuda())
    with np.errstate(invalid="ignore"):
        refs = orc.gated_scan_grad(G, to_np(hn), D, dhT=E)
        assert np.isposinf(refs[0][:, 2, at:]).all() and np.isfinite(refs[0][:, 1:, :at]).all()
        assert np.isposinf(refs[2][:, 0]).all()
        bounds = [np.nan_to_num(b, nan=0.0, posinf=0.0) for b in
                  orc.gated_scan_grad_bound(G, to_np(hn), D, dhT=E)]
        short = orc.gated_scan_grad_bound(G[:, :, :at], to_np(hn)[:, :, :at], np.nan_to_num(D[:, :, :at], posinf=0.0))
        for b, c in zip(bounds, short):
            if b.ndim == 4:
                b[:, :, :at] = c
            else:
                b[:] = c
        for name, got, ref, b in zip(("dx", "dg", "dh0"), (dx, dg, dh0), refs, bounds):
            close(got, ref, b, name)


@pytest.mark.parametrize("d,P", [(2, 1), (10, 5)])
def test_rotary_as_many_heads_as_there_may_be(cuda_lib, d, P):
    # the steps from share to share of the heads end just below 2^31; d = 10: 43 GB, in place
    H = (1 << 31) - 16
    free, _ = torch.cuda.mem_get_info()
    assert free > 60 << 30
    x = torch.ones((1, H, 1, d), dtype=BF16, device="cuda")
    pos = torch.ones((1, 1, 1), dtype=torch.int32, device="cuda")
    table = cuda_lib.new_rotary_table((P,), freqs=[0.5 * np.pi] * P)         # a quarter turn: (1, 1) -> (-1, 1)
    y, _ = cuda_lib.fwd_rotary(x, None, pos, table, (P,), Qo=x)
    want = torch.tensor([-1.0, 1.0] * P, device="cuda").to(BF16)
    for part in y.view(H, d).split(1 << 27):
        assert bool((part == want).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 1, 6000, 64), (2, 40, 3000, 64)])
@pytest.mark.parametrize("cycles,quits", [(0, -1), (2_000_000, 0), (2_000_000, 1)])
def test_gated_scan_ends_when_its_clusters_waits_run_out(cuda_lib, dtype, shape, cycles, quits):
    """Every wait, or those of one CTA of each cluster, as if over at once: the
    others' (2 million cycles, a millisecond) run out in turn, the status says
    so, and the calls after it are right."""
    x, g, _, _, _ = (t.cuda() for t in scan_inputs(shape, dtype, 1))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want, last = cuda_lib.fwd_gated_scan(x, g, dev_status=status)
    for _ in range(3):
        assert cuda_lib.selftest_scan_timeout(x, g, cycles, quits)[2] == 4      # FAVOR_ERR_TIMEOUT
        h, hT = cuda_lib.fwd_gated_scan(x, g, dev_status=status)
        assert torch.equal(h, want) and torch.equal(hT, last)
    h, hT, code = cuda_lib.selftest_scan_timeout(x, g, 2_200_000_000)           # the library's own limit
    assert code == 0 and torch.equal(h, want) and torch.equal(hT, last)
    assert int(status.item()) == 0


def test_arguments_may_be_let_go_after_a_call_on_another_stream(cuda_lib):
    # the other stream has yet to begin when the arguments are freed on the
    # current one, whose next tensors of their sizes must not take their place
    f = cuda_lib
    shape = (1, 4, 4096, 64)
    x, g, dh, h0, _ = (t.cuda() for t in scan_inputs(shape, F32, 1))
    w = torch.ones(64, device="cuda")
    pos = torch.arange(4096, device="cuda", dtype=torch.int32).view(1, 1, -1)
    table = f.new_rotary_table((32,))
    ws = torch.empty(f.bwd_layer_norm_workspace_bytes(1, 4, 4096, 64, F32), dtype=torch.uint8, device="cuda")
    calls = [(f.fwd_gated_scan, (x, g, h0), {}), (f.bwd_gated_scan, (g, x, dh, h0, h0), {}),
             (f.fwd_layer_norm, (x, w, w), {}), (f.bwd_layer_norm, (x, dh, w), dict(workspace=ws)),
             (f.fwd_rotary, (x, dh, pos, table, (32,)), {}), (f.bwd_rotary, (x, dh, pos, table, (32,)), {}),
             (f.gated_scan_step, (h0, h0, h0), {})]
    side = torch.cuda.Stream()
    clone = (lambda v: v.clone() if isinstance(v, torch.Tensor) else v)
    for call, args, more in calls:
        want = call(*map(clone, args), **{k: clone(v) for k, v in more.items()})
        want = want if isinstance(want, tuple) else (want,)
        a, kw = [clone(v) for v in args], {k: clone(v) for k, v in more.items()}
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)                        # about 10 ms
        got = call(*a, **kw, stream=side)
        sizes = [(v.shape, v.dtype) for v in (*a, *kw.values()) if isinstance(v, torch.Tensor)]
        del a, kw
        junk = [torch.full(s, 7, dtype=t, device="cuda") for s, t in sizes]
        torch.cuda.synchronize()
        for u, v in zip(got if isinstance(got, tuple) else (got,), want):
            assert torch.equal(u, v), call.__name__
        del junk


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", ["plain", "tokens", "odd"])
@pytest.mark.parametrize("shape", [(1, 2, 9, 64), (2, 1, 40, 33), (1, 3, 20, 16), (1, 1, 37, 771), (2, 1, 5, 1000),
                                   (1, 1, 3, 8192), (1, 1, 3, 4099)])
def test_layer_norm_of_rows_whose_squares_leave_fp32(cuda_lib, dtype, layout, shape):
    """They are NaN, never zeros; the rows beside them, of all other sizes, are right."""
    _, dy, gamma, beta = norm_inputs(shape, dtype, 2)
    r = gen(3)
    rows, d = shape[0] * shape[1] * shape[2], shape[3]
    x = torch.rand(shape, generator=r) + 0.5
    x[..., ::2] *= -1
    # squares are summed up to d (1.5 2^54)^2 < 2^125 in the good rows, from 2^130 on in the others
    scale = torch.randint(-40, 55, (rows,), generator=r)
    bad = torch.arange(rows) % 3 == 1
    scale[bad] = torch.randint(67, 127, (int(bad.sum()),), generator=r)
    x = torch.ldexp(x, scale.view(shape[:3] + (1,))).to(dtype)
    X, D, W, Z = (to_np(t) for t in (x, dy, gamma, beta))
    xv, dv, wd, zd = view(x, layout), view(dy, layout), gamma.cuda(), beta.cuda()
    bad = bad.view(shape[:3])
    good = ~bad.numpy()
    y = cuda_lib.fwd_layer_norm(xv, wd, zd, 1e-3)
    dx, dgamma, dbeta = cuda_lib.bwd_layer_norm(xv, dv, wd, 1e-3)
    for got in (y, dx):
        assert torch.isnan(got[bad.cuda()]).all()
    assert torch.isnan(dgamma).all()
    close(y[~bad.cuda()], orc.layer_norm(X, W, Z, 1e-3)[good], orc.layer_norm_bound(X, W, Z, 1e-3)[good], "y")
    close(dx[~bad.cuda()], orc.layer_norm_grad(X, D, W, 1e-3)[0][good],
          orc.layer_norm_grad_bound(X, D, W, 1e-3)[0][good], "dx")
    close(dbeta, orc.layer_norm_grad(X, D, W, 1e-3)[2], orc.layer_norm_grad_bound(X, D, W, 1e-3)[2], "dbeta")


@pytest.mark.parametrize("rows,d,odd", [((1 << 24) + 5, 128, False), (1 << 20, 34, True), (70001, 774, True),
                                        (50021, 2050, False), (3001, 12290, True), (300, 512, False)])
def test_layer_norm_weight_sums_miss_no_row(cuda_lib, rows, d, odd):
    """Rows of +1 and -1 with eps = 3: the variance is 1, 1 / sqrt(4) a half, and
    every sum a whole number of halves, ones or (dbeta of column 1) twos within 24
    bits: exact in fp32 in any order.  Half of the rows count at a time, each in
    one of the two."""
    def tensor():
        t = torch.zeros((1, 1, rows, d + (3 if odd else 0)), device="cuda")
        return t[..., 1:d + 1] if odd else t
    x, dy = tensor(), tensor()
    x[..., ::2], x[..., 1::2] = 1.0, -1.0
    assert torch.equal(cuda_lib.fwd_layer_norm(x[:, :, :50], eps=3.0), 0.5 * x[:, :, :50])
    dx = torch.empty_like(x)
    for parity in (0, 1):
        dy.zero_()
        dy[:, :, parity::2] = 1.0
        dy[..., 1] *= 2.0
        _, dgamma, dbeta = cuda_lib.bwd_layer_norm(x, dy, eps=3.0, dX=dx)
        n = float((rows + 1 - parity) // 2)
        want = torch.full((d,), n, device="cuda")
        want[1] = 2 * n
        assert torch.equal(dbeta, want)
        assert torch.equal(dgamma, 0.5 * want * x[0, 0, 0])


def test_calls_on_another_stream_are_captured(cuda_lib):
    # a graph whose capture forks to the other stream and joins it again; arguments are let go inside it
    f = cuda_lib
    x, g, dh, h0, _ = (t.cuda() for t in scan_inputs((2, 2, 700, 64), BF16, 4))
    w = torch.ones(64, device="cuda")
    pos = torch.arange(700, device="cuda", dtype=torch.int32).view(1, 1, -1)
    table = f.new_rotary_table((32,))

    def calls(**kw):
        n = f.fwd_layer_norm(x, w, **kw)
        q, k = f.fwd_rotary(n, dh, pos, table, (32,), **kw)
        h, hT = f.fwd_gated_scan(q, g, h0, **kw)
        grads = f.bwd_gated_scan(g, h, k, h0, **kw)
        return [h, hT, *grads, *f.bwd_layer_norm(x, grads[0], w, **kw)]

    want = calls()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        outs = calls(stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
