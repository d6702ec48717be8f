"""The norms of queries and keys with their rotation at the ends of what their
arguments may be, against the fp64 oracle (tolerances as in test_gpu_qk_norm)."""

import pytest
import torch

import oracle as orc
from helpers import to_np
from test_gpu_sequence import close, gen

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("d", [64, 16, 2])
@pytest.mark.parametrize("power", [-126, -127, -129, -132, -149])
def test_the_smallest_eps(cuda_lib, dtype, pairing, d, power):
    # rows of zeros, rows whose mean square is 2^-132 (every sum of them exact), and ordinary ones: 1 / sqrt(eps) and its
    # multiples are finite, its square need not be
    eps, L = 2.0 ** power, 12
    r = gen(7)
    x = torch.randn((1, 2, L, d), generator=r)
    x[:, :, 3:6] = 0
    x[:, :, 6:9] = 2.0 ** -66 * (1 - 2 * torch.randint(0, 2, (1, 2, 3, d), generator=r))
    x, dy = x.to(dtype), torch.randn(x.shape, generator=r).to(dtype)
    w = 1 + 0.3 * torch.randn(d, generator=r)
    pos = torch.randint(-1000, 1000, (1, 1, L), generator=r, dtype=torch.int32)
    freq, axis = orc.rotary_frequencies((d // 2,))
    ang = (eps, pos.numpy(), freq, axis, pairing == "halves")
    rest = (pos.cuda(), cuda_lib.new_rotary_table((d // 2,)), (d // 2,), pairing, eps)
    y, _ = cuda_lib.fwd_qk_norm_rotary(x.cuda(), None, w.cuda(), None, *rest)
    dx, _, dw, _ = cuda_lib.bwd_qk_norm_rotary(x.cuda(), None, dy.cuda(), None, w.cuda(), None, *rest)
    X, W, D = to_np(x), to_np(w), to_np(dy)
    close(y, orc.qk_norm_rotary(X, W, *ang), orc.qk_norm_rotary_bound(X, W, *ang), "y")
    for name, a, ref, b in zip(("dx", "dw"), (dx, dw), orc.qk_norm_rotary_grad(X, D, W, *ang),
                               orc.qk_norm_rotary_grad_bound(X, D, W, *ang)):
        close(a, ref, b, name)
