"""The norms of queries and keys with their rotation over so many tokens that
every group of lanes walks from token to token with real rows ahead, against the
fp64 oracle (tolerances as in test_gpu_qk_norm)."""

import pytest
import torch

import oracle as orc
from helpers import to_np
from test_gpu_sequence import close

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16

# B, Hq, Hk, L, d, sections: a group takes another token beyond 48 groups (backward 16) an SM, of 2 to 32 tokens a CTA
LONG = [(1, 2, 1, 20011, 512, (200, 56)), (1, 2, 1, 130001, 64, (32,)), (2, 1, 2, 60007, 33, (5, 8)),
        (1, 1, 1, 250007, 16, (4,))]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("case", LONG)
def test_walks_from_token_to_token(cuda_lib, dtype, pairing, case):
    B, Hq, Hk, L, d, sections = case
    r = torch.Generator("cuda").manual_seed(d)
    q, dq, k, dk = (torch.randn((B, h, L, d), generator=r, device="cuda").to(dtype) for h in (Hq, Hq, Hk, Hk))
    wq, wk = (1 + 0.3 * torch.randn(d, generator=r, device="cuda") for _ in range(2))
    pos = torch.randint(-(1 << 20), 1 << 20, (len(sections), B, L), generator=r, device="cuda", dtype=torch.int32)
    rest = (wq, wk, pos, cuda_lib.new_rotary_table(sections), sections, pairing)
    out = cuda_lib.fwd_qk_norm_rotary(q, k, *rest)
    back = cuda_lib.bwd_qk_norm_rotary(q, k, dq, dk, *rest)
    freq, axis = orc.rotary_frequencies(sections)
    ang = (1e-5, pos.cpu().numpy(), freq, axis, pairing == "halves")
    for i, (x, w, dy) in enumerate(((q, wq, dq), (k, wk, dk))):
        X, W, D = to_np(x), to_np(w), to_np(dy)
        close(out[i], orc.qk_norm_rotary(X, W, *ang), orc.qk_norm_rotary_bound(X, W, *ang), i)
        for a, ref, b in zip((back[i], back[i + 2]), orc.qk_norm_rotary_grad(X, D, W, *ang),
                             orc.qk_norm_rotary_grad_bound(X, D, W, *ang)):
            close(a, ref, b, i)
