"""Sizes of the norms' backward workspace up to the most heads that the entry
points take: they follow the launch's grid, a CTA's sums [d] for each side."""

import pytest
import torch

import linear_softmax_attention_gb300 as favor

MOST = (1 << 31) - 16                # Hq + Hk


@pytest.mark.parametrize("heads", [MOST, MOST - 1, MOST - 47, MOST - 48, MOST - 49, 2110000000, 1 << 30, 70000, 65])
@pytest.mark.parametrize("Hk", [0, 1, 64])
def test_workspace_of_many_heads(heads, Hk):
    d = 2
    n = favor.bwd_qk_norm_rotary_workspace_bytes(1, heads - Hk, Hk, 1, d, torch.bfloat16)
    sides = 2 if Hk else 1
    # one token: one CTA beside another for every share of the heads, at most 32768 of them
    assert 0 < n <= 32768 * sides * d * 4 and n % (sides * d * 4) == 0


def test_more_heads_are_refused():
    for Hq, Hk in ((MOST, 1), (1, MOST), (MOST + 1, 0)):
        with pytest.raises(favor.FavorError):
            favor.bwd_qk_norm_rotary_workspace_bytes(1, Hq, Hk, 1, 2, torch.bfloat16)
