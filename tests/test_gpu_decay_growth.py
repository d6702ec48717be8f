"""The decayed attention with growing memories (g > 0), in the range that the
header gives: l^L and its products with what the tensors hold are finite."""

import pytest
import torch

from test_gpu_decay import both, inputs

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


# a few tokens, several segments, one segment of all tokens (as many heads as CTAs run at once); l^L up to e^70
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 2, 12, 64), (2, 2, 400, 64), (1, 2, 1400, 64), (1, 2, 1400, 128), (30, 10, 700, 16)])
def test_growing_memories(cuda_lib, dtype, shape):
    B, H, L, d = shape
    g = torch.linspace(0.0, 70.0 / L, H)
    t = inputs(shape, dtype, 29, g)
    # padding of zeros before the sequences' own tokens (and, for the gradients, behind them)
    pad = 2 * L // 5
    for x in t[1:3]:
        x[:, :, :pad] = 0
    both(cuda_lib, t, 0.1)
    t[3][:, :, L - pad:] = 0
    t[0][:, :, L - pad:] = 0
    both(cuda_lib, t, 0.1, states=False)
