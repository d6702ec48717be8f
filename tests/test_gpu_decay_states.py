"""Calls of the decayed attention that leave states out: the other outputs are
those of the full calls, bit by bit, and the oracle's."""

import pytest
import torch

import oracle as orc
from helpers import to_np
from test_gpu_decay import check, half, inputs

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16

# up to 16 tokens; one chunk and a few, whose states are made beside the passes; one segment beyond 512 tokens (as many heads as
# CTAs run at once); several segments
SHAPES = [(2, 3, 9, 64), (3, 2, 16, 33), (2, 2, 100, 64), (2, 3, 333, 64), (1, 2, 512, 128), (30, 10, 700, 16),
          (15, 10, 600, 72), (2, 1, 2600, 64), (2, 1, 1500, 128), (1, 2, 900, 20)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_calls_without_states(cuda_lib, dtype, states, shape):
    t = inputs(shape, dtype, 17)
    q, k, v, do, g, S0, dST = (x.cuda() for x in t)
    if not states:
        S0 = dST = None
    ends = sorted({0, shape[0] - 1})                     # sequences that the oracle takes
    Q, K, V, D, S, E = (to_np(x[ends]) for x in (*t[:4], *t[5:]))
    G, hf = to_np(t[4]), half(dtype) if shape[2] > 16 else 0.0
    if not states:
        S = E = None
    for lengths in (None, [shape[2] - 1, 0, shape[2] // 2][:shape[0]] if shape[0] <= 3 else None):
        n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
        m = None if lengths is None else [lengths[i] for i in ends]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        full = (cuda_lib.fwd_decay_attention(q, k, v, g, 0.2, S0, n)[0],
                *cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.2, S0, dST, n)[:3])
        o, ST = cuda_lib.fwd_decay_attention(q, k, v, g, 0.2, S0, n, dev_status=status, last_state=False)
        *grads, dS0 = cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.2, S0, dST, n, dev_status=status,
                                                   first_state_grad=False)
        assert ST is None and dS0 is None and int(status.item()) == 0
        assert all(torch.equal(a, b) for a, b in zip((o, *grads), full))
        check(cuda_lib, "fwd", (o[ends],), orc.decay_attention(Q, K, V, G, 0.2, S, m),
              orc.decay_attention_bound(Q, K, V, G, 0.2, S, m, hf), ("o",))
        hb = half(dtype)
        check(cuda_lib, "bwd", [x[ends] for x in grads], orc.decay_attention_grad(Q, K, V, G, D, 0.2, S, E, m),
              orc.decay_attention_grad_bound(Q, K, V, G, D, 0.2, S, E, m, hb), ("dq", "dk", "dv"))


def test_without_states_in_graphs_and_on_streams(cuda_lib):
    for shape in ((4, 8, 333, 64), (2, 2, 1500, 64), (30, 10, 700, 16)):
        t = inputs(shape, BF16, 23)
        q, k, v, do, g, S0, dST = (x.cuda() for x in t)
        want = (cuda_lib.fwd_decay_attention(q, k, v, g, 0.1, S0)[0],
                *cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.1, S0, dST)[:3])
        outs = [torch.empty_like(x) for x in want]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cuda_lib.fwd_decay_attention(q, k, v, g, 0.1, S0, O=outs[0], last_state=False)
            cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.1, S0, dST, dQ=outs[1], dK=outs[2], dV=outs[3],
                                         first_state_grad=False)
        for _ in range(5):
            for x in outs:
                x.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        o, ST = cuda_lib.fwd_decay_attention(q, k, v, g, 0.1, S0, stream=side, last_state=False)
        *grads, dS0 = cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.1, S0, dST, stream=side, first_state_grad=False)
        torch.cuda.current_stream().wait_stream(side)
        assert ST is None and dS0 is None and all(torch.equal(a, b) for a, b in zip((o, *grads), want))


def test_a_state_given_and_left_out_is_refused(cuda_lib):
    q, k, v, do, g, S0, dST = (x.cuda() for x in inputs((1, 2, 20, 16), F32, 3))
    with pytest.raises(cuda_lib.FavorError, match="last_state"):
        cuda_lib.fwd_decay_attention(q, k, v, g, 0.2, S0, ST=S0, last_state=False)
    with pytest.raises(cuda_lib.FavorError, match="first_state_grad"):
        cuda_lib.bwd_decay_attention(q, k, v, g, do, 0.2, S0, dST, dS0=dST, first_state_grad=False)
