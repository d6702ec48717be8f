"""Binding of the causal linear attention with a decay per head
(``include/favor_ops.h``): whole sequences, their gradients and one token at a
time from the carried state.

As in the package itself every function only marshals arguments; the rules
are those of the header.  Q, K, V and O are [B, H, L, d] views with a unit
stride along d (any other strides), states fp32 [B, H, d, d] (key channel,
value channel).  Calls run on the tensors' device, on ``stream`` or that
device's current stream.
"""

from __future__ import annotations

import ctypes
import functools

import torch

from . import FavorError, _DT, load
from .sequence import _INT, _PLAIN, _call, _current_device, _flats, _on, _sizes, _status, _views

__all__ = ["fwd_decay_attention", "bwd_decay_attention", "decay_attention_step", "new_decay_state",
           "decay_attention_workspace_bytes"]

_S2 = ctypes.c_int64 * 2


def declare(lib):
    """Argument and result types of the entry points."""
    i, size, vp, f = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
    lib.favor_fwd_decay_attention.argtypes = [vp] * 8 + [vp] * 4 + [f] + [i] * 5 + [vp, size, vp, vp]
    lib.favor_bwd_decay_attention.argtypes = [vp] * 14 + [vp] * 5 + [f] + [i] * 5 + [vp, size, vp, vp]
    lib.favor_decay_attention_step.argtypes = [vp] * 8 + [vp] * 3 + [f] + [i] * 4 + [vp]
    for name in ("fwd_decay_attention", "bwd_decay_attention", "decay_attention_step"):
        getattr(lib, "favor_" + name).restype = i
    lib.favor_decay_attention_workspace_bytes.argtypes = [i] * 6
    lib.favor_decay_attention_workspace_bytes.restype = size


def new_decay_state(B: int, H: int, d: int, device="cuda") -> torch.Tensor:
    """Zero state of the decayed attention: fp32 [B, H, d, d]."""
    return torch.zeros((B, H, d, d), dtype=torch.float32, device=device)


def decay_attention_workspace_bytes(B: int, H: int, L: int, d: int, dtype, backward: bool = False,
                                    device=None) -> int:
    """Bytes of the workspace of fwd_decay_attention (``backward``: of
    bwd_decay_attention) on `device` (None: the current one), whose number of
    SMs it depends on; 0 where none is needed."""
    if device is not None and device != _current_device():
        with torch.cuda.device(device):
            return decay_attention_workspace_bytes(B, H, L, d, dtype, backward)
    if dtype not in _DT or min(B, H, L, d) < 1 or max(B, H, L, d) > _INT:
        raise FavorError("unsupported shape")
    return load().favor_decay_attention_workspace_bytes(B, H, L, d, _DT[dtype], int(backward))


# a shape's size on a device never changes
_workspace_bytes = functools.lru_cache(maxsize=1024)(decay_attention_workspace_bytes)


def _workspace(what, workspace, B, H, L, d, dt, dev, backward):
    """(tensor to keep, pointer, bytes)"""
    if workspace is None:
        n = _workspace_bytes(B, H, L, d, dt, backward, dev)
        if n == 0:
            return None, None, 0
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise FavorError(f"{what}: the workspace must be contiguous on cuda:{dev}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def fwd_decay_attention(Q, K, V, g, scale=1.0, S0=None, lengths=None, O=None, ST=None, workspace=None,
                        dev_status=None, stream=None, last_state=True):
    """O_t = scale S_t^T Q_t of S_t = exp(g) S_{t-1} + K_t V_t^T over the tokens
    of Q, K, V [B, H, L, d], from the state S0 (None: zeros).  g: the logarithms
    of the heads' decays, fp32 [H], <= 0.  lengths: int32 [B], tokens of each
    sequence (None: L); rows behind them are not used, and 0 in O.  Returns
    (O, ST), ST the state behind each sequence's last token; ST may be S0.
    last_state=False leaves it out (None)."""
    if stream is not None:
        return _on(stream, fwd_decay_attention, Q, K, V, g, scale, S0, lengths, O, ST, workspace, dev_status, None,
                   last_state)
    what = "favor_fwd_decay_attention"
    B, H, L, d, dt, dev = _sizes(what, "Q", Q, True)
    if O is None:
        O = torch.empty_like(Q, memory_format=_PLAIN)
    state = (B, H, d, d)
    if not last_state:
        if ST is not None:
            raise FavorError(f"{what}: ST given with last_state=False")
    elif ST is None:
        ST = torch.empty(state, dtype=torch.float32, device=dev)
    workspace, ws, nbytes = _workspace(what, workspace, B, H, L, d, dt, dev, False)
    _call(what, dev,
          (*_views(what, ("Q", "K", "V", "O"), (Q, K, V, O), Q.shape, dt, dev), *_flats(what, ("g",), (g,), (H,), dev),
           *_flats(what, ("lengths",), (lengths,), (B,), dev, torch.int32),
           *_flats(what, ("S0", "ST"), (S0, ST), state, dev), scale, B, H, L, d, _DT[dt], ws, nbytes,
           _status(what, dev_status, dev)))
    return O, ST


def bwd_decay_attention(Q, K, V, g, dO, scale=1.0, S0=None, dST=None, lengths=None, dQ=None, dK=None, dV=None,
                        dS0=None, workspace=None, dev_status=None, stream=None, first_state_grad=True):
    """Gradients (dQ, dK, dV, dS0) of fwd_decay_attention for those of its
    outputs, dO and dST (None: zeros); the other arguments as there.  dS0 may
    be dST; first_state_grad=False leaves it out (None).  The decays are
    constants and have none."""
    if stream is not None:
        return _on(stream, bwd_decay_attention, Q, K, V, g, dO, scale, S0, dST, lengths, dQ, dK, dV, dS0, workspace,
                   dev_status, None, first_state_grad)
    what = "favor_bwd_decay_attention"
    B, H, L, d, dt, dev = _sizes(what, "Q", Q, True)
    if dQ is None:
        dQ = torch.empty_like(Q, memory_format=_PLAIN)
    if dK is None:
        dK = torch.empty_like(Q, memory_format=_PLAIN)
    if dV is None:
        dV = torch.empty_like(Q, memory_format=_PLAIN)
    state = (B, H, d, d)
    if not first_state_grad:
        if dS0 is not None:
            raise FavorError(f"{what}: dS0 given with first_state_grad=False")
    elif dS0 is None:
        dS0 = torch.empty(state, dtype=torch.float32, device=dev)
    workspace, ws, nbytes = _workspace(what, workspace, B, H, L, d, dt, dev, True)
    _call(what, dev,
          (*_views(what, ("Q", "K", "V", "dO", "dQ", "dK", "dV"), (Q, K, V, dO, dQ, dK, dV), Q.shape, dt, dev),
           *_flats(what, ("g",), (g,), (H,), dev), *_flats(what, ("lengths",), (lengths,), (B,), dev, torch.int32),
           *_flats(what, ("S0", "dST", "dS0"), (S0, dST, dS0), state, dev), scale, B, H, L, d, _DT[dt], ws, nbytes,
           _status(what, dev_status, dev)))
    return dQ, dK, dV, dS0


def decay_attention_step(q, k, v, g, state, scale=1.0, o=None, new_state=None, stream=None):
    """One token: q, k, v [B, H, d] views with a unit stride along d, state fp32
    [B, H, d, d].  Writes exp(g) state + k v^T to new_state (None: in place) and
    returns (o, new_state), o = scale new_state^T q in q's dtype."""
    if stream is not None:
        return _on(stream, decay_attention_step, q, k, v, g, state, scale, o, new_state)
    what = "favor_decay_attention_step"
    dt, shape, dev = q.dtype, q.shape, q.get_device()
    if dev < 0 or dt not in _DT or len(shape) != 3:
        raise FavorError(f"{what}: q must be an fp32 or bf16 CUDA tensor [B, H, d]")
    B, H, d = shape
    if B < 1 or H < 1 or d < 1 or B > _INT or H > _INT or d > _INT:
        raise FavorError(f"{what}: q has an empty or oversized axis: {list(shape)}")
    if o is None:
        o = torch.empty(shape, dtype=dt, device=dev)
    if new_state is None:
        new_state = state
    args = []
    for t in (q, k, v, o):
        if t.shape != shape or t.dtype is not dt or t.get_device() != dev:
            raise FavorError(f"{what}: {'qkvo'[len(args) // 2]} must be a {dt} tensor {list(shape)} on cuda:{dev}, "
                             f"not {t.dtype} {list(t.shape)} on {t.device}")
        args.append(t.data_ptr())
        if t.is_contiguous():
            args.append(None)
            continue
        st = t.stride()
        if st[2] != 1 and d > 1:
            raise FavorError(f"{what}: {'qkvo'[len(args) // 2]} must have a unit stride along its last axis")
        args.append(_S2(st[0], st[1]))
    if state is None or new_state is None:
        raise FavorError(f"{what}: a state is needed (new_decay_state)")
    _call(what, dev,
          (*args, *_flats(what, ("g",), (g,), (H,), dev),
           *_flats(what, ("state", "new_state"), (state, new_state), (B, H, d, d), dev), scale, B, H, d, _DT[dt]))
    return o, new_state
