"""Binding of the sequence operators (``include/favor_ops.h``): layer norm and
rotary positions of queries and keys, and the gated linear recurrence.

As in the package itself every function only marshals arguments; the rules
are those of the header.  Tensors are [B, H, L, d] views with a unit stride
along d (any other strides); where a function says so, [B, L, d] stands for
H = 1.  Calls run on the tensors' device, on ``stream`` or that device's
current stream.
"""

from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import FavorError, _DT, _check, load

__all__ = ["fwd_gated_scan", "bwd_gated_scan", "gated_scan_step", "new_gated_scan_state", "fwd_layer_norm",
           "bwd_layer_norm", "bwd_layer_norm_workspace_bytes", "fwd_rotary", "bwd_rotary", "new_rotary_table"]

PAIRINGS = {"adjacent": 0, "halves": 1}              # favor_pairing
MAX_AXES = 4
_S3 = ctypes.c_int64 * 3
_NORM_MAX_D = 16384


def declare(lib):
    """Argument and result types of the entry points."""
    i, size, vp, f = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
    sizes = [i, i, i, i, i, vp]                       # B, H, L, d, dtype, stream
    lib.favor_fwd_gated_scan.argtypes = [vp] * 6 + [vp, vp] + sizes + [vp]
    lib.favor_bwd_gated_scan.argtypes = [vp] * 10 + [vp, vp, vp] + sizes + [vp]
    lib.favor_gated_scan_step.argtypes = [vp] * 5 + [i, i, i, i, vp]
    lib.favor_fwd_layer_norm.argtypes = [vp] * 4 + [vp, vp, f] + sizes
    lib.favor_bwd_layer_norm.argtypes = [vp] * 6 + [vp, vp, vp, f] + [i, i, i, i, i, vp, size, vp]
    lib.favor_bwd_layer_norm_workspace_bytes.argtypes = [i, i, i, i, i]
    lib.favor_fwd_rotary.argtypes = [vp] * 8 + [i] * 5 + [vp, i, i, vp, vp, i, i, vp]
    lib.favor_bwd_rotary.argtypes = lib.favor_fwd_rotary.argtypes
    for name in ("fwd_gated_scan", "bwd_gated_scan", "gated_scan_step", "fwd_layer_norm", "bwd_layer_norm",
                 "fwd_rotary", "bwd_rotary"):
        getattr(lib, "favor_" + name).restype = i
    lib.favor_bwd_layer_norm_workspace_bytes.restype = size


def _tensor(what, name, t, shape, dtype, device):
    """Pointer and strides (None: contiguous) of a view [B, H, L, d]."""
    if t.dtype != dtype or t.device != device or tuple(t.shape) != shape:
        raise FavorError(f"{what}: {name} must be a {dtype} tensor {list(shape)} on {device}, "
                         f"not {t.dtype} {list(t.shape)} on {t.device}")
    if t.is_contiguous():
        return t.data_ptr(), None
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise FavorError(f"{what}: {name} must have a unit stride along its last axis")
    return t.data_ptr(), (_S3(*st[:3]) if len(st) == 4 else _S3(st[0], 0, st[1]))


def _flat(what, name, t, shape, device):
    """Pointer of a contiguous fp32 tensor, None for None."""
    if t is None:
        return None
    if t.dtype != torch.float32 or t.device != device or tuple(t.shape) != shape or not t.is_contiguous():
        raise FavorError(f"{what}: {name} must be a contiguous fp32 tensor {list(shape)} on {device}")
    return t.data_ptr()


def _status(what, t, device):
    """Pointer of the optional device status, int32."""
    if t is None:
        return None
    if t.dtype != torch.int32 or t.device != device or t.numel() < 1:
        raise FavorError(f"{what}: dev_status must be an int32 tensor on {device}")
    return t.data_ptr()


def _sizes(what, name, t, dims=(3, 4)):
    """(B, H, L, d, shape) of a CUDA tensor [B, H, L, d] or [B, L, d]."""
    if not t.is_cuda or t.dtype not in _DT or t.dim() not in dims:
        raise FavorError(f"{what}: {name} must be an fp32 or bf16 CUDA tensor [B, H, L, d]"
                         + (" or [B, L, d]" if 3 in dims else ""))
    shape = tuple(t.shape)
    B, H, L, d = shape if len(shape) == 4 else (shape[0], 1, shape[1], shape[2])
    if min(B, H, L, d) < 1 or max(B, H, L, d) >= 1 << 31:
        raise FavorError(f"{what}: {name} has an empty or oversized axis: {list(shape)}")
    return B, H, L, d, shape


def _run(what, device, stream, args, made=()):
    """The call `what` on the tensors' device.  `made`: tensors allocated here
    on the current stream, used on `stream`."""
    fn = getattr(load(), what)
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _run(what, device, stream, args, made)
    current = torch.cuda.current_stream(device)
    if stream is None:
        stream = current
    else:
        if stream.device != device:
            raise FavorError(f"{what}: the stream belongs to {stream.device}, the tensors to {device}")
        if stream != current:
            for t in made:
                t.record_stream(stream)
    _check(fn(*args, stream.cuda_stream), what)


def new_gated_scan_state(B: int, H: int, d: int, device="cuda") -> torch.Tensor:
    """Zero state of the gated recurrence: fp32 [B, H, d]."""
    return torch.zeros((B, H, d), dtype=torch.float32, device=device)


def _state_shape(shape):
    return (shape[0], shape[1], shape[3]) if len(shape) == 4 else (shape[0], shape[2])


def fwd_gated_scan(X, G, h0=None, O=None, hT=None, dev_status=None, stream=None):
    """h_t = exp(G_t) h_{t-1} + X_t over the tokens of X, G [B, H, L, d] (or
    [B, L, d]), from the state h0 (fp32 [B, H, d] or [B, d], None: zeros).
    Returns (O, hT): every h_t in X's dtype and layout, and the last one in
    fp32.  A gate of minus infinity starts a new sequence; G = 0 with X = 0
    carries the state over padding.  O may be X or G, hT may be h0."""
    what = "favor_fwd_gated_scan"
    B, H, L, d, shape = _sizes(what, "X", X)
    dev, dt = X.device, X.dtype
    made = []
    if O is None:
        O = torch.empty_like(X)
        made.append(O)
    if hT is None:
        hT = torch.empty(_state_shape(shape), dtype=torch.float32, device=dev)
        made.append(hT)
    xp, xs = _tensor(what, "X", X, shape, dt, dev)
    gp, gs = _tensor(what, "G", G, shape, dt, dev)
    op, os_ = _tensor(what, "O", O, shape, dt, dev)
    state = _state_shape(shape)
    _run(what, dev, stream, (xp, xs, gp, gs, op, os_, _flat(what, "h0", h0, state, dev),
                             _flat(what, "hT", hT, state, dev), B, H, L, d, _DT[dt],
                             _status(what, dev_status, dev)), made)
    return O, hT


def bwd_gated_scan(G, O, dO, h0=None, dhT=None, dX=None, dG=None, dh0=None, dev_status=None, stream=None):
    """Gradients (dX, dG, dh0) of fwd_gated_scan for those of its outputs, dO
    and dhT (None: zeros); O is its output and h0 its initial state.  dX may
    be dO, dG may be G, dh0 may be dhT.  For a gate broadcast over an axis sum
    dG over it."""
    what = "favor_bwd_gated_scan"
    B, H, L, d, shape = _sizes(what, "G", G)
    dev, dt = G.device, G.dtype
    state = _state_shape(shape)
    made = []
    if dX is None:
        dX = torch.empty_like(dO)
        made.append(dX)
    if dG is None:
        dG = torch.empty_like(G)
        made.append(dG)
    if dh0 is None:
        dh0 = torch.empty(state, dtype=torch.float32, device=dev)
        made.append(dh0)
    args = []
    for name, t in (("G", G), ("O", O), ("dO", dO), ("dX", dX), ("dG", dG)):
        args += _tensor(what, name, t, shape, dt, dev)
    args += [_flat(what, "h0", h0, state, dev), _flat(what, "dhT", dhT, state, dev),
             _flat(what, "dh0", dh0, state, dev), B, H, L, d, _DT[dt], _status(what, dev_status, dev)]
    _run(what, dev, stream, args, made)
    return dX, dG, dh0


def gated_scan_step(x, g, state, o=None, new_state=None, stream=None):
    """One token: x, g contiguous [B, H, d], state fp32 [B, H, d].  Writes
    exp(g) state + x to new_state (None: in place) and returns (o, new_state),
    o the new state in x's dtype."""
    what = "favor_gated_scan_step"
    if not x.is_cuda or x.dtype not in _DT or x.dim() != 3:
        raise FavorError(f"{what}: x must be an fp32 or bf16 CUDA tensor [B, H, d]")
    shape = tuple(x.shape)
    dev, dt = x.device, x.dtype
    if min(shape) < 1:
        raise FavorError(f"{what}: x has an empty axis: {list(shape)}")
    made = ()
    if o is None:
        o = torch.empty_like(x, memory_format=torch.contiguous_format)
        made = (o,)
    new_state = state if new_state is None else new_state
    ptrs = []
    for name, t in (("x", x), ("g", g), ("o", o)):
        if t.dtype != dt or t.device != dev or tuple(t.shape) != shape or not t.is_contiguous():
            raise FavorError(f"{what}: {name} must be a contiguous {dt} tensor {list(shape)} on {dev}")
        ptrs.append(t.data_ptr())
    _run(what, dev, stream, (*ptrs, _flat(what, "state", state, shape, dev),
                             _flat(what, "new_state", new_state, shape, dev), *shape, _DT[dt]), made)
    return o, new_state


def fwd_layer_norm(X, gamma=None, beta=None, eps=1e-5, Y=None, stream=None):
    """Layer norm of X [B, H, L, d] (or [B, L, d]) over d, with gamma and beta
    (fp32 [d], None: 1 and 0).  Returns Y, contiguous where none is given (as
    the attention takes it); Y may be X."""
    what = "favor_fwd_layer_norm"
    B, H, L, d, shape = _sizes(what, "X", X)
    dev, dt = X.device, X.dtype
    made = ()
    if Y is None:
        Y = torch.empty(shape, dtype=dt, device=dev)
        made = (Y,)
    xp, xs = _tensor(what, "X", X, shape, dt, dev)
    yp, ys = _tensor(what, "Y", Y, shape, dt, dev)
    _run(what, dev, stream, (xp, xs, yp, ys, _flat(what, "gamma", gamma, (d,), dev),
                             _flat(what, "beta", beta, (d,), dev), float(eps), B, H, L, d, _DT[dt]), made)
    return Y


def bwd_layer_norm_workspace_bytes(B: int, H: int, L: int, d: int, dtype) -> int:
    if min(B, H, L, d) < 1 or d > _NORM_MAX_D or B * H * L >= 1 << 31:
        raise FavorError("unsupported shape")
    return load().favor_bwd_layer_norm_workspace_bytes(B, H, L, d, _DT[dtype])


def bwd_layer_norm(X, dY, gamma=None, eps=1e-5, dX=None, dgamma=None, dbeta=None, workspace=None, stream=None,
                   weight_grads=True):
    """Gradients (dX, dgamma, dbeta) of fwd_layer_norm for dY; X is its input.
    dgamma and dbeta are fp32 [d], summed over all rows; weight_grads=False
    leaves them out (None, None).  dX may be dY or X."""
    what = "favor_bwd_layer_norm"
    B, H, L, d, shape = _sizes(what, "X", X)
    dev, dt = X.device, X.dtype
    made = []
    if dX is None:
        dX = torch.empty(shape, dtype=dt, device=dev)
        made.append(dX)
    need = 0
    if weight_grads:
        need = bwd_layer_norm_workspace_bytes(B, H, L, d, dt)
        if dgamma is None:
            dgamma = torch.empty(d, dtype=torch.float32, device=dev)
            made.append(dgamma)
        if dbeta is None:
            dbeta = torch.empty(d, dtype=torch.float32, device=dev)
            made.append(dbeta)
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
            made.append(workspace)
    elif dgamma is not None or dbeta is not None:
        raise FavorError(f"{what}: dgamma or dbeta given with weight_grads=False")
    if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
        raise FavorError(f"{what}: the workspace must be contiguous on {dev}")
    args = []
    for name, t in (("X", X), ("dY", dY), ("dX", dX)):
        args += _tensor(what, name, t, shape, dt, dev)
    args += [_flat(what, "gamma", gamma, (d,), dev), _flat(what, "dgamma", dgamma, (d,), dev),
             _flat(what, "dbeta", dbeta, (d,), dev), float(eps), B, H, L, d, _DT[dt],
             workspace.data_ptr() if workspace is not None else None,
             workspace.numel() * workspace.element_size() if workspace is not None else 0]
    _run(what, dev, stream, args, made)
    return dX, dgamma, dbeta


def new_rotary_table(sections, base: float = 10000.0, freqs=None, device="cuda") -> torch.Tensor:
    """Table of the rotary calls: int64 [P] (the bits of a uint64), each pair's
    fraction of a turn per unit of position, a turn being 2^64.  Pair j of an
    axis with n pairs turns by base^(-j / n) radians, or, with ``freqs`` (P
    numbers), pair p by freqs[p]."""
    sections = _sections(tuple(int(n) for n in sections))[0]
    if freqs is None:
        freqs = [float(base) ** (-j / n) for n in sections for j in range(n)]
    else:
        freqs = [float(f) for f in freqs]
        if len(freqs) != sum(sections):
            raise FavorError(f"new_rotary_table: {len(freqs)} frequencies for {sum(sections)} pairs")
    words = []
    for f in freqs:
        if not math.isfinite(f):
            raise FavorError("new_rotary_table: frequencies must be finite")
        word = round(math.fmod(f / (2 * math.pi), 1.0) * 2.0 ** 64) % (1 << 64)
        words.append(word - (1 << 64) if word >= 1 << 63 else word)
    return torch.tensor(words, dtype=torch.int64, device=device)


@functools.lru_cache(maxsize=64)
def _sections(sections):
    """(sections, the C array, pairs)"""
    if not 1 <= len(sections) <= MAX_AXES or min(sections) < 0 or not 1 <= sum(sections) < 1 << 30:
        raise FavorError(f"sections must be 1 to {MAX_AXES} counts of pairs, not {sections}")
    return sections, (ctypes.c_int * len(sections))(*sections), sum(sections)


def _rotary(what, Q, K, pos, table, sections, pairing, Qo, Ko, stream):
    B, Hq, L, d, shape = _sizes(what, "Q", Q, (4,))
    dev, dt = Q.device, Q.dtype
    sections, c_sections, pairs = _sections(tuple(sections))
    if pairing not in PAIRINGS:
        raise FavorError(f"{what}: pairing must be one of {sorted(PAIRINGS)}")
    if 2 * pairs > d:
        raise FavorError(f"{what}: {pairs} pairs do not fit {d} channels")
    n = len(sections)
    ps = tuple(pos.shape)
    if (pos.dtype != torch.int32 or pos.device != dev or not pos.is_contiguous()
            or ps not in ((n, B, L), (n, 1, L))):
        raise FavorError(f"{what}: positions must be contiguous int32 [{n}, {B} or 1, {L}] on {dev}")
    if table.dtype != torch.int64 or table.device != dev or tuple(table.shape) != (pairs,) \
            or not table.is_contiguous():
        raise FavorError(f"{what}: the table must be contiguous int64 [{pairs}] on {dev} (new_rotary_table)")
    made = []
    if Qo is None:
        Qo = torch.empty(shape, dtype=dt, device=dev)
        made.append(Qo)
    args = [*_tensor(what, "Q", Q, shape, dt, dev), *_tensor(what, "its output", Qo, shape, dt, dev)]
    Hk = 0
    if K is not None:
        Hk, kshape = K.shape[1] if K.dim() == 4 else 0, (B, K.shape[1] if K.dim() == 4 else 0, L, d)
        if Hk < 1:
            raise FavorError(f"{what}: K must be [B, Hk, L, d]")
        if Ko is None:
            Ko = torch.empty(kshape, dtype=dt, device=dev)
            made.append(Ko)
        args += [*_tensor(what, "K", K, kshape, dt, dev), *_tensor(what, "its output", Ko, kshape, dt, dev)]
    else:
        if Ko is not None:
            raise FavorError(f"{what}: an output for keys without keys")
        args += [None] * 4
    args += [B, Hq, Hk, L, d, pos.data_ptr(), ps[1], n, c_sections, table.data_ptr(), PAIRINGS[pairing], _DT[dt]]
    _run(what, dev, stream, args, made)
    return Qo, Ko


def fwd_rotary(Q, K, pos, table, sections, pairing="adjacent", Qo=None, Ko=None, stream=None):
    """Rotates Q [B, H, L, d] and K [B, Hk, L, d] (or None) by the tokens'
    positions pos, int32 [axes, B or 1, L].  sections: the pairs of channels
    of each axis; table: new_rotary_table(sections).  pairing: "adjacent"
    (channels 2p and 2p + 1) or "halves" (p and p + pairs); channels behind
    the pairs are copied.  Returns (Qo, Ko), contiguous where none is given;
    Qo may be Q, Ko may be K."""
    return _rotary("favor_fwd_rotary", Q, K, pos, table, sections, pairing, Qo, Ko, stream)


def bwd_rotary(dQo, dKo, pos, table, sections, pairing="adjacent", dQ=None, dK=None, stream=None):
    """Gradients (dQ, dK) of fwd_rotary's inputs for those of its outputs: the
    rotation by the opposite angles; arguments as there."""
    return _rotary("favor_bwd_rotary", dQo, dKo, pos, table, sections, pairing, dQ, dK, stream)
