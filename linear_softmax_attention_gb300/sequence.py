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
_INT = (1 << 31) - 1
_PLAIN = torch.contiguous_format
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)     # None: a torch without CUDA
_current_device = getattr(torch._C, "_cuda_getDevice", None)


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
    lib.favor_selftest_scan_timeout.argtypes = [vp] * 4 + [i] * 5 + [ctypes.c_int64, i, vp, vp]
    lib.favor_selftest_scan_timeout.restype = i


# Small calls are bound by the host's time, so the helpers below ask torch for
# little: device indexes instead of devices, the raw handle of the current
# stream instead of a Stream object.

def _views(what, names, tensors, shape, dtype, index):
    """Pointer and strides (None: contiguous) of each view [B, H, L, d] or [B, L, d], in one list."""
    args = []
    for t in tensors:
        if t.shape != shape or t.dtype is not dtype or t.get_device() != index:
            name = names[len(args) // 2]
            raise FavorError(f"{what}: {name} must be a {dtype} tensor {list(shape)} on cuda:{index}, "
                             f"not {t.dtype} {list(t.shape)} on {t.device}")
        args.append(t.data_ptr())
        if t.is_contiguous():
            args.append(None)
            continue
        st = t.stride()
        if st[-1] != 1 and shape[-1] > 1:
            raise FavorError(f"{what}: {names[len(args) // 2]} must have a unit stride along its last axis")
        args.append(_S3(st[0], st[1], st[2]) if len(st) == 4 else _S3(st[0], 0, st[1]))
    return args


def _flats(what, names, tensors, shape, index, dtype=torch.float32):
    """Pointers of contiguous tensors of one shape, None for None."""
    args = []
    for t in tensors:
        if t is None:
            args.append(None)
        elif t.shape != shape or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
            raise FavorError(f"{what}: {names[len(args)]} must be a contiguous {dtype} tensor {list(shape)} "
                             f"on cuda:{index}")
        else:
            args.append(t.data_ptr())
    return args


def _status(what, t, index):
    """Pointer of the optional device status, int32."""
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.get_device() != index or t.numel() < 1:
        raise FavorError(f"{what}: dev_status must be an int32 tensor on cuda:{index}")
    return t.data_ptr()


def _sizes(what, name, t, four_only=False):
    """B, H, L, d, dtype, device index of a CUDA tensor [B, H, L, d] or [B, L, d]."""
    dims = t.dim()
    if not t.is_cuda or t.dtype not in _DT or (dims != 4 and (four_only or dims != 3)):
        raise FavorError(f"{what}: {name} must be an fp32 or bf16 CUDA tensor [B, H, L, d]"
                         + ("" if four_only else " or [B, L, d]"))
    if dims == 4:
        B, H, L, d = t.shape
    else:
        B, L, d = t.shape
        H = 1
    if B < 1 or H < 1 or L < 1 or d < 1 or B > _INT or H > _INT or L > _INT or d > _INT:
        raise FavorError(f"{what}: {name} has an empty or oversized axis: {list(t.shape)}")
    return B, H, L, d, t.dtype, t.get_device()


def _call(what, index, args):
    """The entry point `what` on device `index`, on its current stream."""
    if index != _current_device():
        with torch.cuda.device(index):
            return _call(what, index, args)
    code = getattr(load(), what)(*args, _raw_stream(index))
    if code != 0:
        _check(code, what)


def _on(stream, fn, t, *args):
    """fn(t, *args) with `stream` as the current one of t's device: what is
    allocated there comes from that stream's memory, which no other stream's
    pending work reads.  The results may then be used on the stream that was
    current before, and the arguments let go: their memory waits for the call."""
    if not t.is_cuda or stream.device != t.device:
        raise FavorError(f"{fn.__name__}: the stream belongs to {stream.device}, the tensors to {t.device}")
    current = torch.cuda.current_stream(t.device)
    if stream == current:
        return fn(t, *args)
    with torch.cuda.stream(stream):
        out = fn(t, *args)
    for a in (t, *args):
        if isinstance(a, torch.Tensor):
            a.record_stream(stream)
    for o in out if isinstance(out, tuple) else (out,):
        if o is not None:
            o.record_stream(current)
    return out


def new_gated_scan_state(B: int, H: int, d: int, device="cuda") -> torch.Tensor:
    """Zero state of the gated recurrence: fp32 [B, H, d]."""
    return torch.zeros((B, H, d), dtype=torch.float32, device=device)


def fwd_gated_scan(X, G, h0=None, O=None, hT=None, dev_status=None, stream=None):
    """h_t = exp(G_t) h_{t-1} + X_t over the tokens of X, G [B, H, L, d] (or
    [B, L, d]), from the state h0 (fp32 [B, H, d] or [B, d], None: zeros).
    Returns (O, hT): every h_t in X's dtype and layout, and the last one in
    fp32.  A gate of minus infinity starts a new sequence; G = 0 with X = 0
    carries the state over padding.  O may be X or G, hT may be h0."""
    if stream is not None:
        return _on(stream, fwd_gated_scan, X, G, h0, O, hT, dev_status)
    what = "favor_fwd_gated_scan"
    B, H, L, d, dt, dev = _sizes(what, "X", X)
    shape = X.shape
    state = (B, H, d) if len(shape) == 4 else (B, d)
    if O is None:
        O = torch.empty_like(X)
    if hT is None:
        hT = torch.empty(state, dtype=torch.float32, device=X.device)
    _call(what, dev,
          (*_views(what, ("X", "G", "O"), (X, G, O), shape, dt, dev), *_flats(what, ("h0", "hT"), (h0, hT), state, dev),
           B, H, L, d, _DT[dt], _status(what, dev_status, dev)))
    return O, hT


def bwd_gated_scan(G, O, dO, h0=None, dhT=None, dX=None, dG=None, dh0=None, dev_status=None, stream=None):
    """Gradients (dX, dG, dh0) of fwd_gated_scan for those of its outputs, dO
    and dhT (None: zeros); O is its output and h0 its initial state.  dX may
    be dO, dG may be G, dh0 may be dhT.  For a gate broadcast over an axis sum
    dG over it."""
    if stream is not None:
        return _on(stream, bwd_gated_scan, G, O, dO, h0, dhT, dX, dG, dh0, dev_status)
    what = "favor_bwd_gated_scan"
    B, H, L, d, dt, dev = _sizes(what, "G", G)
    shape = G.shape
    state = (B, H, d) if len(shape) == 4 else (B, d)
    if dX is None:
        dX = torch.empty_like(dO)
    if dG is None:
        dG = torch.empty_like(G)
    if dh0 is None:
        dh0 = torch.empty(state, dtype=torch.float32, device=G.device)
    _call(what, dev,
          (*_views(what, ("G", "O", "dO", "dX", "dG"), (G, O, dO, dX, dG), shape, dt, dev),
           *_flats(what, ("h0", "dhT", "dh0"), (h0, dhT, dh0), state, dev), B, H, L, d, _DT[dt],
           _status(what, dev_status, dev)))
    return dX, dG, dh0


def gated_scan_step(x, g, state, o=None, new_state=None, stream=None):
    """One token: x, g contiguous [B, H, d], state fp32 [B, H, d].  Writes
    exp(g) state + x to new_state (None: in place) and returns (o, new_state),
    o the new state in x's dtype."""
    if stream is not None:
        return _on(stream, gated_scan_step, x, g, state, o, new_state)
    what = "favor_gated_scan_step"
    dt, shape, dev = x.dtype, x.shape, x.get_device()
    if dev < 0 or dt not in _DT or len(shape) != 3:
        raise FavorError(f"{what}: x must be an fp32 or bf16 CUDA tensor [B, H, d]")
    B, H, d = shape
    if B < 1 or H < 1 or d < 1 or B > _INT or H > _INT or d > _INT:
        raise FavorError(f"{what}: x has an empty or oversized axis: {list(shape)}")
    if o is None:
        o = torch.empty_like(x, memory_format=_PLAIN)
    if new_state is None:
        new_state = state
    _call(what, dev,
          (*_flats(what, ("x", "g", "o"), (x, g, o), shape, dev, dt),
           *_flats(what, ("state", "new_state"), (state, new_state), shape, dev), B, H, d, _DT[dt]))
    return o, new_state


def selftest_scan_timeout(X, G, wait_cycles, quits=-1):
    """favor_selftest_scan_timeout: fwd_gated_scan of contiguous X and G with
    another limit of its clusters' waits, and with those of CTA `quits` of each
    cluster running out at once.  Returns (O, hT, status) after synchronising."""
    what = "favor_selftest_scan_timeout"
    B, H, L, d, dt, dev = _sizes(what, "X", X, True)
    O = torch.empty_like(X, memory_format=_PLAIN)
    hT = torch.empty((B, H, d), dtype=torch.float32, device=X.device)
    status = torch.zeros(1, dtype=torch.int32, device=X.device)
    _call(what, dev, (*_flats(what, ("X", "G", "O"), (X, G, O), X.shape, dev, dt), hT.data_ptr(), B, H, L, d, _DT[dt],
                      wait_cycles, quits, status.data_ptr()))
    return O, hT, int(status.item())


def fwd_layer_norm(X, gamma=None, beta=None, eps=1e-5, Y=None, stream=None):
    """Layer norm of X [B, H, L, d] (or [B, L, d]) over d, with gamma and beta
    (fp32 [d], None: 1 and 0).  Returns Y, contiguous where none is given (as
    the attention takes it); Y may be X."""
    if stream is not None:
        return _on(stream, fwd_layer_norm, X, gamma, beta, eps, Y)
    what = "favor_fwd_layer_norm"
    B, H, L, d, dt, dev = _sizes(what, "X", X)
    shape = X.shape
    if Y is None:
        Y = torch.empty_like(X, memory_format=_PLAIN)
    _call(what, dev,
          (*_views(what, ("X", "Y"), (X, Y), shape, dt, dev),
           *_flats(what, ("gamma", "beta"), (gamma, beta), (d,), dev), eps, B, H, L, d, _DT[dt]))
    return Y


def bwd_layer_norm_workspace_bytes(B: int, H: int, L: int, d: int, dtype, device=None) -> int:
    """Bytes of bwd_layer_norm's workspace on `device` (None: the current
    one), whose number of SMs it depends on."""
    if device is not None and device != _current_device():
        with torch.cuda.device(device):
            return bwd_layer_norm_workspace_bytes(B, H, L, d, dtype)
    n = 0
    if min(B, H, L, d) > 0 and max(B, H, L, d) <= _INT:
        n = load().favor_bwd_layer_norm_workspace_bytes(B, H, L, d, _DT[dtype])
    if n == 0:
        raise FavorError("unsupported shape")
    return n


def bwd_layer_norm(X, dY, gamma=None, eps=1e-5, dX=None, dgamma=None, dbeta=None, workspace=None, stream=None,
                   weight_grads=True):
    """Gradients (dX, dgamma, dbeta) of fwd_layer_norm for dY; X is its input.
    dgamma and dbeta are fp32 [d], summed over all rows; weight_grads=False
    leaves them out (None, None).  dX may be dY or X."""
    if stream is not None:
        return _on(stream, bwd_layer_norm, X, dY, gamma, eps, dX, dgamma, dbeta, workspace, None, weight_grads)
    what = "favor_bwd_layer_norm"
    B, H, L, d, dt, dev = _sizes(what, "X", X)
    shape = X.shape
    if dX is None:
        dX = torch.empty_like(X, memory_format=_PLAIN)
    if weight_grads:
        if dgamma is None:
            dgamma = torch.empty(d, dtype=torch.float32, device=X.device)
        if dbeta is None:
            dbeta = torch.empty(d, dtype=torch.float32, device=X.device)
        if workspace is None:
            workspace = torch.empty(bwd_layer_norm_workspace_bytes(B, H, L, d, dt, dev), dtype=torch.uint8,
                                    device=X.device)
    elif dgamma is not None or dbeta is not None:
        raise FavorError(f"{what}: dgamma or dbeta given with weight_grads=False")
    ws, nbytes = None, 0
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise FavorError(f"{what}: the workspace must be contiguous on cuda:{dev}")
        ws, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _call(what, dev,
          (*_views(what, ("X", "dY", "dX"), (X, dY, dX), shape, dt, dev),
           *_flats(what, ("gamma", "dgamma", "dbeta"), (gamma, dgamma, dbeta), (d,), dev), eps, B, H, L, d, _DT[dt],
           ws, nbytes))
    return dX, dgamma, dbeta


_PI_BITS = 1200          # frequencies are below 2^1024: beyond 2^64 turns' fraction of the largest


@functools.lru_cache(maxsize=None)
def _two_pi():
    """2 pi 2^_PI_BITS in whole numbers, by Machin's formula."""
    guard = 32
    one = 1 << (_PI_BITS + guard)

    def arctan_of_inverse(x):
        total, power, k = 0, one // x, 1
        while power:
            total += power // k if k % 4 == 1 else -(power // k)
            power //= x * x
            k += 2
        return total

    return 8 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239)) >> guard


def new_rotary_table(sections, base: float = 10000.0, freqs=None, device="cuda") -> torch.Tensor:
    """Table of the rotary calls: int64 [P] (the bits of a uint64), each pair's
    fraction of a turn per unit of position, a turn being 2^64, rounded once
    from the frequency in 64-bit floating point.  Pair j of an
    axis with n pairs turns by base^(-j / n) radians, or, with ``freqs`` (P
    numbers), pair p by freqs[p]."""
    sections = _sections(tuple(int(n) for n in sections))[0]
    if freqs is None:
        base = float(base)
        if not (math.isfinite(base) and base > 0):
            raise FavorError(f"new_rotary_table: the base must be positive and finite, not {base}")
        try:
            freqs = [base ** (-j / n) for n in sections for j in range(n)]
        except OverflowError:
            raise FavorError(f"new_rotary_table: frequencies of base {base} are out of range") from None
    else:
        freqs = [float(f) for f in freqs]
        if len(freqs) != sum(sections):
            raise FavorError(f"new_rotary_table: {len(freqs)} frequencies for {sum(sections)} pairs")
    words = []
    for f in freqs:
        if not math.isfinite(f):
            raise FavorError("new_rotary_table: frequencies must be finite")
        n, m = f.as_integer_ratio()                  # n / m radians: 2^64 n / (m 2 pi), to the nearest
        den = m * _two_pi()
        word = ((n << (_PI_BITS + 65)) + den) // (2 * den) % (1 << 64)
        words.append(word - (1 << 64) if word >= 1 << 63 else word)
    return torch.tensor(words, dtype=torch.int64, device=device)


@functools.lru_cache(maxsize=64)
def _sections(sections):
    """(sections, the C array, pairs)"""
    if not 1 <= len(sections) <= MAX_AXES or min(sections) < 0 or not 1 <= sum(sections) < 1 << 30:
        raise FavorError(f"sections must be 1 to {MAX_AXES} counts of pairs, not {sections}")
    return sections, (ctypes.c_int * len(sections))(*sections), sum(sections)


def _rotary(Q, K, what, pos, table, sections, pairing, Qo, Ko, stream):
    if stream is not None:
        return _on(stream, _rotary, Q, K, what, pos, table, sections, pairing, Qo, Ko, None)
    B, Hq, L, d, dt, dev = _sizes(what, "Q", Q, True)
    sections, c_sections, pairs = _sections(sections if type(sections) is tuple else tuple(sections))
    pairing = PAIRINGS.get(pairing)
    if pairing is None:
        raise FavorError(f"{what}: pairing must be one of {sorted(PAIRINGS)}")
    n = len(sections)
    if (pos.dtype is not torch.int32 or pos.get_device() != dev or not pos.is_contiguous()
            or (pos.shape != (n, B, L) and pos.shape != (n, 1, L))):
        raise FavorError(f"{what}: positions must be contiguous int32 [{n}, {B} or 1, {L}] on cuda:{dev}")
    if Qo is None:
        Qo = torch.empty_like(Q, memory_format=_PLAIN)
    views = _views(what, ("Q", "Q's output"), (Q, Qo), Q.shape, dt, dev)
    Hk = 0
    if K is not None:
        Hk = K.shape[1] if K.dim() == 4 else 0
        if Hk < 1 or Hk > _INT:
            raise FavorError(f"{what}: K must be [B, Hk, L, d]")
        shape = (B, Hk, L, d)
        if Ko is None:
            Ko = torch.empty_like(K, memory_format=_PLAIN)
        views += _views(what, ("K", "K's output"), (K, Ko), shape, dt, dev)
    elif Ko is None:
        views += (None, None, None, None)
    else:
        raise FavorError(f"{what}: an output for keys without keys")
    _call(what, dev,
          (*views, B, Hq, Hk, L, d, pos.data_ptr(), pos.shape[1], n, c_sections,
           *_flats(what, ("the table (new_rotary_table)",), (table,), (pairs,), dev, torch.int64), pairing, _DT[dt]))
    return Qo, Ko


def fwd_rotary(Q, K, pos, table, sections, pairing="adjacent", Qo=None, Ko=None, stream=None):
    """Rotates Q [B, H, L, d] and K [B, Hk, L, d] (or None) by the tokens'
    positions pos, int32 [axes, B or 1, L].  sections: the pairs of channels
    of each axis; table: new_rotary_table(sections).  pairing: "adjacent"
    (channels 2p and 2p + 1) or "halves" (p and p + pairs); channels behind
    the pairs are copied.  Returns (Qo, Ko), contiguous where none is given;
    Qo may be Q, Ko may be K."""
    return _rotary(Q, K, "favor_fwd_rotary", pos, table, sections, pairing, Qo, Ko, stream)


def bwd_rotary(dQo, dKo, pos, table, sections, pairing="adjacent", dQ=None, dK=None, stream=None):
    """Gradients (dQ, dK) of fwd_rotary's inputs for those of its outputs: the
    rotation by the opposite angles; arguments as there."""
    return _rotary(dQo, dKo, "favor_bwd_rotary", pos, table, sections, pairing, dQ, dK, stream)
