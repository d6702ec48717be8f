"""Argument checks of the decayed attention and of the norms with rotation that
need no GPU: the C ABI refuses before anything is launched, the binding before
it calls."""

import ctypes

import pytest
import torch

import linear_softmax_attention_gb300 as favor
from test_abi_cpu import lib  # noqa: F401  (the built library)

BAD, UNSUPPORTED, LAUNCHED = 1, 2, 3
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="addresses of this test are not memory")
NAN, INF = float("nan"), float("inf")

# B = 1, H = 2, L = 8, d = 8 in fp32: 512 bytes a tensor, 512 a state
FWD = dict(q=0x10000, k=0x20000, v=0x30000, o=0x40000, g=0x50000, lengths=0x60000, S0=0x70000, ST=0x80000, scale=1.0,
           B=1, H=2, L=8, d=8, dt=0, ws=None, n=0, st=None)


def s3(*s):
    return (ctypes.c_int64 * 3)(*s)


def fwd(lib, **kw):
    a = {**FWD, "strides": {}, **kw}
    s = a["strides"]
    return lib.favor_fwd_decay_attention(a["q"], s.get("q"), a["k"], s.get("k"), a["v"], s.get("v"), a["o"], s.get("o"),
                                         a["g"], a["lengths"], a["S0"], a["ST"], a["scale"], a["B"], a["H"], a["L"],
                                         a["d"], a["dt"], a["ws"], a["n"], None, None)


def bwd(lib, **kw):
    a = {**FWD, "do": 0x40000, "dq": 0x90000, "dk": 0xa0000, "dv": 0xb0000, "dST": 0x80000, "dS0": 0xc0000,
         "strides": {}, **kw}
    s = a["strides"]
    args = []
    for name in ("q", "k", "v", "do", "dq", "dk", "dv"):
        args += [a[name], s.get(name)]
    return lib.favor_bwd_decay_attention(*args, a["g"], a["lengths"], a["S0"], a["dST"], a["dS0"], a["scale"], a["B"],
                                         a["H"], a["L"], a["d"], a["dt"], a["ws"], a["n"], None, None)


def step(lib, **kw):
    a = dict(q=0x10000, k=0x20000, v=0x30000, o=0x40000, g=0x50000, state=0x70000, new=0x70000, scale=1.0, B=1, H=2,
             d=8, dt=0, s=None)
    a.update(kw)
    return lib.favor_decay_attention_step(a["q"], a["s"], a["k"], None, a["v"], None, a["o"], None, a["g"], a["state"],
                                          a["new"], a["scale"], a["B"], a["H"], a["d"], a["dt"], None)


def test_decay_attention_refusals(lib):  # noqa: F811
    for call in (fwd, bwd):
        for name in ("B", "H", "L", "d"):
            assert call(lib, **{name: 0}) == BAD
            assert call(lib, **{name: -3}) == BAD
        assert call(lib, dt=2) == BAD
        assert call(lib, d=129) == UNSUPPORTED
        assert call(lib, B=1 << 10, H=1 << 10) == UNSUPPORTED
        assert call(lib, L=(1 << 30) + 1) == UNSUPPORTED
        for name in ("q", "k", "v", "g"):
            assert call(lib, **{name: None}) == BAD
            assert call(lib, **{name: 0x50002}) == BAD          # not on an element
        assert call(lib, lengths=0x60002) == BAD
        assert call(lib, S0=0x70002) == BAD
        for scale in (NAN, INF):
            assert call(lib, scale=scale) == BAD
        assert call(lib, strides={"k": s3(64, -8, 8)}) == BAD   # a negative stride
    outputs = {fwd: ("o", "ST"), bwd: ("dq", "dk", "dv", "dS0")}
    inputs = {fwd: ("q", "k", "v", "g", "lengths"), bwd: ("q", "k", "v", "do", "g", "lengths")}
    for call in (fwd, bwd):
        base = {**FWD, "do": 0x40000, "dq": 0x90000, "dk": 0xa0000, "dv": 0xb0000, "dST": 0x80000, "dS0": 0xc0000}
        for out in outputs[call]:
            for name in inputs[call] + ("S0",):
                if not (out == "ST" and name == "S0"):
                    assert call(lib, **{out: base[name]}) == BAD, (out, name)
            assert call(lib, **{out: base["S0"] + 4}) == BAD
            for other in outputs[call]:
                if other != out:
                    assert call(lib, **{out: base[other]}) == BAD, (out, other)
    assert fwd(lib, o=None) == BAD and bwd(lib, dk=None) == BAD
    assert bwd(lib, dq=0x80000) == BAD                          # dST
    assert fwd(lib, strides={"o": s3(0, 0, 8)}) == BAD          # two heads of o in one place
    for kw in (dict(q=None), dict(g=None), dict(state=None), dict(new=None), dict(o=0x10000), dict(o=0x70000),
               dict(new=0x70004), dict(new=0x10000), dict(new=0x50000), dict(o=0x50000), dict(d=0), dict(dt=7),
               dict(q=0x10002), dict(scale=NAN)):
        assert step(lib, **kw) == BAD, kw
    assert step(lib, d=129) == UNSUPPORTED and step(lib, B=1 << 10, H=1 << 10) == UNSUPPORTED


@no_gpu
def test_calls_that_pass_reach_the_launch(lib):  # noqa: F811
    assert fwd(lib) == LAUNCHED and bwd(lib) == LAUNCHED and step(lib) == LAUNCHED
    assert fwd(lib, ST=None, S0=None, lengths=None) == LAUNCHED
    assert fwd(lib, ST=0x70000) == LAUNCHED                     # ST in the place of S0
    assert bwd(lib, dS0=0x80000) == LAUNCHED                    # dS0 in the place of dST
    assert bwd(lib, dS0=None, dST=None, S0=None, lengths=None) == LAUNCHED
    assert fwd(lib, strides={"k": s3(0, 0, 8), "v": s3(0, 0, 0)}) == LAUNCHED       # broadcast inputs
    assert step(lib, new=0x90000) == LAUNCHED
    assert step(lib, s=(ctypes.c_int64 * 2)(100, 10)) == LAUNCHED
    assert step(lib, s=(ctypes.c_int64 * 2)(100, -10)) == BAD


def test_decay_attention_workspace(lib):  # noqa: F811
    size = favor.decay_attention_workspace_bytes
    assert size(1, 2, 8, 8, torch.float32) == 0                 # one segment: none
    n = size(1, 2, 30000, 64, torch.bfloat16)
    assert n > 0 and n % (64 * 64 * 4) == 0 and size(1, 2, 30000, 64, torch.bfloat16, True) > 0
    assert lib.favor_decay_attention_workspace_bytes(1, 2, 30000, 129, 0, 0) == 0
    assert lib.favor_decay_attention_workspace_bytes(0, 2, 30000, 64, 0, 0) == 0
    for bad in [(0, 1, 1, 1, torch.float32), (1, 1, 1 << 31, 1, torch.float32), (1, 1, 8, 8, torch.float16)]:
        with pytest.raises(favor.FavorError):
            size(*bad)
    big = dict(L=30000, d=64, q=1 << 30, k=2 << 30, v=3 << 30, o=4 << 30, ST=5 << 30, S0=6 << 30, ws=7 << 30,
               n=favor.decay_attention_workspace_bytes(1, 2, 30000, 64, torch.float32))
    assert fwd(lib, **{**big, "ws": None}) == BAD
    assert fwd(lib, **{**big, "ws": (7 << 30) + 128}) == BAD    # not on 256 bytes
    assert fwd(lib, **{**big, "n": big["n"] - 1}) == BAD
    for name in ("q", "k", "v", "o", "S0", "ST", "g", "lengths"):
        at = {**FWD, **big}[name]
        assert fwd(lib, **{**big, "ws": at - at % 256}) == BAD, name


QK = dict(q=0x10000, qo=0x20000, k=0x30000, ko=0x40000, wq=0x50000, wk=0x60000, eps=1e-5, B=1, Hq=2, Hk=1, L=8, d=8,
          pos=0x70000, pB=1, sections=(1, 2), table=0x80000, pairing=0, dt=0, dqo=0x90000, dko=0xa0000, dq=0xb0000,
          dk=0xc0000, dwq=0xd0000, dwk=0xe0000, ws=0x100000, n=1 << 30)


def qk(lib, back=False, **kw):
    a = {**QK, **kw}
    sec = (ctypes.c_int * len(a["sections"]))(*a["sections"]) if a["sections"] is not None else None
    n = a.get("axes", len(a["sections"] or (1,)))
    turns = (a["eps"], a["B"], a["Hq"], a["Hk"], a["L"], a["d"], a["pos"], a["pB"], n, sec, a["table"], a["pairing"],
             a["dt"])
    if not back:
        return lib.favor_fwd_qk_norm_rotary(a["q"], None, a["qo"], None, a["k"], None, a["ko"], None, a["wq"], a["wk"],
                                            *turns, None)
    return lib.favor_bwd_qk_norm_rotary(a["q"], None, a["dqo"], None, a["dq"], None, a["k"], None, a["dko"], None,
                                        a["dk"], None, a["wq"], a["wk"], a["dwq"], a["dwk"], *turns, a["ws"], a["n"],
                                        None)


def test_qk_norm_refusals(lib):  # noqa: F811
    for back in (False, True):
        def call(**kw):
            return qk(lib, back, **kw)
        for name in ("B", "Hq", "L", "d"):
            assert call(**{name: 0}) == BAD
        assert call(Hk=0) == BAD
        for kw in (dict(dt=2), dict(eps=0.0), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(pairing=2),
                   dict(sections=None), dict(sections=(0,)), dict(sections=(5,)), dict(sections=(-1, 2)),
                   dict(axes=0), dict(axes=5), dict(pB=3), dict(pos=None), dict(table=None), dict(table=0x80004),
                   dict(q=None), dict(q=0x10002), dict(wq=0x50002), dict(k=None)):
            assert call(**kw) == BAD, kw
        assert call(d=513, sections=(2,)) == UNSUPPORTED
        assert call(B=1 << 16, Hq=1 << 15) == UNSUPPORTED
    # outputs on what is read, or on one another
    for out, ok in (("qo", "q"), ("ko", "k")):
        for name in ("q", "k", "wq", "wk", "pos", "table", "qo", "ko"):
            if name not in (out, ok):
                assert qk(lib, **{out: QK[name]}) == BAD, (out, name)
        assert qk(lib, **{out: QK[ok] + 4}) == BAD
    for out, ok in (("dq", ("q", "dqo")), ("dk", ("k", "dko")), ("dwq", ()), ("dwk", ())):
        for name in ("q", "k", "dqo", "dko", "wq", "wk", "pos", "table", "dq", "dk", "dwq", "dwk", "ws"):
            if name != out and name not in ok:
                assert qk(lib, True, **{out: QK[name]}) == BAD, (out, name)
    for kw in (dict(ws=None), dict(ws=0x100080), dict(n=16), dict(dq=None), dict(dqo=None), dict(dko=None),
               dict(dk=None), dict(dwq=0xd0002)):
        assert qk(lib, True, **kw) == BAD, kw


@no_gpu
def test_qk_norm_calls_that_pass_reach_the_launch(lib):  # noqa: F811
    assert qk(lib) == LAUNCHED and qk(lib, True) == LAUNCHED
    none = dict(k=None, ko=None, wk=None)
    assert qk(lib, **none) == LAUNCHED and qk(lib, wq=None, wk=None) == LAUNCHED
    assert qk(lib, qo=QK["q"], ko=QK["k"]) == LAUNCHED
    assert qk(lib, True, dq=QK["q"], dk=QK["dko"]) == LAUNCHED
    assert qk(lib, True, k=None, dko=None, dk=None, wk=None, dwk=None) == LAUNCHED
    assert qk(lib, True, dwq=None, dwk=None, ws=None, n=0) == LAUNCHED
    assert qk(lib, True, dwq=None) == LAUNCHED


def test_qk_norm_workspace(lib):  # noqa: F811
    size = favor.bwd_qk_norm_rotary_workspace_bytes
    assert size(1, 2, 0, 8, 8, torch.float32) > 0
    for bad in [(0, 1, 1, 1, 8), (1, 1, -1, 1, 8), (1, 1, 1, 1, 513), (1, 1, 1 << 31, 1, 8), (1 << 16, 1 << 15, 1, 1, 8)]:
        with pytest.raises(favor.FavorError):
            size(*bad, torch.float32)


def test_binding_refuses_cpu_tensors_and_odd_arguments():
    x = torch.zeros(1, 2, 8, 16)
    g = torch.zeros(2)
    s = torch.zeros(1, 2, 16, 16)
    pos = torch.zeros((1, 1, 8), dtype=torch.int32)
    table = favor.new_rotary_table((8,), device="cpu")
    for call in [lambda: favor.fwd_decay_attention(x, x, x, g), lambda: favor.bwd_decay_attention(x, x, x, g, x),
                 lambda: favor.decay_attention_step(x[:, :, 0], x[:, :, 0], x[:, :, 0], g, s),
                 lambda: favor.fwd_qk_norm_rotary(x, x, None, None, pos, table, (8,)),
                 lambda: favor.bwd_qk_norm_rotary(x, x, x, x, None, None, pos, table, (8,))]:
        with pytest.raises(favor.FavorError, match="CUDA tensor"):
            call()
