"""Argument checks of the sequence operators that need no GPU: the C ABI
refuses before anything is launched.  A call that passes every check reaches
the launch, which on a machine without a GPU is status 3; the tests that rely
on that use addresses that are never followed and skip where a GPU is."""

import ctypes
import os
import random
import re
from fractions import Fraction

import numpy as np
import pytest
import torch

import linear_softmax_attention_gb300 as favor
from test_abi_cpu import lib  # noqa: F401  (the built library)

BAD, UNSUPPORTED, LAUNCHED = 1, 2, 3
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="addresses of this test are not memory")


def s3(*s):
    return (ctypes.c_int64 * 3)(*s)


def scan(lib, **kw):
    a = dict(x=0x1000, xs=None, g=0x2000, gs=None, h=0x3000, hs=None, h0=0x4000, hT=0x5000, B=1, H=2, L=8, d=8, dt=0)
    a.update(kw)
    return lib.favor_fwd_gated_scan(a["x"], a["xs"], a["g"], a["gs"], a["h"], a["hs"], a["h0"], a["hT"], a["B"],
                                    a["H"], a["L"], a["d"], a["dt"], None, None)


def scan_bwd(lib, **kw):
    a = dict(g=0x1000, h=0x2000, dh=0x3000, dx=0x4000, dg=0x5000, h0=0x6000, dhT=0x7000, dh0=0x8000, B=1, H=2, L=8,
             d=8, dt=0, s=None)
    a.update(kw)
    return lib.favor_bwd_gated_scan(a["g"], None, a["h"], None, a["dh"], None, a["dx"], a["s"], a["dg"], None,
                                    a["h0"], a["dhT"], a["dh0"], a["B"], a["H"], a["L"], a["d"], a["dt"], None, None)


def step(lib, **kw):
    a = dict(x=0x1000, g=0x2000, h=0x3000, state=0x4000, new=0x4000, B=1, H=2, d=8, dt=0)
    a.update(kw)
    return lib.favor_gated_scan_step(a["x"], a["g"], a["h"], a["state"], a["new"], a["B"], a["H"], a["d"], a["dt"],
                                     None)


def norm(lib, **kw):
    a = dict(x=0x10000, xs=None, y=0x20000, ys=None, gamma=0x30000, beta=0x40000, eps=1e-5, B=1, H=2, L=8, d=8, dt=0)
    a.update(kw)
    return lib.favor_fwd_layer_norm(a["x"], a["xs"], a["y"], a["ys"], a["gamma"], a["beta"], a["eps"], a["B"],
                                    a["H"], a["L"], a["d"], a["dt"], None)


def norm_bwd(lib, **kw):
    a = dict(x=0x1000, dy=0x2000, dx=0x3000, gamma=0x4000, dgamma=0x5000, dbeta=0x6000, eps=1e-5, B=1, H=2, L=8, d=8,
             dt=0, ws=0x100000, nbytes=1 << 30)
    a.update(kw)
    return lib.favor_bwd_layer_norm(a["x"], None, a["dy"], None, a["dx"], None, a["gamma"], a["dgamma"], a["dbeta"],
                                    a["eps"], a["B"], a["H"], a["L"], a["d"], a["dt"], a["ws"], a["nbytes"], None)


def rotary(lib, name="favor_fwd_rotary", **kw):
    a = dict(q=0x1000, qs=None, qo=0x2000, qos=None, k=0x3000, ks=None, ko=0x4000, kos=None, B=1, Hq=2, Hk=1, L=8,
             d=8, pos=0x5000, pB=1, sections=(1, 2), table=0x6000, pairing=0, dt=0)
    a.update(kw)
    n = len(a["sections"]) if a["sections"] is not None else 1
    sec = (ctypes.c_int * n)(*a["sections"]) if a["sections"] is not None else None
    return getattr(lib, name)(a["q"], a["qs"], a["qo"], a["qos"], a["k"], a["ks"], a["ko"], a["kos"], a["B"], a["Hq"],
                              a["Hk"], a["L"], a["d"], a["pos"], a["pB"], a.get("n", n), sec, a["table"],
                              a["pairing"], a["dt"], None)


def test_gated_scan_refusals(lib):  # noqa: F811
    for call in (scan, scan_bwd):
        for name in ("B", "H", "L", "d"):
            assert call(lib, **{name: 0}) == BAD
            assert call(lib, **{name: -3}) == BAD
        assert call(lib, dt=2) == BAD
        assert call(lib, g=None) == BAD
        assert call(lib, h=None) == BAD
        assert call(lib, g=0x1002) == BAD                   # not on an element
        assert call(lib, h0=0x6002) == BAD
        assert call(lib, B=1 << 20, H=1 << 10, d=2) == UNSUPPORTED
    # 2 heads x 8 tokens x 8 channels fp32: 512 bytes
    assert scan(lib, x=None) == BAD
    assert scan(lib, h=0x1004) == BAD                       # h runs into x
    assert scan(lib, h=0x2000 - 512 + 4) == BAD             # h runs into g
    assert scan(lib, hT=0x3000) == BAD                      # hT inside h
    assert scan(lib, hT=0x1000) == BAD
    assert scan(lib, h0=0x3000) == BAD
    assert scan(lib, hT=0x4004) == BAD                      # hT runs into h0
    assert scan(lib, hs=s3(0, 0, 8)) == BAD                 # two heads of h in one place
    assert scan(lib, hs=s3(0, 64, 7)) == BAD                # rows of h overlap
    assert scan(lib, hs=s3(0, 64, -8)) == BAD
    assert scan(lib, xs=s3(0, 64, -8)) == BAD
    assert scan(lib, xs=s3(0, 1 << 62, 8)) == BAD
    assert scan(lib, h=0x1000, hs=s3(0, 8, 16)) == BAD      # x in another order
    for name in ("dh", "dx", "dg"):
        assert scan_bwd(lib, **{name: None}) == BAD
    assert scan_bwd(lib, dx=0x2000) == BAD                  # dx may not be h
    assert scan_bwd(lib, dg=0x2000) == BAD
    assert scan_bwd(lib, dg=0x4000) == BAD                  # dx and dg
    assert scan_bwd(lib, dx=0x1000) == BAD                  # dx in the place of g
    assert scan_bwd(lib, dg=0x3000) == BAD
    assert scan_bwd(lib, dh0=0x6000) == BAD                 # dh0 in the place of h0
    assert scan_bwd(lib, s=s3(0, 0, 8)) == BAD
    for name in ("x", "g", "h", "state", "new"):
        assert step(lib, **{name: None}) == BAD
    assert step(lib, new=0x4004) == BAD
    assert step(lib, new=0x1000) == BAD
    assert step(lib, h=0x4000) == BAD
    assert step(lib, d=0) == BAD
    assert step(lib, dt=-1) == BAD
    assert step(lib, B=1 << 20, H=1 << 10, d=2) == UNSUPPORTED


def test_layer_norm_refusals(lib):  # noqa: F811
    for call in (norm, norm_bwd):
        for name in ("B", "H", "L", "d"):
            assert call(lib, **{name: 0}) == BAD
        assert call(lib, dt=9) == BAD
        assert call(lib, x=None) == BAD
        for eps in (0.0, -1e-5, float("nan"), float("inf")):
            assert call(lib, eps=eps) == BAD
        assert call(lib, gamma=0x4001) == BAD
        assert call(lib, d=16385) == UNSUPPORTED
        assert call(lib, B=1 << 16, H=1 << 8, L=1 << 8) == UNSUPPORTED
    assert norm(lib, y=None) == BAD
    assert norm(lib, y=0x10004) == BAD
    assert norm(lib, y=0x30000) == BAD                      # y over gamma
    assert norm_bwd(lib, dy=None) == BAD
    assert norm_bwd(lib, dx=None) == BAD
    assert norm_bwd(lib, dgamma=0x4000) == BAD              # over gamma
    assert norm_bwd(lib, dgamma=0x6000) == BAD              # dgamma and dbeta
    assert norm_bwd(lib, dbeta=0x3010) == BAD               # inside dx
    assert norm_bwd(lib, ws=None) == BAD
    assert norm_bwd(lib, ws=0x100080) == BAD
    assert norm_bwd(lib, nbytes=4) == BAD
    assert norm_bwd(lib, ws=0x1000) == BAD                  # the workspace over x
    ok = lib.favor_bwd_layer_norm_workspace_bytes
    assert ok(1, 1, 1000, 512, 1) > 0
    assert ok(0, 1, 1, 8, 0) == 0 and ok(1, 1, 1, 16385, 0) == 0 and ok(1, 1, 1, 8, 3) == 0
    assert ok(1 << 16, 1 << 8, 1 << 8, 8, 0) == 0


@pytest.mark.parametrize("name", ["favor_fwd_rotary", "favor_bwd_rotary"])
def test_rotary_refusals(lib, name):  # noqa: F811
    def call(**kw):
        return rotary(lib, name, **kw)

    for key in ("B", "Hq", "L", "d", "Hk"):
        assert call(**{key: 0}) == BAD
    for key in ("q", "qo", "k", "ko", "pos", "table", "sections"):
        assert call(**{key: None}) == BAD
    assert call(dt=2) == BAD
    assert call(pairing=2) == BAD
    assert call(n=0) == BAD
    assert call(sections=(1, 1, 1, 1, 0)) == BAD
    assert call(sections=(-1, 3)) == BAD
    assert call(sections=(0, 0)) == BAD
    assert call(sections=(3, 2)) == BAD                     # 10 channels of 8
    assert call(B=4, pB=2) == BAD
    assert call(pos=0x5002) == BAD
    assert call(table=0x6004) == BAD
    assert call(qo=0x1010) == BAD
    assert call(ko=0x2000) == BAD
    assert call(ko=0x1000) == BAD
    assert call(qo=0x3000) == BAD                           # q_out over k
    assert call(qo=0x5000) == BAD                           # over the positions
    assert call(qo=0x6000) == BAD                           # over the table
    assert call(d=20000) == UNSUPPORTED
    assert call(Hq=1 << 16, L=1 << 15) == UNSUPPORTED
    assert call(B=1, Hq=(1 << 31) - 9, L=1, k=None, ko=None, Hk=0) == UNSUPPORTED
    assert call(B=1, Hq=(1 << 31) - 19, L=1, Hk=4) == UNSUPPORTED


@no_gpu
def test_what_is_allowed_reaches_the_launch(lib):  # noqa: F811
    assert scan(lib) == LAUNCHED
    assert scan(lib, h0=None, hT=None) == LAUNCHED
    assert scan(lib, h=0x1000, hT=0x4000) == LAUNCHED       # in place, both
    assert scan(lib, h=0x2000) == LAUNCHED                  # the gates' place
    assert scan(lib, gs=s3(0, 0, 0)) == LAUNCHED            # a broadcast gate
    assert scan_bwd(lib) == LAUNCHED
    assert scan_bwd(lib, dx=0x3000, dg=0x1000, dh0=0x7000) == LAUNCHED
    assert step(lib) == LAUNCHED and step(lib, new=0x5000, h=0x1000) == LAUNCHED
    assert norm(lib) == LAUNCHED
    assert norm(lib, y=0x10000, gamma=None, beta=None) == LAUNCHED
    assert norm_bwd(lib) == LAUNCHED
    assert norm_bwd(lib, dgamma=None, dbeta=None, ws=None, nbytes=0) == LAUNCHED
    assert rotary(lib) == LAUNCHED
    assert rotary(lib, k=None, ko=None, Hk=0) == LAUNCHED
    assert rotary(lib, qo=0x1000, ko=0x3000) == LAUNCHED
    # queries and keys of one joint buffer [1, 8, 3, 2, 8] fp32, both in place
    s = s3(0, 8, 48)
    assert rotary(lib, q=0x1000, qs=s, qo=0x1000, qos=s, k=0x1040, ks=s, ko=0x1040, kos=s, Hk=2) == LAUNCHED
    assert rotary(lib, q=0x1000, qs=s, qo=0x1000, qos=s, k=0x1020, ks=s, ko=0x1020, kos=s, Hk=2) == BAD


def _elements(p, n, s, e):
    return {p + e * (i * s[0] + j * s[1] + k * s[2] + c) + w for i in range(n[0]) for j in range(n[1])
            for k in range(n[2]) for c in range(n[3]) for w in range(e)}


@no_gpu
def test_overlaps_against_the_sets_of_addresses(lib):  # noqa: F811
    # views of small buffers: what is let through never shares a byte, and
    # with the same strides nothing disjoint is refused
    rng = random.Random(4)
    seen = {BAD: 0, LAUNCHED: 0}
    for _ in range(3000):
        n = [rng.randint(1, 3) for _ in range(3)] + [rng.randint(1, 4)]
        order = [0, 1, 2]
        rng.shuffle(order)
        s, inner = [0, 0, 0], n[3] + rng.choice([0, 0, 3])
        for i in order:
            s[i] = inner
            inner = inner * n[i] + rng.choice([0, 0, 2])
        same = rng.random() < 0.7
        t = s if same else [n[1] * n[2] * n[3], n[2] * n[3], n[3]]
        at = 0x10000 + 4 * rng.randint(-40, 40)
        code = norm(lib, x=0x10000, xs=s3(*s), y=at, ys=s3(*t), gamma=None, beta=None, B=n[0], H=n[1], L=n[2], d=n[3])
        shared = bool(_elements(0x10000, n, s, 4) & _elements(at, n, t, 4))
        if at == 0x10000 and all(a == b or m == 1 for a, b, m in zip(s, t, n)):
            assert code == LAUNCHED
            continue
        seen[code] += 1
        assert code == BAD if shared else code in ((LAUNCHED,) if same else (LAUNCHED, BAD)), (n, s, t, at)
    assert min(seen.values()) > 300


def test_rotary_table():
    t = favor.new_rotary_table((2, 3), base=100.0, device="cpu")
    assert t.dtype == torch.int64 and tuple(t.shape) == (5,)
    turns = [100.0 ** (-j / n) / (2 * np.pi) for n in (2, 3) for j in range(n)]
    assert np.allclose(t.numpy() / 2.0 ** 64, turns, rtol=1e-15)
    # the same fraction of a turn, whole turns and negative ones
    f = [0.25 * np.pi, -0.25 * np.pi, 1.5 * np.pi, np.pi]
    t = favor.new_rotary_table((4,), freqs=f, device="cpu").numpy()
    assert np.allclose(t[:3] / 2.0 ** 64, [0.125, -0.125, -0.25], atol=1e-15)
    assert abs(t[3] / 2.0 ** 63) == pytest.approx(1.0)
    for bad in [dict(sections=()), dict(sections=(0,)), dict(sections=(-1, 4)), dict(sections=(1,) * 5),
                dict(sections=(2,), freqs=[1.0]), dict(sections=(1,), freqs=[float("inf")])]:
        with pytest.raises(favor.FavorError):
            favor.new_rotary_table(device="cpu", **bad)


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 2, 8, 16)
    pos = torch.zeros((1, 1, 8), dtype=torch.int32)
    table = favor.new_rotary_table((8,), device="cpu")
    for call in [lambda: favor.fwd_gated_scan(x, x), lambda: favor.bwd_gated_scan(x, x, x),
                 lambda: favor.gated_scan_step(x[:, :, 0].contiguous(), x[:, :, 0].contiguous(), x[:, :, 0]),
                 lambda: favor.fwd_layer_norm(x), lambda: favor.bwd_layer_norm(x, x),
                 lambda: favor.fwd_rotary(x, x, pos, table, (8,)), lambda: favor.bwd_rotary(x, None, pos, table, (8,))]:
        with pytest.raises(favor.FavorError, match="CUDA tensor"):
            call()


def test_scan_timeout_hook_refusals(lib):  # noqa: F811
    def call(x=0x1000, g=0x2000, h=0x3000, hT=0x5000, L=8, dt=0, cycles=0, status=0x6000):
        return lib.favor_selftest_scan_timeout(x, g, h, hT, 1, 2, L, 8, dt, cycles, -1, status, None)

    for bad in (dict(x=None), dict(g=None), dict(h=None), dict(status=None), dict(L=0), dict(dt=2), dict(cycles=-1),
                dict(cycles=2_200_000_001), dict(hT=0x3000)):
        assert call(**bad) == BAD


def test_waits_for_other_ctas_stores_acquire_at_cluster_scope():
    # st.async from another CTA releases at cluster scope: a wait of CTA scope would not order the reads behind it,
    # which no run shows
    csrc = os.path.join(os.path.dirname(favor.__file__), "csrc")
    scan = open(os.path.join(csrc, "scan.cu")).read()
    assert "st.async" in scan and re.findall(r"mbar_(?:try_|test_)?wait\w*\(", scan)
    assert set(re.findall(r"mbar_(?:try_|test_)?wait\w*", scan)) == {"mbar_try_wait_cluster"}
    fs = open(os.path.join(csrc, "tc_fs.cu")).read()
    assert set(re.findall(r"(mbar_\w*wait\w*)\(&land_(?:full|free)", fs)) == {"mbar_wait_cluster"}


def test_layer_norm_workspace_is_sized_on_the_tensors_device(monkeypatch):
    # devices of a process may differ in their number of SMs; a library and tensors that stand in for device 1,
    # while device 0 is current
    from linear_softmax_attention_gb300 import sequence

    class OnDevice1(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 1

    def tensor(*shape, dtype=torch.float32, device=None):
        return torch.zeros(shape[0] if len(shape) == 1 and isinstance(shape[0], tuple) else shape,
                           dtype=dtype).as_subclass(OnDevice1)

    current, seen = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.before

    class Library:
        def favor_bwd_layer_norm_workspace_bytes(self, *_):
            seen.append(("size", current[0]))
            return 4096 if current[0] == 1 else 256

        def favor_bwd_layer_norm(self, *args):
            seen.append(("call", current[0], args[-2]))
            return 0

    monkeypatch.setattr(sequence, "load", Library)
    monkeypatch.setattr(sequence, "_current_device", lambda: current[0])
    monkeypatch.setattr(sequence, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch, "empty", tensor)
    x = tensor(1, 2, 8, 16)
    favor.bwd_layer_norm(x, x)
    assert seen == [("size", 1), ("call", 1, 4096)] and current == [0]
    assert favor.bwd_layer_norm_workspace_bytes(1, 2, 8, 16, torch.float32) == 256
    assert favor.bwd_layer_norm_workspace_bytes(1, 2, 8, 16, torch.float32, device=1) == 4096


def test_rotary_table_words_are_exact():
    pi = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    freqs = [1.0, 0.1, 1e-4, 1e-30, -7.5, np.pi, 123456.789, 1e30]
    want = [round(Fraction(f) / (2 * pi) * 2 ** 64) % 2 ** 64 for f in freqs]
    table = favor.new_rotary_table((len(freqs),), freqs=freqs, device="cpu")
    assert [w % 2 ** 64 for w in table.tolist()] == want
    assert favor.new_rotary_table((2,), freqs=[1.7e308, 5e-324], device="cpu").shape == (2,)


@pytest.mark.parametrize("base", [0.0, -10000.0, float("nan"), float("inf"), 5e-324])
def test_rotary_table_refuses_bases_without_frequencies(base):
    with pytest.raises(favor.FavorError):
        favor.new_rotary_table((64,), base=base, device="cpu")
