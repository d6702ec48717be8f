"""Cases of two operators that a layer has around and beside the FAVOR+ attention.

  decay   causal linear attention whose memory fades, with one decay per head,
            o_t = scale sum_{s <= t} exp((t - s) g) (q_t . k_s) v_s + scale exp((t + 1) g) q_t S0,
          over the tokens of [B, H, L, d]: whole sequences ("fwd"), their gradients ("bwd")
          and one token from the carried state ("step")
  qknorm  root-mean-square norm of each head's queries and keys, with weights, and their
          rotation by positions, in one pass ("fwd", its gradients "bwd")

With ``own`` false the operators run in their plain form (elementary torch
operations in 32 bits, angles in 64), with ``own`` true through the
framework's entry points.
"""

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
BASE = 10000.0
CHUNK = 128          # tokens that the plain form of the decayed attention takes together
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one new token for each of 256 sequences of 8 heads (the decode workload's sizes)
        {"name": "decay-step-bf16", "op": "decay", "dir": "step", "dtype": "bf16", "B": 256, "H": 8, "L": 1, "d": 64,
         "state": True, "ragged": False, "tokens": False},
        # a short prompt of a few sequences of unlike lengths, states kept for the tokens to come
        {"name": "decay-fwd-bf16-prompt", "op": "decay", "dir": "fwd", "dtype": "bf16", "B": 4, "H": 8, "L": 333,
         "d": 64, "state": True, "ragged": True, "tokens": True},
        # training: 8 x 4096 tokens, 8 heads of 64
        {"name": "decay-fwd-bf16", "op": "decay", "dir": "fwd", "dtype": "bf16", "B": 8, "H": 8, "L": 4096, "d": 64,
         "state": False, "ragged": False, "tokens": False},
        # one long sequence, 16 heads of 128, out of the projection's token-major output
        {"name": "decay-fwd-bf16-long", "op": "decay", "dir": "fwd", "dtype": "bf16", "B": 1, "H": 16, "L": 65536,
         "d": 128, "state": True, "ragged": False, "tokens": True},
        # an odd batch in 32 bits
        {"name": "decay-fwd-f32-odd", "op": "decay", "dir": "fwd", "dtype": "f32", "B": 3, "H": 5, "L": 1777, "d": 40,
         "state": True, "ragged": True, "tokens": False},
        # training on images as sequences: 2 x 12288 pixels, gradients
        {"name": "decay-bwd-bf16", "op": "decay", "dir": "bwd", "dtype": "bf16", "B": 2, "H": 8, "L": 12288, "d": 64,
         "state": False, "ragged": False, "tokens": False},
        # gradients in 32 bits, sequences of unlike lengths
        {"name": "decay-bwd-f32", "op": "decay", "dir": "bwd", "dtype": "f32", "B": 2, "H": 4, "L": 2048, "d": 64,
         "state": True, "ragged": True, "tokens": True},
        # one new token of 256 sequences at far positions
        {"name": "qknorm-step-bf16", "op": "qknorm", "dir": "fwd", "dtype": "bf16", "B": 256, "H": 8, "Hk": 8, "L": 1,
         "d": 64, "axes": 1, "rot": 64, "halves": True, "tokens": False},
        # the queries and keys of one long sequence, read out of the joint projection's output
        {"name": "qknorm-fwd-bf16-long", "op": "qknorm", "dir": "fwd", "dtype": "bf16", "B": 1, "H": 16, "Hk": 16,
         "L": 65536, "d": 128, "axes": 1, "rot": 128, "halves": True, "tokens": True},
        # images: rows and columns of 96 x 128 pixels
        {"name": "qknorm-fwd-f32-image", "op": "qknorm", "dir": "fwd", "dtype": "f32", "B": 2, "H": 8, "Hk": 8,
         "L": 12288, "d": 64, "axes": 2, "rot": 64, "halves": False, "tokens": False},
        # video: time, height and width; gradients, with fewer key heads
        {"name": "qknorm-bwd-bf16-video", "op": "qknorm", "dir": "bwd", "dtype": "bf16", "B": 1, "H": 16, "Hk": 4,
         "L": 65536, "d": 128, "axes": 3, "rot": 128, "halves": True, "tokens": True},
        # gradients at an odd width in 32 bits, some channels without a position
        {"name": "qknorm-bwd-f32-odd", "op": "qknorm", "dir": "bwd", "dtype": "f32", "B": 3, "H": 5, "Hk": 5,
         "L": 1111, "d": 90, "axes": 2, "rot": 60, "halves": False, "tokens": False},
    ]


def _spread(rng, low, high):
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op, direction = rng.choice([("decay", "step"), ("decay", "fwd"), ("decay", "fwd"), ("decay", "fwd"),
                                ("decay", "bwd"), ("decay", "bwd"), ("qknorm", "fwd"), ("qknorm", "fwd"),
                                ("qknorm", "bwd"), ("qknorm", "bwd")])
    case = {"op": op, "dir": direction, "dtype": rng.choice(["f32", "bf16", "bf16"]), "tokens": rng.random() < 0.5}
    case["H"] = _spread(rng, 1, 16)
    if op == "decay":
        case["B"] = _spread(rng, 1, 300) if direction == "step" else _spread(rng, 1, 8)
        case["d"] = rng.choice([16, 32, 40, 64, 64, 64, 80, 96, 128, 128, rng.randint(1, 128)])
        case["L"] = 1 if direction == "step" else _spread(rng, 2, 65536)
        case["state"] = direction == "step" or rng.random() < 0.5
        case["ragged"] = direction != "step" and rng.random() < 0.3
        case["tokens"] = case["tokens"] and direction != "step"
        most = 1 << (25 if direction == "bwd" else 26)
    else:
        case["axes"] = rng.choice([1, 1, 2, 3])
        case["d"] = rng.choice([32, 64, 64, 96, 128, 128, 256, 2 * rng.randint(8, 64)])
        case["rot"] = case["d"] if rng.random() < 0.7 else 2 * rng.randint(case["axes"], case["d"] // 2)
        case["B"] = _spread(rng, 1, 64)
        case["Hk"] = max(1, case["H"] // rng.choice([1, 1, 2, 4]))
        case["L"] = 1 if rng.random() < 0.2 else _spread(rng, 2, 65536)
        case["halves"] = rng.random() < 0.5
        most = 1 << 26
    case["L"] = max(1, min(case["L"], most // (case["B"] * case["H"] * case["d"])))
    return case


# --- inputs -------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)


def _heads(case, t, part=None):
    """Values [B, H, L, d] in the case's type; with "tokens" as a view of a
    [B, L, H, d] buffer (`part`: one of the three parts of a [B, L, 3, H, d] one)."""
    t = t.to(_TYPES[case["dtype"]])
    if not case["tokens"]:
        return t.contiguous()
    B, H, L, d = t.shape
    if part is None:
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    joint = torch.zeros((B, L, 3, H, d), device=DEV, dtype=t.dtype)
    joint[:, :, part] = t.transpose(1, 2)
    return joint[:, :, part].transpose(1, 2)


def _lengths(case):
    """Tokens of each sequence: all of them, or between about half and all."""
    B, L = case["B"], case["L"]
    if not case["ragged"]:
        return None
    return [max(1, L - b * L // (2 * B)) for b in range(B)]


def _decays(case, gen):
    """Logarithms of the decays, one per head: memories of about two tokens to
    some thousands."""
    H = case["H"]
    at = (torch.arange(H, device=DEV) + torch.rand(H, generator=gen, device=DEV)) / H
    return -torch.exp(math.log(0.5) - at * 7.0)


def _sections(case):
    """Pairs of each axis: an even share, what is left over to the last."""
    pairs, axes = case["rot"] // 2, case["axes"]
    share = max(1, pairs // axes)
    return tuple([share] * (axes - 1) + [pairs - share * (axes - 1)])


def _frequencies(case):
    """Radians per unit of position for each pair (float64), and each pair's axis."""
    sections = _sections(case)
    freq = torch.cat([BASE ** (-torch.arange(n, dtype=torch.float64) / n) for n in sections])
    axis = torch.cat([torch.full((n,), i, dtype=torch.int64) for i, n in enumerate(sections)])
    return freq, axis


def _positions(case, gen):
    B, L, axes = case["B"], case["L"], case["axes"]
    if L == 1:                                   # one token of each sequence, each at its own position
        return torch.randint(0, 1000000, (axes, B, 1), generator=gen, device=DEV, dtype=torch.int32)
    t = torch.arange(L, device=DEV, dtype=torch.int32)
    start = int(torch.randint(0, 5000, (1,), generator=gen, device=DEV))
    if axes == 1:
        grid = (t + start,)
    elif axes == 2:
        grid = (t // 128, t % 128)
    else:
        grid = (t // 1024 + start, t // 32 % 32, t % 32)
    return torch.stack(grid).reshape(axes, 1, L).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    B, H, L, d = (case[k] for k in "BHLd")
    st = {"case": case}
    if case["op"] == "decay":
        st["g"] = _decays(case, gen)
        st["scale"] = d ** -0.5
        # the state of the tokens before: about as large as its decay lets it grow
        grown = (1 - torch.exp(2 * st["g"])).rsqrt().view(1, H, 1, 1)
        st["s0"] = _normal(gen, B, H, d, d) * grown if case["state"] else None
        for i, n in enumerate("qkv"):
            st[n] = _heads(case, _normal(gen, B, H, L, d), part=i)
        if case["dir"] == "step":
            for n in "qkv":
                st[n] = st[n].reshape(B, H, d).contiguous()
            st["next"] = torch.empty_like(st["s0"])
            return st
        lengths = _lengths(case)
        st["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
        if case["dir"] == "bwd":
            st["do"] = _heads(case, _normal(gen, B, H, L, d))
            st["dlast"] = _normal(gen, B, H, d, d) if case["state"] else None
        return st
    for i, n, heads in ((0, "q", H), (1, "k", case["Hk"])):
        x = _normal(gen, B, heads, L, d) * (0.5 + 2 * torch.rand((B, heads, L, 1), generator=gen, device=DEV))
        st[n] = _heads(case, x, part=i if heads > 1 else None)
        st["w" + n] = 1 + 0.2 * _normal(gen, d)
        if case["dir"] == "bwd":
            st["d" + n] = _heads(case, _normal(gen, B, heads, L, d))
    st["pos"] = _positions(case, gen)
    freq, axis = _frequencies(case)
    # what a turn is in the framework's table: 2^64
    st["table"] = torch.round(freq / (2 * math.pi) * 2.0 ** 64).to(torch.int64).to(DEV)
    st["freq"], st["axis"] = freq.to(DEV), axis.to(DEV)
    st["sections"] = _sections(case)
    return st


# --- plain forms ----------------------------------------------------------------

def _chunked(t, n):
    """[B, H, L, d] -> fp32 [B, H, n, CHUNK, d], zeros behind the last token."""
    B, H, L, d = t.shape
    out = torch.zeros((B, H, n * CHUNK, d), device=t.device, dtype=torch.float32)
    out[:, :, :L] = t
    return out.view(B, H, n, CHUNK, d)


def _plain_decay(st):
    case = st["case"]
    t = _TYPES[case["dtype"]]
    B, H, L, d = (case[k] for k in "BHLd")
    g, scale = st["g"], st["scale"]
    if case["dir"] == "step":
        q, k, v = (st[n].float() for n in "qkv")
        s = torch.exp(g).view(1, H, 1, 1) * st["s0"] + k.unsqueeze(-1) * v.unsqueeze(-2)
        return {"o": (scale * (q.unsqueeze(-1) * s).sum(-2)).to(t), "state": s}
    n = -(-L // CHUNK)
    i = torch.arange(CHUNK, device=DEV)
    lengths = st["lengths"] if st["lengths"] is not None else torch.full((B,), L, device=DEV, dtype=torch.int32)
    # tokens of each chunk, [B, 1, n, 1]
    have = (lengths.view(B, 1) - CHUNK * torch.arange(n, device=DEV).view(1, n)).clamp(0, CHUNK).view(B, 1, n, 1)
    real = (i < have).unsqueeze(-1)                                                    # [B, 1, n, CHUNK, 1]
    gh = g.view(1, H, 1, 1)
    apart = (i.view(-1, 1) - i.view(1, -1)).float()
    fade = torch.where(apart >= 0, torch.exp(g.view(H, 1, 1) * apart.clamp(min=0)), 0.0).view(1, H, 1, CHUNK, CHUNK)
    since = torch.exp(gh * (i + 1).float()).unsqueeze(-1)                              # from the chunk's start
    until = torch.exp(gh * (have - 1 - i).clamp(min=0).float()).unsqueeze(-1) * real   # to its last token
    whole = torch.exp(gh * have.float()).unsqueeze(-1)                                 # [B, H, n, 1, 1]
    q, k, v = (torch.where(real, _chunked(st[x], n), 0.0) for x in "qkv")
    gain = torch.matmul((k * until).transpose(-1, -2), v)
    s = st["s0"] if st["s0"] is not None else torch.zeros((B, H, d, d), device=DEV)
    starts = []
    for c in range(n):
        starts.append(s)
        s = whole[:, :, c] * s + gain[:, :, c]
    start = torch.stack(starts, 2)

    def rows(x):
        return x.view(B, H, n * CHUNK, d)[:, :, :L].to(t).contiguous()

    if case["dir"] == "fwd":
        o = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * fade, v) + since * torch.matmul(q, start)
        return {"o": rows(torch.where(real, scale * o, 0.0)), "last": s}
    do = torch.where(real, _chunked(st["do"], n), 0.0) * scale
    gain = torch.matmul((q * since).transpose(-1, -2), do)
    r = st["dlast"] if st["dlast"] is not None else torch.zeros((B, H, d, d), device=DEV)
    ends = []
    for c in reversed(range(n)):
        ends.append(r)
        r = whole[:, :, c] * r + gain[:, :, c]
    end = torch.stack(ends[::-1], 2)
    m = torch.matmul(do, v.transpose(-1, -2)) * fade
    dq = torch.matmul(m, k) + since * torch.matmul(do, start.transpose(-1, -2))
    dk = torch.matmul(m.transpose(-1, -2), q) + until * torch.matmul(v, end.transpose(-1, -2))
    m = torch.matmul(q, k.transpose(-1, -2)) * fade
    dv = torch.matmul(m.transpose(-1, -2), do) + until * torch.matmul(k, end)
    return {"dq": rows(dq), "dk": rows(dk), "dv": rows(dv), "ds0": r}


def _turn(x, cos, sin, rot, halves):
    """The first `rot` channels of x (32 bits) as pairs turned by the angles."""
    u = x[..., :rot]
    a, b = (u[..., : rot // 2], u[..., rot // 2:]) if halves else (u[..., 0::2], u[..., 1::2])
    a, b = a * cos - b * sin, a * sin + b * cos
    u = torch.cat([a, b], -1) if halves else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([u, x[..., rot:]], -1)


def _plain_qknorm(st):
    case = st["case"]
    t = _TYPES[case["dtype"]]
    angle = (st["pos"][st["axis"]].permute(1, 2, 0).double() * st["freq"]).unsqueeze(1)      # [B or 1, 1, L, pairs]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    out = {}
    for n in ("q", "k"):
        x, w = st[n].float(), st["w" + n]
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        x = x * r
        if case["dir"] == "fwd":
            out[n] = _turn(x * w, cos, sin, case["rot"], case["halves"]).to(t).contiguous()
            continue
        dn = _turn(st["d" + n].float(), cos, -sin, case["rot"], case["halves"])
        dx = dn * w
        dx = r * (dx - x * (dx * x).mean(-1, keepdim=True))
        out["d" + n], out["dw" + n] = dx.to(t).contiguous(), (dn * x).sum((0, 1, 2))
    return out


# --- one pass -------------------------------------------------------------------

def run(state):
    st, case = state, state["case"]
    if not own:
        return {"decay": _plain_decay, "qknorm": _plain_qknorm}[case["op"]](st)
    import linear_softmax_attention_gb300 as favor

    if case["op"] == "decay":
        if case["dir"] == "step":
            o, new = favor.decay_attention_step(st["q"], st["k"], st["v"], st["g"], st["s0"], scale=st["scale"],
                                                new_state=st["next"])
            return {"o": o, "state": new}
        if case["dir"] == "fwd":
            o, last = favor.fwd_decay_attention(st["q"], st["k"], st["v"], st["g"], scale=st["scale"], S0=st["s0"],
                                                lengths=st["lengths"])
            return {"o": o, "last": last}
        dq, dk, dv, ds0 = favor.bwd_decay_attention(st["q"], st["k"], st["v"], st["g"], st["do"], scale=st["scale"],
                                                    S0=st["s0"], dST=st["dlast"], lengths=st["lengths"])
        return {"dq": dq, "dk": dk, "dv": dv, "ds0": ds0}
    pairing = "halves" if case["halves"] else "adjacent"
    if case["dir"] == "fwd":
        q, k = favor.fwd_qk_norm_rotary(st["q"], st["k"], st["wq"], st["wk"], st["pos"], st["table"], st["sections"],
                                        pairing=pairing, eps=EPS)
        return {"q": q, "k": k}
    dq, dk, dwq, dwk = favor.bwd_qk_norm_rotary(st["q"], st["k"], st["dq"], st["dk"], st["wq"], st["wk"], st["pos"],
                                                st["table"], st["sections"], pairing=pairing, eps=EPS)
    return {"dq": dq, "dwq": dwq, "dk": dk, "dwk": dwk}


def work(case):
    size = {"f32": 4, "bf16": 2}[case["dtype"]]
    B, H, L, d = (case[k] for k in "BHLd")
    n = B * H * L * d
    if case["op"] == "decay":
        state = 4 * B * H * d * d
        lengths = _lengths(case)
        real = n if lengths is None else H * d * sum(lengths)        # tokens that are read; all rows are written
        if case["dir"] == "bwd":     # q, k, v, do in; dq, dk, dv and ds0 out
            return {"bytes": (4 * real + 3 * n) * size + state * (3 if case["state"] else 1) + 4 * H,
                    "flops": 10 * real * d}
        return {"bytes": (3 * real + n) * size + state * (2 if case["state"] else 1) + 4 * H, "flops": 4 * real * d}
    n += B * case["Hk"] * L * d
    positions = case["axes"] * (B if L == 1 else 1) * L
    rest = 4 * positions + 4 * case["rot"] + 8 * d
    if case["dir"] == "bwd":         # the rows and their gradients in, the rows' and the weights' gradients out
        return {"bytes": 3 * n * size + rest + 8 * d, "flops": 13 * n}
    return {"bytes": 2 * n * size + rest, "flops": 7 * n}


# --- the definitions in 64 bits ---------------------------------------------------

def _exact_decay(case, st):
    B, H, L, d = (case[k] for k in "BHLd")
    a, scale = torch.exp(st["g"].double()).view(1, H, 1, 1), st["scale"]
    s = st["s0"].double().clone() if st["s0"] is not None else torch.zeros((B, H, d, d), device=DEV,
                                                                          dtype=torch.float64)
    if case["dir"] == "step":
        q, k, v = (st[n].double() for n in "qkv")
        s = a * s + torch.einsum("bhi,bhj->bhij", k, v)
        return {"o": scale * torch.einsum("bhi,bhij->bhj", q, s), "state": s}
    ends = _lengths(case) or [L] * B
    q, k, v = (st[n].permute(2, 0, 1, 3).double() for n in "qkv")       # [L, B, H, d]

    def at(t):           # the sequences that have a token t come first: their number
        return sum(1 for e in ends if e > t)

    assert ends == sorted(ends, reverse=True)
    o = torch.zeros_like(q)
    if case["dir"] == "fwd":
        for t in range(L):
            b = at(t)
            if b == 0:
                break
            s[:b] = a * s[:b] + k[t, :b].unsqueeze(-1) * v[t, :b].unsqueeze(-2)
            o[t, :b] = scale * torch.matmul(q[t, :b].unsqueeze(-2), s[:b]).squeeze(-2)
        return {"o": o.permute(1, 2, 0, 3), "last": s}
    do = st["do"].permute(2, 0, 1, 3).double()
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    for t in range(L):                                   # o_t = scale S_t^T q_t
        b = at(t)
        if b == 0:
            break
        s[:b] = a * s[:b] + k[t, :b].unsqueeze(-1) * v[t, :b].unsqueeze(-2)
        o[t, :b] = scale * torch.matmul(s[:b], do[t, :b].unsqueeze(-1)).squeeze(-1)
    r = st["dlast"].double().clone() if st["dlast"] is not None else torch.zeros_like(s)
    for t in reversed(range(L)):                         # r: what reaches S_t
        b = at(t)
        if b == 0:
            continue
        r[:b] += scale * q[t, :b].unsqueeze(-1) * do[t, :b].unsqueeze(-2)
        dk[t, :b] = torch.matmul(r[:b], v[t, :b].unsqueeze(-1)).squeeze(-1)
        dv[t, :b] = torch.matmul(k[t, :b].unsqueeze(-2), r[:b]).squeeze(-2)
        r[:b] *= a
    return {"dq": o.permute(1, 2, 0, 3), "dk": dk.permute(1, 2, 0, 3), "dv": dv.permute(1, 2, 0, 3), "ds0": r}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "decay":
        return _exact_decay(case, st)
    pos = st["pos"].double()
    turn = []
    for axis, n in enumerate(_sections(case)):
        j = torch.arange(n, device=DEV, dtype=torch.float64)
        turn.append(pos[axis].unsqueeze(-1) * torch.pow(torch.tensor(BASE, device=DEV, dtype=torch.float64), -j / n))
    turn = torch.cat(turn, -1).unsqueeze(1)
    pairs = turn.shape[-1]
    turn = torch.polar(torch.ones_like(turn), turn)
    out = {}
    for name in ("q", "k"):
        x, w = st[name].double(), st["w" + name].double()
        r = x.square().sum(-1, keepdim=True).div(case["d"]).add(EPS).sqrt().reciprocal()

        def rotated(y, z):
            u = y[..., : 2 * pairs]
            u = torch.complex(u[..., :pairs], u[..., pairs:]) if case["halves"] else torch.view_as_complex(
                u.reshape(*u.shape[:-1], pairs, 2).contiguous())
            u = u * z
            u = torch.cat([u.real, u.imag], -1) if case["halves"] else torch.view_as_real(u).flatten(-2)
            return torch.cat([u, y[..., 2 * pairs:]], -1)

        if case["dir"] == "fwd":
            out[name] = rotated(x * r * w, turn)
            continue
        # y = R (w x r): what reaches x r is w R^T dy, and r's own share is along x
        back = rotated(st["d" + name].double(), turn.conj())
        out["dw" + name] = torch.einsum("bhli,bhli,bhlj->i", back, x, r)
        back = back * w
        along = torch.einsum("bhli,bhli->bhl", back, x).unsqueeze(-1)
        out["d" + name] = back * r - x * (along * r ** 3 / case["d"])
    return out
