"""Cases of the sequence operators that stand beside the FAVOR+ attention.

Three operators, each in the directions and types that a program uses:

  scan    the gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t over the
          tokens of [B, H, L, d] ("fwd", its gradients "bwd", one token "step")
  norm    layer norm over the last axis ("fwd", "bwd" with the weight's gradient)
  rotary  rotation of queries and keys by positions on one to three axes
          ("fwd", "bwd" the inverse rotation of the gradients)

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
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one new token for each of 256 sequences of 8 heads (the decode workload's sizes)
        {"name": "scan-step-bf16", "op": "scan", "dir": "step", "dtype": "bf16", "B": 256, "H": 8, "L": 1, "d": 64,
         "packed": 0, "tokens": False},
        # protein sequences: 4 x 8192 tokens, 8 heads of 64
        {"name": "scan-fwd-bf16", "op": "scan", "dir": "fwd", "dtype": "bf16", "B": 4, "H": 8, "L": 8192, "d": 64,
         "packed": 0, "tokens": False},
        # one long sequence over a wide model, channels side by side in memory
        {"name": "scan-fwd-f32-long", "op": "scan", "dir": "fwd", "dtype": "f32", "B": 1, "H": 16, "L": 65536, "d": 128,
         "packed": 0, "tokens": True},
        # training on images as sequences: 2 x 12288 pixels, several packed into each row
        {"name": "scan-bwd-bf16", "op": "scan", "dir": "bwd", "dtype": "bf16", "B": 2, "H": 8, "L": 12288, "d": 64,
         "packed": 5, "tokens": False},
        # a short odd batch in 32 bits
        {"name": "scan-bwd-f32-odd", "op": "scan", "dir": "bwd", "dtype": "f32", "B": 3, "H": 5, "L": 1777, "d": 40,
         "packed": 2, "tokens": True},
        # the residual rows of eight new tokens, model width 512
        {"name": "norm-fwd-f32-few", "op": "norm", "dir": "fwd", "dtype": "f32", "B": 8, "H": 1, "L": 1, "d": 512,
         "affine": True, "tokens": False},
        # the queries of the long-sequence workload, read out of the joint projection's output
        {"name": "norm-fwd-bf16-queries", "op": "norm", "dir": "fwd", "dtype": "bf16", "B": 1, "H": 16, "L": 65536,
         "d": 128, "affine": False, "tokens": True},
        # training: the rows of 8 x 4096 tokens, model width 512
        {"name": "norm-bwd-bf16", "op": "norm", "dir": "bwd", "dtype": "bf16", "B": 8, "H": 1, "L": 4096, "d": 512,
         "affine": True, "tokens": False},
        # an odd width in 32 bits
        {"name": "norm-bwd-f32-odd", "op": "norm", "dir": "bwd", "dtype": "f32", "B": 3, "H": 1, "L": 1111, "d": 771,
         "affine": True, "tokens": False},
        # one new token of 256 sequences at far positions
        {"name": "rotary-step-bf16", "op": "rotary", "dir": "fwd", "dtype": "bf16", "B": 256, "H": 8, "Hk": 8, "L": 1,
         "d": 64, "axes": 1, "rot": 64, "halves": True, "tokens": False},
        # images: rows and columns of 96 x 128 pixels
        {"name": "rotary-image-f32", "op": "rotary", "dir": "fwd", "dtype": "f32", "B": 2, "H": 8, "Hk": 8, "L": 12288,
         "d": 64, "axes": 2, "rot": 64, "halves": False, "tokens": True},
        # video: time, height and width; the gradients of queries and of fewer key heads
        {"name": "rotary-video-bwd-bf16", "op": "rotary", "dir": "bwd", "dtype": "bf16", "B": 1, "H": 16, "Hk": 4,
         "L": 65536, "d": 128, "axes": 3, "rot": 128, "halves": True, "tokens": False},
    ]


def _spread(rng, low, high):
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op, direction = rng.choice([("scan", "step"), ("scan", "fwd"), ("scan", "fwd"), ("scan", "bwd"), ("scan", "bwd"),
                                ("norm", "fwd"), ("norm", "fwd"), ("norm", "bwd"), ("norm", "bwd"),
                                ("rotary", "fwd"), ("rotary", "fwd"), ("rotary", "bwd")])
    case = {"op": op, "dir": direction, "dtype": rng.choice(["f32", "bf16", "bf16"]), "tokens": rng.random() < 0.5}
    if op == "scan":
        case["B"] = _spread(rng, 1, 300) if direction == "step" else _spread(rng, 1, 8)
        case["H"] = _spread(rng, 1, 16)
        case["d"] = rng.choice([16, 40, 64, 64, 80, 96, 128, 128, rng.randint(1, 128)])
        case["L"] = 1 if direction == "step" else _spread(rng, 2, 65536)
        case["packed"] = rng.choice([0, 0, rng.randint(1, 9)])
        most = 1 << 26
    elif op == "norm":
        if rng.random() < 0.5:      # heads of queries and keys
            case["H"], case["d"] = _spread(rng, 2, 16), rng.choice([32, 64, 64, 96, 128, 128, rng.randint(8, 128)])
        else:                       # rows of the model's width
            case["H"], case["d"] = 1, rng.choice([256, 512, 512, 1024, 2048, rng.randint(129, 4100)])
        case["B"] = _spread(rng, 1, 16)
        case["L"] = _spread(rng, 1, 65536)
        case["affine"] = direction == "bwd" or rng.random() < 0.6
        most = 1 << 27
    else:
        case["axes"] = rng.choice([1, 2, 2, 3])
        case["d"] = rng.choice([32, 64, 64, 96, 128, 128, 2 * rng.randint(8, 64)])
        case["rot"] = case["d"] if rng.random() < 0.7 else 2 * rng.randint(case["axes"], case["d"] // 2)
        case["B"] = _spread(rng, 1, 64)
        case["H"] = _spread(rng, 1, 16)
        case["Hk"] = max(1, case["H"] // rng.choice([1, 1, 2, 4]))
        case["L"] = 1 if rng.random() < 0.2 else _spread(rng, 2, 65536)
        case["halves"] = rng.random() < 0.5
        most = 1 << 26
    rows = case["B"] * case["H"] * case["d"]
    case["L"] = max(1, min(case["L"], most // rows))
    return case


# --- inputs -------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)


def _heads(case, t, heads=None, part=None):
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


def _gates(case, gen):
    """Log gates as they come from a gated layer: a decay per channel between
    about two tokens and some thousands, moved by the token; with "packed" the
    first token of each further sequence in a row drops the state."""
    B, H, L, d = (case[k] for k in "BHLd")
    slow = torch.exp(torch.rand((1, H, 1, d), generator=gen, device=DEV) * 6.2 - 7.0)
    g = -2 * slow * torch.sigmoid(_normal(gen, B, H, L, d))
    if case["packed"] and L > 1:
        first = torch.randint(1, L, (case["packed"],), generator=gen, device=DEV)
        g[:, :, first] = -math.inf
    return g


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    B, H, L, d = (case[k] for k in "BHLd")
    st = {"case": case}
    if case["op"] == "scan":
        g = _gates(case, gen)
        x = _normal(gen, B, H, L, d) * torch.sqrt(1 - torch.exp(2 * g))
        st["h0"] = _normal(gen, B, H, d)
        if case["dir"] == "step":
            st["g"], st["x"] = (t.reshape(B, H, d).to(_TYPES[case["dtype"]]).contiguous() for t in (g, x))
            st["next"] = torch.empty_like(st["h0"])
            return st
        st["g"] = _heads(case, g)
        if case["dir"] == "fwd":
            st["x"] = _heads(case, x)
        else:
            st["h"] = _heads(case, _scan(torch.exp(st["g"].float()), x, st["h0"])[0])
            st["dh"] = _heads(case, _normal(gen, B, H, L, d))
            st["dlast"] = _normal(gen, B, H, d)
    elif case["op"] == "norm":
        x = _normal(gen, B, H, L, d) * (0.5 + 2 * torch.rand((B, H, L, 1), generator=gen, device=DEV))
        x += _normal(gen, B, H, L, 1)
        st["x"] = _heads(case, x, part=0 if case["H"] > 1 else None)
        st["gamma"] = 1 + 0.2 * _normal(gen, d) if case["affine"] else None
        st["beta"] = 0.2 * _normal(gen, d) if case["affine"] else None
        if case["dir"] == "bwd":
            st["dy"] = _heads(case, _normal(gen, B, H, L, d))
    else:
        st["q"] = _heads(case, _normal(gen, B, H, L, d))
        st["k"] = _heads(case, _normal(gen, B, case["Hk"], L, d))
        st["pos"] = _positions(case, gen)
        freq, axis = _frequencies(case)
        # what a turn is in the framework's table: 2^64
        st["table"] = torch.round(freq / (2 * math.pi) * 2.0 ** 64).to(torch.int64).to(DEV)
        st["freq"], st["axis"] = freq.to(DEV), axis.to(DEV)
        st["sections"] = _sections(case)
    return st


# --- plain forms ----------------------------------------------------------------

def _scan(a, x, h0):
    """h_t = a_t h_{t-1} + x_t along the second last axis in 32 bits, by
    doubling the span that each token has seen; and the last h."""
    x = torch.cat([x[..., :1, :] + a[..., :1, :] * h0.unsqueeze(-2), x[..., 1:, :]], -2)
    n = 1
    while n < x.shape[-2]:
        x = torch.cat([x[..., :n, :], x[..., n:, :] + a[..., n:, :] * x[..., :-n, :]], -2)
        a = torch.cat([a[..., :n, :], a[..., n:, :] * a[..., :-n, :]], -2)
        n *= 2
    return x, x[..., -1, :]


def _plain_scan(st):
    t = _TYPES[st["case"]["dtype"]]
    a = torch.exp(st["g"].float())
    if st["case"]["dir"] == "step":
        h = a * st["h0"] + st["x"].float()
        return {"h": h.to(t), "state": h}
    if st["case"]["dir"] == "fwd":
        h, last = _scan(a, st["x"].float(), st["h0"])
        return {"h": h.to(t), "last": last.contiguous()}
    dh = st["dh"].float()
    back = a.flip(-2)
    c = _scan(back, back * dh.flip(-2), st["dlast"])[0].flip(-2)     # c_t = a_t (dh_t + c_{t+1})
    dx = dh + torch.cat([c[..., 1:, :], st["dlast"].unsqueeze(-2)], -2)
    before = torch.cat([st["h0"].unsqueeze(-2), st["h"].float()[..., :-1, :]], -2)
    return {"dx": dx.to(t), "dg": (c * before).to(t), "dh0": c[..., 0, :].contiguous()}


def _plain_norm(st):
    t = _TYPES[st["case"]["dtype"]]
    x = st["x"].float()
    x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    x = x * r
    if st["case"]["dir"] == "fwd":
        y = x * st["gamma"] + st["beta"] if st["gamma"] is not None else x
        return {"y": y.to(t).contiguous()}
    dy = st["dy"].float()
    dn = dy * st["gamma"]
    dx = r * (dn - dn.mean(-1, keepdim=True) - x * (dn * x).mean(-1, keepdim=True))
    return {"dx": dx.to(t).contiguous(), "dgamma": (dy * x).sum((0, 1, 2)), "dbeta": dy.sum((0, 1, 2))}


def _turn(x, cos, sin, rot, halves):
    u = x[..., :rot].float()
    a, b = (u[..., : rot // 2], u[..., rot // 2:]) if halves else (u[..., 0::2], u[..., 1::2])
    a, b = a * cos - b * sin, a * sin + b * cos
    u = torch.cat([a, b], -1) if halves else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([u.to(x.dtype), x[..., rot:]], -1)


def _plain_rotary(st):
    case = st["case"]
    angle = st["pos"][st["axis"]].permute(1, 2, 0).double() * st["freq"]          # [B or 1, L, pairs]
    angle = (-angle if case["dir"] == "bwd" else angle).unsqueeze(1)
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    return {n: _turn(st[n], cos, sin, case["rot"], case["halves"]).contiguous() for n in ("q", "k")}


# --- one pass -------------------------------------------------------------------

def run(state):
    case = state["case"]
    if not own:
        return {"scan": _plain_scan, "norm": _plain_norm, "rotary": _plain_rotary}[case["op"]](state)
    import linear_softmax_attention_gb300 as favor

    st = state
    if case["op"] == "scan":
        if case["dir"] == "step":
            h, new = favor.gated_scan_step(st["x"], st["g"], st["h0"], new_state=st["next"])
            return {"h": h, "state": new}
        if case["dir"] == "fwd":
            h, last = favor.fwd_gated_scan(st["x"], st["g"], h0=st["h0"])
            return {"h": h, "last": last}
        dx, dg, dh0 = favor.bwd_gated_scan(st["g"], st["h"], st["dh"], h0=st["h0"], dhT=st["dlast"])
        return {"dx": dx, "dg": dg, "dh0": dh0}
    if case["op"] == "norm":
        if case["dir"] == "fwd":
            return {"y": favor.fwd_layer_norm(st["x"], st["gamma"], st["beta"], EPS)}
        dx, dgamma, dbeta = favor.bwd_layer_norm(st["x"], st["dy"], st["gamma"], EPS)
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    call = favor.fwd_rotary if case["dir"] == "fwd" else favor.bwd_rotary
    q, k = call(st["q"], st["k"], st["pos"], st["table"], st["sections"],
                pairing="halves" if case["halves"] else "adjacent")
    return {"q": q, "k": k}


def work(case):
    size = {"f32": 4, "bf16": 2}[case["dtype"]]
    B, H, L, d = (case[k] for k in "BHLd")
    n, rows = B * H * L * d, B * H * d
    if case["op"] == "scan":
        if case["dir"] == "bwd":     # g, h, dh in; dx, dg out; h0, dlast in, dh0 out
            return {"bytes": 5 * n * size + 12 * rows, "flops": 4 * n}
        return {"bytes": 3 * n * size + 8 * rows, "flops": 3 * n}
    if case["op"] == "norm":
        if case["dir"] == "bwd":
            return {"bytes": 3 * n * size + 12 * d, "flops": 16 * n}
        return {"bytes": 2 * n * size + (8 * d if case["affine"] else 0), "flops": 8 * n}
    n += B * case["Hk"] * L * d
    positions = case["axes"] * (B if L == 1 else 1) * L
    return {"bytes": 2 * n * size + 4 * positions + 4 * case["rot"], "flops": 3 * n}


# --- the definitions in 64 bits ---------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "scan":
        g, h = st["g"].double(), st["h0"].double()
        if case["dir"] == "step":
            h = st["x"].double() + h * g.exp()
            return {"h": h, "state": h}
        if case["dir"] == "fwd":
            g, x = (t.permute(2, 0, 1, 3).contiguous().double() for t in (st["g"], st["x"]))
            g.exp_()
            for t in range(case["L"]):
                h = torch.addcmul(x[t], g[t], h, out=x[t])
            return {"h": x.permute(1, 2, 0, 3), "last": h.clone()}
        g, before, dh = (t.permute(2, 0, 1, 3).contiguous().double() for t in (st["g"], st["h"], st["dh"]))
        before = torch.cat([h.unsqueeze(0), before[:-1]])
        g.exp_()
        dg, carry = torch.empty_like(g), st["dlast"].double()
        for t in reversed(range(case["L"])):
            dh[t] += carry                       # all that reaches h_t
            carry = torch.mul(g[t], dh[t], out=dg[t])
        dh0 = carry.clone()
        return {"dx": dh.permute(1, 2, 0, 3), "dg": (dg * before).permute(1, 2, 0, 3), "dh0": dh0}
    if case["op"] == "norm":
        x = st["x"].double()
        var, mean = torch.var_mean(x, dim=-1, correction=0, keepdim=True)
        s = (var + EPS).sqrt()
        n = (x - mean) / s
        if case["dir"] == "fwd":
            return {"y": n if st["gamma"] is None else n * st["gamma"].double() + st["beta"].double()}
        dy, d = st["dy"].double(), case["d"]
        dn = dy * st["gamma"].double()
        # d y_j / d x_i = gamma_j (delta_ij - 1/d - n_i n_j / d) / s
        dx = (dn - dn.sum(-1, keepdim=True) / d - n * ((dn * n).sum(-1, keepdim=True) / d)) / s
        return {"dx": dx, "dgamma": torch.einsum("bhli,bhli->i", dy, n), "dbeta": torch.einsum("bhli->i", dy)}
    sign = -1.0 if case["dir"] == "bwd" else 1.0
    pos = st["pos"].double()
    turn, at = [], 0
    for axis, n in enumerate(_sections(case)):
        j = torch.arange(n, device=DEV, dtype=torch.float64)
        turn.append(pos[axis].unsqueeze(-1) * torch.pow(torch.tensor(BASE, device=DEV, dtype=torch.float64), -j / n))
        at += n
    turn = torch.cat(turn, -1).unsqueeze(1) * sign
    turn = torch.polar(torch.ones_like(turn), turn)
    out = {}
    for name in ("q", "k"):
        x = st[name].double()
        u = x[..., : 2 * at]
        z = torch.complex(u[..., :at], u[..., at:]) if case["halves"] else torch.complex(u[..., 0::2], u[..., 1::2])
        z = z * turn
        u = torch.cat([z.real, z.imag], -1) if case["halves"] else torch.view_as_real(z).flatten(-2)
        out[name] = torch.cat([u, x[..., 2 * at:]], -1)
    return out
