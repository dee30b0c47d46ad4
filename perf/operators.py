"""Layer norm, rotary positions and the gated recurrence: cases to time, and their plain forms.

Each case is one call of one operator at one size.  ``run`` computes it with
elementary torch operations, or (``own``) with the library's kernels.
"""
import math
import random

import torch

own = False

CHUNK = 64  # tokens between two saved states of the gated recurrence
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# elements a drawn case may have at most, by operator (those of the largest listed case)
MOST = {"layernorm": 16384 * 2048, "rotary": 2 * 8 * 16 * 2048 * 64, "gatedrec": 8 * 2048 * 1024}


def listed():
    return [
        # the norm before a decode step's projections: 128 sequences, one token each
        {"name": "ln_fwd_decode", "op": "layernorm_fwd", "dtype": "bf16", "rows": 128, "D": 1024,
         "residual": True},
        # the norm of a training or prefill step: 8 sequences of 2048 tokens
        {"name": "ln_fwd_layer", "op": "layernorm_fwd", "dtype": "bf16", "rows": 16384, "D": 1024,
         "residual": True},
        # its gradient at the wide layer shape, the largest call
        {"name": "ln_bwd_wide", "op": "layernorm_bwd", "dtype": "bf16", "rows": 16384, "D": 2048,
         "residual": True},
        # fp32, a width and a row count that no vector divides
        {"name": "ln_bwd_odd_f32", "op": "layernorm_bwd", "dtype": "f32", "rows": 3001, "D": 999,
         "residual": False},
        # decode: one token for each of 128 sequences, each at its own position
        {"name": "rot_fwd_decode", "op": "rotary_fwd", "dtype": "bf16", "B": 128, "Hq": 16, "Hk": 16,
         "L": 1, "D": 64, "rot": 64, "layout": "half", "scaling": "none", "pos": "each"},
        # prefill or training of the window layer
        {"name": "rot_fwd_layer", "op": "rotary_fwd", "dtype": "bf16", "B": 8, "Hq": 16, "Hk": 16,
         "L": 2048, "D": 64, "rot": 64, "layout": "half", "scaling": "none", "pos": "shared"},
        # a long context: far positions, frequencies scaled by parts, half of each head
        # rotated, fewer key heads than query heads
        {"name": "rot_fwd_long", "op": "rotary_fwd", "dtype": "bf16", "B": 1, "Hq": 16, "Hk": 4,
         "L": 16000, "D": 128, "rot": 64, "layout": "interleaved", "scaling": "parts", "pos": "far"},
        # the gradient (fp32, as the window attention's backward gives it)
        {"name": "rot_bwd_layer", "op": "rotary_bwd", "dtype": "f32", "B": 8, "Hq": 16, "Hk": 16,
         "L": 2048, "D": 64, "rot": 64, "layout": "half", "scaling": "none", "pos": "shared"},
        # decode: one token for each of 128 sequences
        {"name": "rec_step_decode", "op": "gatedrec_step", "dtype": "bf16", "B": 128, "D": 1024},
        # training: 8 sequences of 2048 tokens, states kept for the gradient
        {"name": "rec_fwd_layer", "op": "gatedrec_fwd", "dtype": "bf16", "B": 8, "L": 2048,
         "D": 1024, "ragged": False, "h0": False},
        # one long prompt that continues a state: few channels, a long axis
        {"name": "rec_fwd_long", "op": "gatedrec_fwd", "dtype": "bf16", "B": 1, "L": 16384,
         "D": 1000, "ragged": False, "h0": True},
        # the gradient of a padded batch
        {"name": "rec_bwd_ragged", "op": "gatedrec_bwd", "dtype": "bf16", "B": 8, "L": 2048,
         "D": 1024, "ragged": True, "h0": True},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["layernorm_fwd", "layernorm_bwd", "rotary_fwd", "rotary_bwd", "gatedrec_fwd",
                     "gatedrec_bwd", "gatedrec_step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    most = MOST[op.split("_")[0]]
    if dtype == "f32":
        most //= 2
    if op.startswith("layernorm"):
        D = rng.choice([_spread(rng, 17, 8192), 8 * _spread(rng, 8, 1024), 1024, 2048])
        return {"op": op, "dtype": dtype, "D": D, "rows": _spread(rng, 1, most // D),
                "residual": rng.random() < 0.5}
    if op.startswith("rotary"):
        D = rng.choice([64, 128, 2 * rng.randint(16, 128)])
        most = most // 2 if op == "rotary_bwd" and dtype == "bf16" else most
        Hk = rng.choice([1, 2, 4, 16])
        Hq = Hk * rng.choice([1, 2, 4])
        B = _spread(rng, 1, 128)
        return {"op": op, "dtype": dtype if op == "rotary_fwd" else "f32", "B": B, "Hq": Hq,
                "Hk": Hk, "L": _spread(rng, 1, max(1, min(16384, most // (B * (Hq + Hk) * D)))),
                "D": D, "rot": rng.choice([D, D, 2 * rng.randint(4, D // 2)]),
                "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "parts"]),
                "pos": rng.choice(["shared", "each", "far"])}
    D = rng.choice([_spread(rng, 33, 4096), 64 * _spread(rng, 1, 64), 1024, 2048])
    B = _spread(rng, 1, 128)
    if op == "gatedrec_step":
        return {"op": op, "dtype": dtype, "B": B, "D": D}
    return {"op": op, "dtype": dtype, "B": B, "D": D,
            "L": _spread(rng, 1, max(1, min(16384, most // (B * D)))),
            "ragged": rng.random() < 0.5, "h0": rng.random() < 0.5}


def _lengths(case):
    """The lengths of a padded batch: a full one, an empty one, the rest in between."""
    r = random.Random(case["B"] * 1000003 + case["L"] * 101 + case["D"])
    n = [r.randint(1, case["L"]) for _ in range(case["B"])]
    n[0] = case["L"]
    if case["B"] > 3:
        n[-1] = 0
    return n


def _frequencies(case):
    """Turns per position of each pair, in 64 bits: base 10000; scaled for an 8 times longer
    context linearly, or by parts (pairs that turn less than once over the original 2048
    tokens are slowed, those that turn more than four times are not)."""
    rot = case["rot"]
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot) / (2 * math.pi)
    if case["scaling"] == "linear":
        f = f / 8
    elif case["scaling"] == "parts":
        keep = ((f * 2048 - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        f = f * (keep + (1 - keep) / 8)
    return f


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    op = case["op"]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)

    def empty(*shape, dtype=dt):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    s = {"case": case}
    f32 = torch.float32
    if op.startswith("layernorm"):
        rows, D = case["rows"], case["D"]
        s["w"] = 1 + normal(D, scale=0.1, dtype=f32)
        s["b"] = normal(D, scale=0.1, dtype=f32)
        if op == "layernorm_fwd":
            s["x"] = normal(rows, D)
            s["res"] = normal(rows, D, scale=2.0) if case["residual"] else None
            s["y"], s["r"] = empty(rows, D), empty(rows, D) if case["residual"] else None
            s["mean"], s["rstd"] = empty(rows, dtype=f32), empty(rows, dtype=f32)
        else:
            s["r"] = normal(rows, D, scale=2.0) + normal(rows, 1, scale=0.5)
            s["dy"] = normal(rows, D)
            s["dres"] = normal(rows, D, dtype=f32) if case["residual"] else None
            r = s["r"].double()
            s["mean"] = r.mean(1).float()
            s["rstd"] = ((r - r.mean(1, keepdim=True)).square().mean(1) + EPS).rsqrt().float()
            s["dx"] = empty(rows, D, dtype=f32)
            s["dw"], s["db"] = empty(D, dtype=f32), empty(D, dtype=f32)
            s["ws"] = _layernorm_workspace(rows, D)
    elif op.startswith("rotary"):
        B, L, D = case["B"], case["L"], case["D"]
        s["q"], s["k"] = normal(B, case["Hq"], L, D), normal(B, case["Hk"], L, D)
        s["qo"], s["ko"] = torch.zeros_like(s["q"]), torch.zeros_like(s["k"])
        s["freqs"] = _frequencies(case).cuda()
        s["mscale"] = 1.25 if case["scaling"] == "parts" else 1.0
        s["pos"] = 0
        if case["pos"] == "far":
            s["pos"] = 1000000 + seed % 1000
        elif case["pos"] == "each":
            s["pos"] = torch.randint(0, 100000, (B,), generator=gen, device="cuda")
    else:
        B, D = case["B"], case["D"]
        # a bias of its own for each channel: memories from a few tokens to some hundreds
        bias = torch.rand(D, generator=gen, device="cuda") * 6
        if op == "gatedrec_step":
            s["x"], s["g"], s["y"] = normal(B, D), (normal(B, D, dtype=f32) + bias).to(dt), empty(B, D)
            s["h"] = normal(B, D, dtype=f32)
            return s
        L = case["L"]
        s["x"] = normal(B, L, D)
        s["g"] = (normal(B, L, D, dtype=f32) + bias).to(dt)
        s["h0"] = normal(B, D, dtype=f32) if case["h0"] else None
        s["lengths"] = torch.tensor(_lengths(case), device="cuda") if case["ragged"] else None
        n = -(-L // CHUNK)
        if op == "gatedrec_fwd":
            s["y"], s["h_last"] = empty(B, L, D), empty(B, D, dtype=f32)
            s["h_chunks"] = empty(B, n, D, dtype=f32)
        else:
            s["dy"] = normal(B, L, D)
            s["dh_last"] = normal(B, D, dtype=f32)
            s["h_chunks"] = _forward(s)[2]
            s["dx"], s["dg"] = empty(B, L, D, dtype=f32), empty(B, L, D, dtype=f32)
            s["dh0"] = empty(B, D, dtype=f32)
    return s


def _layernorm_workspace(rows, D):
    """Scratch that holds the partial sums of dweight and dbias: at most 512 parts."""
    return torch.empty(512 * 2 * D, dtype=torch.float32, device="cuda")


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from h_{-1} = 0, by doubling the span."""
    step, L = 1, a.shape[1]
    while step < L:
        head_a, head_b = a[:, :step], b[:, :step]
        b = torch.cat([head_b, b[:, step:] + a[:, step:] * b[:, :-step]], 1)
        a = torch.cat([head_a, a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return b


def _inside(s):
    """Which tokens are inside their sequence, [B, L, 1]."""
    B, L = s["x"].shape[:2]
    t = torch.arange(L, device="cuda")
    n = s["lengths"]
    return (t < n[:, None] if n is not None else (t >= 0).expand(B, L))[:, :, None]


def _states(s):
    """Gates a, 1 - a and x in 32 bits (outside a sequence: a = 1, x = 0) and the states h."""
    inside = _inside(s)
    g, x = s["g"].float(), torch.where(inside, s["x"].float(), 0.0)
    a = torch.where(inside, torch.sigmoid(g), 1.0)
    na = torch.where(inside, torch.sigmoid(-g), 0.0)
    b = na * x
    if s["h0"] is not None:
        b = torch.cat([(b[:, 0] + a[:, 0] * s["h0"])[:, None], b[:, 1:]], 1)
    return inside, a, na, x, _scan(a, b)


def _previous(s, h):
    """h_{t-1} for every t."""
    first = s["h0"] if s["h0"] is not None else torch.zeros_like(h[:, 0])
    return torch.cat([first[:, None], h[:, :-1]], 1)


def _forward(s):
    inside, _, _, _, h = _states(s)
    # the states saved for the gradient: those that enter tokens 0, CHUNK, 2 CHUNK, ...
    chunks = torch.where(inside, _previous(s, h), 0.0)[:, ::CHUNK].contiguous()
    return torch.where(inside, h, 0.0).to(s["x"].dtype), h[:, -1].contiguous(), chunks


def _backward(s):
    inside, a, na, x, h = _states(s)
    dy = torch.where(inside, s["dy"].float(), 0.0)
    dy = torch.cat([dy[:, :-1], (dy[:, -1] + s["dh_last"])[:, None]], 1)
    following = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    lam = _scan(following.flip(1), dy.flip(1)).flip(1)
    return na * lam, lam * (_previous(s, h) - x) * a * na, a[:, 0] * lam[:, 0]


def _rotate(x, cos, sin, rot, layout):
    """x [B, H, L, D] in 32 bits, cos and sin [B or 1, 1, L, rot / 2]."""
    if layout == "half":
        u, v = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([u * cos - v * sin, u * sin + v * cos], -1)
    else:
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([u * cos - v * sin, u * sin + v * cos], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rotary(s):
    case = s["case"]
    t = torch.arange(case["L"], device="cuda", dtype=torch.float64)
    pos = s["pos"]
    # angles of far positions in 64 bits, whole turns taken off
    p = (pos.double()[:, None] if torch.is_tensor(pos) else float(pos)) + t
    turns = p.reshape(-1, 1, case["L"], 1) * s["freqs"]
    angle = 2 * math.pi * (turns - torch.round(turns))
    if case["op"] == "rotary_bwd":
        angle = -angle
    cos, sin = (s["mscale"] * torch.cos(angle)).float(), (s["mscale"] * torch.sin(angle)).float()
    return [_rotate(s[n].float(), cos, sin, case["rot"], case["layout"]).to(s[n].dtype)
            for n in ("q", "k")]


def _plain_layernorm(s):
    if s["case"]["op"] == "layernorm_fwd":
        x = s["x"]
        r = (x.float() + s["res"].float()).to(x.dtype) if s["res"] is not None else x
        z = r.float()
        mean = z.mean(1, keepdim=True)
        z = z - mean
        rstd = 1 / torch.sqrt((z * z).mean(1, keepdim=True) + EPS)
        y = (z * rstd * s["w"] + s["b"]).to(x.dtype)
        return [y, mean[:, 0], rstd[:, 0]] + ([r] if s["res"] is not None else [])
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (s["r"].float() - s["mean"][:, None]) * rstd
    t = dy * s["w"]
    dx = rstd * (t - t.mean(1, keepdim=True) - xh * (t * xh).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"]
    return [dx, (dy * xh).sum(0), dy.sum(0)]


def _plain_step(s):
    g = s["g"].float()
    s["h"].copy_(torch.sigmoid(g) * s["h"] + torch.sigmoid(-g) * s["x"].float())
    return [s["h"].to(s["x"].dtype), s["h"]]


def _plain(s):
    op = s["case"]["op"]
    if op.startswith("layernorm"):
        return _plain_layernorm(s)
    if op.startswith("rotary"):
        return _plain_rotary(s)
    if op == "gatedrec_step":
        return _plain_step(s)
    return list(_forward(s) if op == "gatedrec_fwd" else _backward(s))


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _own(s):
    import linear_attention_lm_b200 as lab

    case = s["case"]
    op = case["op"]
    if op == "layernorm_fwd":
        lab.based_layernorm_fwd(s["x"], s["w"], s["b"], s["y"], eps=EPS, residual=s["res"],
                                resid_out=s["r"], mean=s["mean"], rstd=s["rstd"])
        return [s["y"], s["mean"], s["rstd"]] + ([s["r"]] if s["res"] is not None else [])
    if op == "layernorm_bwd":
        lab.based_layernorm_bwd(s["dy"], s["r"], s["w"], s["mean"], s["rstd"], s["dx"], s["dw"],
                                s["db"], dresid=s["dres"], workspace=s["ws"])
        return [s["dx"], s["dw"], s["db"]]
    if op == "rotary_fwd":
        lab.based_rotary_fwd(s["q"], s["k"], s["qo"], s["ko"], s["freqs"], pos=s["pos"],
                             layout=case["layout"], mscale=s["mscale"])
        return [s["qo"], s["ko"]]
    if op == "rotary_bwd":
        lab.based_rotary_bwd(s["q"], s["k"], s["qo"], s["ko"], s["freqs"], pos=s["pos"],
                             layout=case["layout"], mscale=s["mscale"])
        return [s["qo"], s["ko"]]
    if op == "gatedrec_step":
        lab.based_gatedrec_step(s["x"], s["g"], s["h"], s["y"])
        return [s["y"], s["h"]]
    if op == "gatedrec_fwd":
        lab.based_gatedrec_fwd(s["x"], s["g"], s["y"], h0=s["h0"], h_last=s["h_last"],
                               h_chunks=s["h_chunks"], lengths=s["lengths"])
        return [s["y"], s["h_last"], s["h_chunks"]]
    lab.based_gatedrec_bwd(s["x"], s["g"], s["dy"], s["h_chunks"], s["dx"], s["dg"],
                           dh_last=s["dh_last"], dh0=s["dh0"], lengths=s["lengths"])
    return [s["dx"], s["dg"], s["dh0"]]


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op.startswith("layernorm"):
        n, D, rows, res = case["rows"] * case["D"], case["D"], case["rows"], case["residual"]
        if op == "layernorm_fwd":
            return {"bytes": n * e * (4 if res else 2) + 8 * D + 8 * rows, "flops": 9 * n}
        return {"bytes": n * (2 * e + (8 if res else 4)) + 12 * D + 8 * rows, "flops": 13 * n}
    if op.startswith("rotary"):
        n = case["B"] * (case["Hq"] + case["Hk"]) * case["L"]
        return {"bytes": 2 * n * case["D"] * e + 4 * case["rot"], "flops": 3 * n * case["rot"]}
    if op == "gatedrec_step":
        n = case["B"] * case["D"]
        return {"bytes": n * (3 * e + 8), "flops": 8 * n}
    B, D, L = case["B"], case["D"], case["L"]
    tokens = sum(_lengths(case)) if case["ragged"] else B * L
    ends = 4 * B * D
    saved = 4 * D * (sum(-(-n // CHUNK) for n in _lengths(case)) if case["ragged"]
                     else B * -(-L // CHUNK))
    if op == "gatedrec_fwd":
        return {"bytes": tokens * D * 2 * e + B * L * D * e + saved + ends * (2 if case["h0"] else 1),
                "flops": 8 * tokens * D}
    return {"bytes": tokens * D * 3 * e + 8 * B * L * D + saved + 2 * ends, "flops": 18 * tokens * D}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_layernorm(s):
    w = s["w"].double()
    if s["case"]["op"] == "layernorm_fwd":
        z = s["x"].double()
        if s["res"] is not None:
            # the residual stream is kept in the inputs' type, and that is what is normalised
            z = (z + s["res"].double()).to(s["x"].dtype).double()
        var, mean = torch.var_mean(z, dim=1, correction=0)
        rstd = (var + EPS) ** -0.5
        y = torch.addcmul(s["b"].double(), torch.einsum("rd,r->rd", z - mean.unsqueeze(1), rstd), w)
        return [y, mean, rstd] + ([z] if s["res"] is not None else [])
    # by the Jacobian of z -> xh:  (I - 1 1^T / D - xh xh^T / D) / sigma
    D = s["case"]["D"]
    dy, rstd = s["dy"].double(), s["rstd"].double()
    xh = torch.einsum("rd,r->rd", s["r"].double() - s["mean"].double().unsqueeze(1), rstd)
    t = torch.einsum("rd,d->rd", dy, w)
    along = torch.einsum("rd,rd->r", t, xh) / D
    dx = torch.einsum("rd,r->rd", t - t.sum(1).unsqueeze(1) / D - torch.einsum("r,rd->rd", along, xh), rstd)
    if s["dres"] is not None:
        dx += s["dres"].double()
    return [dx, torch.einsum("rd,rd->d", dy, xh), torch.einsum("rd->d", dy)]


def _exact_rotary(s):
    """Each pair as a complex number times m e^{i angle}; the gradient with the conjugate."""
    case = s["case"]
    L, rot = case["L"], case["rot"]
    out = []
    for n in ("q", "k"):
        x = s[n].double().clone()
        if case["layout"] == "half":
            z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot])
        else:
            z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2).contiguous())
        for b in range(case["B"]):
            start = int(s["pos"][b]) if torch.is_tensor(s["pos"]) else s["pos"]
            angle = torch.outer(torch.arange(start, start + L, device="cuda").double(),
                                s["freqs"] * (2 * math.pi))
            turn = torch.polar(torch.full_like(angle, s["mscale"]), angle)
            z[b] *= turn.conj() if case["op"] == "rotary_bwd" else turn
        if case["layout"] == "half":
            x[..., :rot // 2], x[..., rot // 2:rot] = z.real, z.imag
        else:
            x[..., :rot] = torch.view_as_real(z).flatten(-2)
        out.append(x)
    return out


def _exact_gatedrec(s):
    """Token by token, from the recurrence itself."""
    op = s["case"]["op"]
    if op == "gatedrec_step":
        e = torch.exp(-s["g"].double())
        h = (s["h"].double() + e * s["x"].double()) / (1 + e)
        return [h, h]
    B, L, D = s["x"].shape
    n = s["lengths"] if s["lengths"] is not None else torch.full((B,), L, device="cuda")
    h = s["h0"].double() if s["h0"] is not None else torch.zeros(B, D, dtype=torch.float64, device="cuda")
    y = torch.zeros(B, L, D, dtype=torch.float64, device="cuda")
    before = torch.zeros(B, L, D, dtype=torch.float64, device="cuda")
    for t in range(L):
        live = (n > t).double()[:, None]
        before[:, t] = h * live
        keep = torch.sigmoid(s["g"][:, t].double())
        h = torch.lerp(h, keep * h + (1 - keep) * s["x"][:, t].double(), live)
        y[:, t] = h * live
    if op == "gatedrec_fwd":
        return [y, h, before[:, ::CHUNK]]
    dx, dg = torch.zeros_like(y), torch.zeros_like(y)
    d = s["dh_last"].double()
    for t in range(L - 1, -1, -1):
        live = (n > t).double()[:, None]
        keep = torch.sigmoid(s["g"][:, t].double())
        d = d + s["dy"][:, t].double() * live
        dx[:, t] = (1 - keep) * d * live
        dg[:, t] = keep * (1 - keep) * (before[:, t] - s["x"][:, t].double()) * d * live
        d = torch.lerp(d, keep * d, live)
    return [dx, dg, d]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("layernorm"):
        return _exact_layernorm(s)
    if case["op"].startswith("rotary"):
        return _exact_rotary(s)
    return _exact_gatedrec(s)
