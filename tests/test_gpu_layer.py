"""GPU parity of layer norm, rotary positions and the gated recurrence through
the binding, against the fp64 oracle on the same inputs.

Tolerances are derived.  A rounding to bf16 is off by at most 2^-8 of the value,
one to fp32 by 2^-24.  Sums of the layer norm have at most 32 terms per thread,
then 5 shuffles, then at most 32 warps: fewer than 70 roundings in a row, taken
as 80 for a sum and the operations around it (U below).  The gated recurrence's
bound is a recursion of its own, beside its test."""
import numpy as np
import pytest
import torch

import linear_attention_lm_b200 as lab
import oracle
from linear_attention_lm_b200 import build as lab_build
from oracle import grad, layer

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U = 80 * 2.0 ** -24
GUARD = 64  # elements around every output that have to stay as they were


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lab_build.build()
    lab.load_library()
    torch.cuda.set_device(0)


def gen(seed, shape, dtype="f32", scale=1.0, shift=0.0):
    r = np.random.Generator(np.random.PCG64(seed))
    a = r.standard_normal(shape) * scale + shift
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(DT[dtype]).cuda()


def f64(t):
    return None if t is None else t.double().cpu().numpy()


class Out:
    """Outputs filled with 77 inside larger buffers; check() looks at the rims."""

    def __init__(self):
        self.all = []

    def __call__(self, shape, dtype):
        n = int(np.prod(shape))
        buf = torch.full((n + 2 * GUARD,), 77.0, dtype=dtype, device="cuda")
        self.all.append((buf, n))
        return buf[GUARD:GUARD + n].view(shape)

    def check(self):
        torch.cuda.synchronize()
        for buf, n in self.all:
            assert bool((buf[:GUARD] == 77).all()) and bool((buf[GUARD + n:] == 77).all())
        assert lab.based_get_device_error() == 0


def within(got, want, bound, name=""):
    got = f64(got) if torch.is_tensor(got) else got
    assert np.all(np.isfinite(got)), name
    bad = np.abs(got - want) - bound
    assert got.size == 0 or np.max(bad) <= 0, (name, np.max(bad), np.unravel_index(np.argmax(bad), bad.shape))


# ------------------------------------------------------------------ layer norm

def ln_stats(r):
    """|mean| and mean|r| of every row, over the row's deviation: the size of the
    rounding errors of r - mean."""
    return (np.abs(r.mean(-1)) + np.abs(r).mean(-1))[..., None]


LN_SIZES = [(3, 1), (5, 7), (1001, 17), (77, 33), (515, 100), (21, 400), (300, 64), (1, 250), (9, 256), (130, 257), (3, 999), (33, 1000),
            (64, 1024), (700, 1024), (7, 1028), (20, 2048), (5, 4100), (3, 8191), (4, 8192),
            (2, 16383), (3, 16384)]


@pytest.mark.parametrize("rows,D", LN_SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("residual,bias,shift", [(False, True, 0.0), (True, False, 0.0),
                                                 (True, True, 30.0)])
def test_layernorm(rows, D, dtype, residual, bias, shift):
    dt, eps = DT[dtype], 1e-5
    x, w = gen(rows, (rows, D), dtype, shift=shift), gen(D, (D,), scale=0.3, shift=1.0)
    b = gen(D + 1, (D,)) if bias else None
    res = gen(rows + 1, (rows, D), dtype, scale=2.0) if residual else None
    out = Out()
    y, mean, rstd = out((rows, D), dt), out((rows,), torch.float32), out((rows,), torch.float32)
    r = out((rows, D), dt) if residual else None
    lab.based_layernorm_fwd(x, w, b, y, eps, res, r, mean, rstd)
    out.check()
    stream = x
    if residual:
        want = torch.from_numpy(f64(x) + f64(res)).to(dt)
        assert torch.equal(r.cpu(), want)
        stream = r
    ref, m, s = layer.layernorm(f64(stream), f64(w), f64(b), eps)
    size = ln_stats(f64(stream))
    within(mean, m, U * size[..., 0], "mean")
    # d rstd = rstd^3 * (mean of z dz): dz is U size, so at most rstd^2 U size, and U of its own
    rel = (U + U * size * s[..., None])
    within(rstd, s, s * rel[..., 0], "rstd")
    sw = s[..., None] * np.abs(f64(w))
    free = np.abs(ref) if b is None else np.abs(ref) + np.abs(f64(b))
    within(y, ref, STEP[dtype] * np.abs(ref) + 1.01 * (2 * rel * free + U * size * sw), "y")


@pytest.mark.parametrize("rows,D", LN_SIZES + [(5000, 1024), (3000, 40), (2000, 999)])
@pytest.mark.parametrize("dtype,residual", [("bf16", False), ("bf16", True), ("f32", True)])
def test_layernorm_gradient(rows, D, dtype, residual):
    eps = 1e-5
    r = gen(rows, (rows, D), dtype, scale=2.0, shift=0.5)
    dy, w = gen(rows + 2, (rows, D), dtype), gen(D, (D,), scale=0.3, shift=1.0)
    dres = gen(rows + 3, (rows, D)) if residual else None
    _, mean, rstd = layer.layernorm(f64(r), f64(w), None, eps)
    out = Out()
    dx, dw, db = out((rows, D), torch.float32), out((D,), torch.float32), out((D,), torch.float32)
    lab.based_layernorm_bwd(dy, r, w, torch.tensor(mean, dtype=torch.float32).cuda(),
                            torch.tensor(rstd, dtype=torch.float32).cuda(), dx, dw, db, dres)
    out.check()
    dy64, w64, r64 = f64(dy), f64(w), f64(r)
    want = layer.layernorm_grad(dy64, r64, w64, eps, f64(dres))
    s = rstd[:, None]
    xh, t = (r64 - mean[:, None]) * s, dy64 * w64
    e_xh = U * (np.abs(xh) + s * ln_stats(r64))
    avg = lambda v: v.mean(-1, keepdims=True)  # noqa: E731
    along = avg(np.abs(t * xh))
    bound = s * (U * (np.abs(t) + avg(np.abs(t)) + np.abs(xh) * along) + e_xh * along +
                 np.abs(xh) * avg(np.abs(t) * e_xh)) + 2.0 ** -23 * (np.abs(want[0]))
    if residual:
        bound = bound + 2.0 ** -23 * np.abs(f64(dres))
    within(dx, want[0], bound, "dx")
    # a thread adds its rows one after another: at most `rows` roundings, then U's
    n = rows * 2.0 ** -24 + U
    within(dw, want[1], (np.abs(dy64) * e_xh + n * np.abs(dy64 * xh)).sum(0), "dw")
    within(db, want[2], n * np.abs(dy64).sum(0), "db")


def test_layernorm_gradient_against_differences():
    """<dx, d> against the oracle's forward along d: with a step of 1e-4 and third
    derivatives of size 1 each of the 600 values is about 1e-8 off, beside the
    kernel's own error (some U of the terms)."""
    rows, D = 6, 100
    x, w, dy, d = (f64(gen(i, s)) for i, s in enumerate([(rows, D), (D,), (rows, D), (rows, D)]))
    f = lambda z: float((layer.layernorm(z, w, None, 1e-5)[0] * dy).sum())  # noqa: E731
    want = (f(x + 1e-4 * d) - f(x - 1e-4 * d)) / 2e-4
    as32 = lambda a: torch.tensor(a, dtype=torch.float32).cuda()  # noqa: E731
    _, mean, rstd = lab.layernorm(as32(x), as32(w), return_stats=True)
    dx, _, _ = lab.layernorm_grad(as32(dy), as32(x), as32(w), mean, rstd)
    assert abs(float((f64(dx) * d).sum()) - want) <= U * np.abs(f64(dx) * d).sum() * 4 + 1e-5


def test_layernorm_special_rows():
    """A constant row has variance 0 and gives the bias; NaN and infinity stay in their row."""
    D = 300
    x = gen(1, (5, D), "bf16")
    x[1], x[2, 7], x[3, 0] = 3.0, float("nan"), float("inf")
    w, b = gen(2, (D,)), gen(3, (D,))
    y, mean, rstd = lab.layernorm(x, w, b, return_stats=True)
    assert torch.equal(y[1], b.bfloat16())
    assert bool(y[2].isnan().all()) and bool(y[3].isnan().any())
    clean = lab.layernorm(x[[0, 4]].contiguous(), w, b)
    assert torch.equal(y[[0, 4]], clean)


def test_layernorm_in_place_and_empty():
    x, res, w = gen(1, (50, 1024), "bf16"), gen(2, (50, 1024), "bf16"), gen(3, (1024,))
    y, r = lab.layernorm(x, w, residual=res)
    a, b = x.clone(), res.clone()
    lab.based_layernorm_fwd(a, w, None, a, residual=b, resid_out=b)
    assert torch.equal(a, y) and torch.equal(b, r)
    dres = gen(4, (50, 1024))
    _, mean, rstd = lab.layernorm(r, w, return_stats=True)
    dx, dw, db = lab.layernorm_grad(x, r, w, mean, rstd, dres)
    again = lab.based_layernorm_bwd(x, r, w, mean, rstd, dres, torch.empty_like(dw),
                                    torch.empty_like(db), dres)
    assert all(torch.equal(u, v) for u, v in zip((dx, dw, db), again))
    empty = x[:0]
    assert lab.layernorm(empty, w).shape == (0, 1024)
    dx, dw, db = lab.layernorm_grad(empty, empty, w, mean[:0], rstd[:0])
    assert not dw.any() and not db.any()


def test_layernorm_gradient_repeats_its_bits():
    r, dy, w = gen(1, (3000, 1024), "bf16"), gen(2, (3000, 1024), "bf16"), gen(3, (1024,))
    _, mean, rstd = lab.layernorm(r, w, return_stats=True)
    first = lab.layernorm_grad(dy, r, w, mean, rstd)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, lab.layernorm_grad(dy, r, w, mean, rstd)))


# ------------------------------------------------------------------ rotary

def rotary_bound(x, ref, freqs, pos, L, layout, mscale, dtype):
    """Angle: fp64 product and table 2^-50 of the turns (in radians), the fp32
    remainder, sine and products 2^-21; both values of a pair take part."""
    rot = 2 * len(freqs)
    start = np.broadcast_to(np.asarray(pos), (x.shape[0],)).reshape(-1, 1, 1, 1)
    turns = (start + np.arange(L).reshape(1, 1, -1, 1)) * freqs
    rel = abs(mscale) * (2.0 ** -21 + 2 * np.pi * turns * 2.0 ** -50)
    bound = STEP[dtype] * np.abs(ref)
    if layout == "half":
        both = np.abs(x[..., :rot // 2]) + np.abs(x[..., rot // 2:rot])
        bound[..., :rot // 2] += both * rel
        bound[..., rot // 2:rot] += both * rel
    else:
        both = np.abs(x[..., 0:rot:2]) + np.abs(x[..., 1:rot:2])
        bound[..., 0:rot:2] += both * rel
        bound[..., 1:rot:2] += both * rel
    return bound


@pytest.mark.parametrize("B,Hq,Hk,L,D,rot", [
    (2, 3, 3, 130, 64, 64), (1, 16, 16, 1, 128, 128), (3, 4, 1, 33, 128, 64), (2, 8, 2, 17, 96, 40),
    (1, 1, 1, 5, 7, 2), (2, 2, 1, 9, 90, 90), (2, 1, 2, 65, 80, 36), (1, 2, 2, 3, 256, 192),
    (130, 2, 2, 1, 64, 64), (1, 40, 9, 300, 64, 32)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("per_seq", [False, True])
def test_rotary(B, Hq, Hk, L, D, rot, layout, dtype, per_seq):
    freqs = lab.rotary_freqs(rot, scaling="by_parts", factor=4.0, original_len=512)
    q, k = gen(1, (B, Hq, L, D), dtype), gen(2, (B, Hk, L, D), dtype)
    r = np.random.Generator(np.random.PCG64(D))
    pos = r.integers(0, 2 ** 31 - L, B) if per_seq else 1000003
    on_gpu = torch.from_numpy(pos).cuda() if per_seq else pos
    out = Out()
    qo, ko = out(q.shape, q.dtype), out(k.shape, k.dtype)
    lab.based_rotary_fwd(q, k, qo, ko, freqs, on_gpu, layout, 1.25)
    out.check()
    f = f64(freqs)
    for got, x in ((qo, f64(q)), (ko, f64(k))):
        ref = layer.rotary(x, f, pos, layout, 1.25)
        within(got, ref, rotary_bound(x, ref, f, pos, L, layout, 1.25, dtype))
    lab.based_rotary_fwd(q, k, q, k, freqs, on_gpu, layout, 1.25)  # in place
    assert torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 32), (50, 30)])
def test_rotary_gradient(layout, D, rot):
    freqs = lab.rotary_freqs(rot)
    dq, dk = gen(1, (2, 4, 70, D)), gen(2, (2, 2, 70, D))
    out = Out()
    a, b = out(dq.shape, dq.dtype), out(dk.shape, dk.dtype)
    lab.based_rotary_bwd(dq, dk, a, b, freqs, 77, layout, 0.5)
    out.check()
    f = f64(freqs)
    for got, x in ((a, f64(dq)), (b, f64(dk))):
        ref = layer.rotary(x, f, 77, layout, 0.5, inverse=True)
        within(got, ref, rotary_bound(x, ref, f, 77, 70, layout, 0.5, "f32"))
    # against differences: the map is linear, so <R^T dq, d> = <dq, R d> without a step
    d = gen(3, dq.shape)
    along = f64(dq) * layer.rotary(f64(d), f, 77, layout, 0.5)
    terms = np.abs(f64(a) * f64(d)).sum() + np.abs(along).sum()
    assert abs((f64(a) * f64(d)).sum() - along.sum()) <= 2.0 ** -19 * terms


def test_rotary_one_of_the_two():
    freqs = lab.rotary_freqs(64)
    q, k = gen(1, (2, 4, 9, 64), "bf16"), gen(2, (2, 4, 9, 64), "bf16")
    both = lab.rotary(q, k, freqs, 3)
    assert torch.equal(lab.rotary(q, None, freqs, 3)[0], both[0])
    assert torch.equal(lab.rotary(None, k, freqs, 3)[1], both[1])
    assert lab.rotary(q[:, :, :0].contiguous(), None, freqs)[0].shape == (2, 4, 0, 64)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(64, 34), (64, 36), (126, 40), (51, 20)])
def test_rotary_passes_the_rest_bit_for_bit(layout, D, rot):
    """What is not turned is copied, infinities and NaN too, and stays out of what is."""
    x = gen(1, (2, 3, 9, D), "bf16")
    x[..., rot] = float("inf")
    x[0, :, :, rot + 1:] = float("nan")
    clean = x.clone()
    clean[..., rot:] = 0.0
    y = lab.rotary(x, None, lab.rotary_freqs(rot), 5, layout)[0]
    want = lab.rotary(clean, None, lab.rotary_freqs(rot), 5, layout)[0]
    assert torch.equal(y[..., :rot], want[..., :rot])
    assert torch.equal(y[..., rot:].view(torch.int16), x[..., rot:].view(torch.int16))


def test_rotary_position_out_of_range():
    """Sequences with a position outside [0, 2^31 - L] stay untouched and are reported."""
    freqs, L = lab.rotary_freqs(64), 5
    q = gen(1, (5, 2, L, 64), "bf16")
    pos = torch.tensor([4, -1, 2 ** 31 - L + 1, 2 ** 62, 2 ** 31 - L], device="cuda")
    qo = torch.full_like(q, 77.0)
    lab.based_rotary_fwd(q, None, qo, None, freqs, pos)
    assert lab.based_get_device_error() == 1
    assert lab.based_get_device_error() == 0
    assert bool((qo[1:4] == 77).all())
    good = torch.tensor([4, 0, 0, 0, 2 ** 31 - L], device="cuda")
    want = lab.rotary(q, None, freqs, good)[0]
    assert torch.equal(qo[[0, 4]], want[[0, 4]])


# ------------------------------------------------------------------ gated recurrence

def rec_bounds(x, g, h0, dy=None, dh=None, lengths=None):
    """Bounds of |h_t error|, and with dy of dx, dg, dh0.

    The smaller of a, 1 - a is off by tau of itself (2^x to 2^-22, its argument's
    rounding |g| 2^-23, a division to 2^-22), and the other by as much plus a
    rounding.  With H the recurrence of the absolute values, a step adds
    min(a, 1-a) tau (H_{t-1} + |x|) and at most eight roundings of a H + (1-a)|x|
    (two operations, and the partial products and sums of a scan in pieces)."""
    B, L, D = x.shape
    a, n = layer._gates(g)
    with np.errstate(invalid="ignore"):
        tau = 2.0 ** -20 + np.minimum(np.abs(g), 128.0) * 2.0 ** -22
    small = np.minimum(a, n) * tau
    live = np.ones((B, L)) if lengths is None else np.arange(L) < np.asarray(lengths)[:, None]
    H = np.zeros((B, D)) if h0 is None else np.abs(h0)
    E = np.zeros((B, D))
    Hs, Es, Hb, Eb = (np.zeros((B, L, D)) for _ in range(4))
    for t in range(L):
        on = live[:, t, None] > 0
        Hb[:, t], Eb[:, t] = np.where(on, H, 0), np.where(on, E, 0)
        ax = np.where(on, np.abs(x[:, t]), 0)
        H2 = a[:, t] * H + n[:, t] * ax
        E2 = a[:, t] * E + small[:, t] * (H + ax) + 8 * 2.0 ** -24 * H2
        H, E = np.where(on, H2, H), np.where(on, E2, E)
        Hs[:, t], Es[:, t] = np.where(on, H, 0), np.where(on, E, 0)
    if dy is None:
        return Es, E, Eb
    lam = np.zeros((B, D)) if dh is None else np.abs(dh)
    e = np.zeros((B, D))
    bx, bg = np.zeros((B, L, D)), np.zeros((B, L, D))
    r = 2.0 ** -22
    for t in range(L - 1, -1, -1):
        on = live[:, t, None] > 0
        l = lam + np.where(on, np.abs(dy[:, t]), 0)
        el = e + 4 * 2.0 ** -24 * l
        an, ax = a[:, t] * n[:, t], np.where(on, np.abs(x[:, t]), 0)
        bx[:, t] = np.where(on, n[:, t] * el + n[:, t] * (tau[:, t] + r) * l, 0)
        bg[:, t] = np.where(on, an * (el * (Hb[:, t] + ax) + l * Eb[:, t] +
                                      l * (Hb[:, t] + ax) * (2 * tau[:, t] + 2 * r)), 0)
        lam2 = a[:, t] * l
        e2 = a[:, t] * el + small[:, t] * l + 8 * 2.0 ** -24 * lam2
        lam, e = np.where(on, lam2, lam), np.where(on, e2, e)
    return bx, bg, e


REC_SIZES = [(1, 1, 1), (3, 2, 33), (2, 63, 64), (1, 64, 100), (2, 65, 1000), (4, 130, 256),
             (1, 700, 40), (1, 1025, 1024), (2, 257, 2050), (5, 31, 8), (1, 4100, 72), (40, 20, 64),
             (3, 3000, 24), (128, 40, 256), (150, 64, 130), (130, 17, 151), (9, 16, 21),
             (240, 100, 500)]


def rec_inputs(B, L, D, dtype, ragged):
    x = gen(B + L, (B, L, D), dtype)
    g = gen(L + D, (B, L, D), "f32")
    g = (g + torch.rand(D, generator=torch.Generator().manual_seed(D)).cuda() * 6).to(DT[dtype])
    n = None
    if ragged:
        n = torch.randint(0, L + 1, (B,), generator=torch.Generator().manual_seed(B)).cuda()
        n[0] = L
        if B > 1:
            n[-1] = 0
        for b in range(B):  # what lies past the end is not looked at
            x[b, int(n[b]):] = float("nan")
            g[b, int(n[b]):] = float("inf")
    return x, g, n


def masked(t, n):
    a = f64(t)
    if n is not None:
        for b in range(len(n)):
            a[b, int(n[b]):] = 0.0
    return a


@pytest.mark.parametrize("B,L,D", REC_SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ragged,start", [(False, False), (True, True)])
def test_gatedrec(B, L, D, dtype, ragged, start):
    x, g, n = rec_inputs(B, L, D, dtype, ragged)
    h0 = gen(5, (B, D)) if start else None
    out = Out()
    y, last = out((B, L, D), DT[dtype]), out((B, D), torch.float32)
    chunks = out((B, -(-L // 64), D), torch.float32)
    lab.based_gatedrec_fwd(x, g, y, h0, last, chunks, n)
    out.check()
    lens = None if n is None else n.tolist()
    x64, g64 = masked(x, n), masked(g, n)
    ry, rl, rb = layer.gatedrec(x64, g64, f64(h0), lens)
    by, bl, bb = rec_bounds(x64, g64, f64(h0), lengths=lens)
    within(y, ry, STEP[dtype] * np.abs(ry) + 1.01 * by, "y")
    within(last, rl, bl, "h_last")
    within(chunks, rb[:, ::64], bb[:, ::64], "h_chunks")


@pytest.mark.parametrize("B,L,D", REC_SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ragged,ends", [(False, False), (True, True)])
def test_gatedrec_gradient(B, L, D, dtype, ragged, ends):
    x, g, n = rec_inputs(B, L, D, dtype, ragged)
    dy = gen(3, (B, L, D), dtype)
    h0, dh = (gen(5, (B, D)), gen(6, (B, D))) if ends else (None, None)
    _, chunks = lab.gatedrec(x, g, h0, n, for_grad=True)
    if n is not None:
        for b in range(B):
            dy[b, int(n[b]):] = float("nan")
    out = Out()
    dx, dg, dh0 = out((B, L, D), torch.float32), out((B, L, D), torch.float32), out((B, D), torch.float32)
    lab.based_gatedrec_bwd(x, g, dy, chunks, dx, dg, dh, dh0, n)
    out.check()
    lens = None if n is None else n.tolist()
    a = [masked(t, n) for t in (x, g, dy)]
    want = layer.gatedrec_grad(*a, f64(h0), f64(dh), lens)
    bx, bg, b0 = rec_bounds(a[0], a[1], f64(h0), a[2], f64(dh), lens)
    within(dx, want[0], bx + 2.0 ** -24 * np.abs(want[0]), "dx")
    within(dg, want[1], bg + 2.0 ** -24 * np.abs(want[1]), "dg")
    within(dh0, want[2], b0, "dh0")


def test_gatedrec_gradient_against_differences():
    """Along a direction, against the oracle's forward: with a step of 1e-4 the 3600
    values are together less than 1e-5 off (1e-8 / 6 each, of either sign)."""
    B, L, D = 2, 150, 12
    x, g, dy, ex, eg = (f64(gen(i, (B, L, D))) for i in range(5))
    h0, dh, e0 = (f64(gen(9 + i, (B, D))) for i in range(3))

    def f(s):
        y, last, _ = layer.gatedrec(x + s * ex, g + s * eg, h0 + s * e0)
        return float((y * dy).sum() + (last * dh).sum())

    want = (f(1e-4) - f(-1e-4)) / 2e-4
    as32 = lambda a: torch.tensor(a, dtype=torch.float32).cuda()  # noqa: E731
    _, chunks = lab.gatedrec(as32(x), as32(g), as32(h0), for_grad=True)
    dx, dg, d0 = lab.gatedrec_grad(as32(x), as32(g), as32(dy), chunks, as32(dh))
    terms = [f64(dx) * ex, f64(dg) * eg, f64(d0) * e0]
    size = sum(np.abs(t).sum() for t in terms)
    assert abs(sum(t.sum() for t in terms) - want) <= 2.0 ** -18 * size + 1e-5


def test_gatedrec_special_gates():
    """Logits of infinity keep or replace the state exactly; huge ones do not overflow."""
    B, L, D = 1, 200, 64
    x, h0 = gen(1, (B, L, D)), gen(2, (B, D))
    g = torch.full((B, L, D), float("inf"), device="cuda")
    y, last = lab.gatedrec(x, g, h0, return_state=True)
    assert torch.equal(last, h0) and torch.equal(y, h0[:, None].expand(B, L, D))
    assert torch.equal(lab.gatedrec(x, -g, h0), x)
    for big in (100.0, 1e30):
        y = lab.gatedrec(x, torch.full_like(g, big), h0)
        assert torch.equal(y, h0[:, None].expand(B, L, D))
        assert torch.equal(lab.gatedrec(x, torch.full_like(g, -big), h0), x)
    g = gen(3, (B, L, D))
    g[:, 100] = -float("inf")  # starts anew: what came before has no part
    first = lab.gatedrec(x, g, h0)
    x[:, :100] += 5.0
    assert torch.equal(lab.gatedrec(x, g, h0)[:, 100:], first[:, 100:])


def test_gatedrec_empty():
    x = torch.empty(3, 0, 40, device="cuda")
    h0 = gen(1, (3, 40))
    y, last, chunks = lab.gatedrec(x, x, h0, return_state=True, for_grad=True)
    assert torch.equal(last, h0) and chunks.shape == (3, 0, 40)
    dx, dg, dh0 = lab.gatedrec_grad(x, x, x, chunks, h0)
    assert torch.equal(dh0, h0)


@pytest.mark.parametrize("L", [70, 14])
def test_gatedrec_length_out_of_range(L):
    x, g = gen(1, (4, L, 96), "bf16"), gen(2, (4, L, 96), "bf16")
    n = torch.tensor([L, L + 1, -1, L // 2], device="cuda")
    y, last = torch.full_like(x, 77.0), torch.full((4, 96), 77.0, device="cuda")
    chunks = torch.full((4, -(-L // 64), 96), 77.0, device="cuda")
    lab.based_gatedrec_fwd(x, g, y, None, last, chunks, n)
    assert lab.based_get_device_error() == 1
    assert bool((y[1:3] == 77).all() and (last[1:3] == 77).all() and (chunks[1:3] == 77).all())
    ok = torch.tensor([L, 0, 0, L // 2], device="cuda")
    wy, wl, wc = lab.gatedrec(x, g, None, ok, return_state=True, for_grad=True)
    for got, want in ((y, wy), (last, wl), (chunks, wc)):
        assert torch.equal(got[[0, 3]], want[[0, 3]])
    dx, dg = torch.full((4, L, 96), 77.0, device="cuda"), torch.full((4, L, 96), 77.0, device="cuda")
    dh0 = torch.full((4, 96), 77.0, device="cuda")
    lab.based_gatedrec_bwd(x, g, x, chunks, dx, dg, None, dh0, n)
    assert lab.based_get_device_error() == 1
    assert bool((dx[1:3] == 77).all() and (dg[1:3] == 77).all() and (dh0[1:3] == 77).all())
    assert lab.based_get_device_error() == 0


@pytest.mark.parametrize("B,D", [(1, 1), (3, 33), (128, 1024), (7, 100), (2, 2050)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gatedrec_step_continues_the_sequence(B, D, dtype):
    """Steps after a prefill against one pass of the oracle over all tokens."""
    L, n = 70, 5
    x, g = gen(1, (B, L + n, D), dtype), gen(2, (B, L + n, D), dtype)
    _, h = lab.gatedrec(x[:, :L].contiguous(), g[:, :L].contiguous(), return_state=True)
    ry, rl, _ = layer.gatedrec(f64(x), f64(g))
    by, bl, _ = rec_bounds(f64(x), f64(g), None)
    for t in range(L, L + n):
        y = lab.gatedrec_step(x[:, t].clone(), g[:, t].clone(), h)  # aligned copies
        within(y, ry[:, t], STEP[dtype] * np.abs(ry[:, t]) + 1.01 * by[:, t])
    within(h, rl, bl)


def test_gatedrec_state_in_place_and_bits():
    x, g = gen(1, (2, 900, 1024), "bf16"), gen(2, (2, 900, 1024), "bf16")
    h = gen(3, (2, 1024))
    first = lab.gatedrec(x, g, h, return_state=True, for_grad=True)
    grads = lab.gatedrec_grad(x, g, x, first[2], h)
    for _ in range(3):
        again = lab.gatedrec(x, g, h, return_state=True, for_grad=True)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        more = lab.gatedrec_grad(x, g, x, again[2], h)
        assert all(torch.equal(a, b) for a, b in zip(grads, more))
    state = h.clone()  # h_last may be h0, dh0 may be dh_last
    lab.based_gatedrec_fwd(x, g, torch.empty_like(x), state, state)
    assert torch.equal(state, first[1])
    lab.based_gatedrec_bwd(x, g, x, first[2], torch.empty_like(grads[0]), torch.empty_like(grads[1]),
                           h, h)
    assert torch.equal(h, grads[2])


def test_gatedrec_wait_runs_out_then_recovers():
    """One CTA of a cluster leaves out a send: the receiver gives up after 1 ms, the
    error is recorded, nothing faults, and the next call is as the first."""
    x, g = gen(1, (1, 6000, 64), "bf16"), gen(2, (1, 6000, 64), "bf16")
    first = lab.gatedrec(x, g, return_state=True, for_grad=True)
    grads = lab.gatedrec_grad(x, g, x, first[2])
    assert lab.based_get_device_error() == 0
    for call in (lambda: lab.gatedrec(x, g), lambda: lab.gatedrec_grad(x, g, x, first[2])):
        lab.based_debug_stall(lab.STALL_GATEDREC, 1_000_000)
        try:
            call()
            assert lab.based_get_device_error() == 4
        finally:
            lab.based_debug_stall(lab.STALL_NONE, 2_000_000_000)
    again = lab.gatedrec(x, g, return_state=True, for_grad=True)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    assert all(torch.equal(a, b) for a, b in zip(grads, lab.gatedrec_grad(x, g, x, first[2])))
    assert lab.based_get_device_error() == 0


# ------------------------------------------------------------------ together

def test_refusals_name_the_argument():
    x, w = gen(1, (4, 64), "bf16"), gen(2, (64,))
    with pytest.raises(TypeError, match="weight"):
        lab.layernorm(x, w.bfloat16())
    with pytest.raises(ValueError, match="weight"):
        lab.layernorm(x, w[:32])
    with pytest.raises(ValueError, match="contiguous"):
        lab.layernorm(x.t().contiguous().t(), w)
    with pytest.raises(TypeError):
        lab.layernorm(x.half(), w)
    with pytest.raises(lab.BasedError):
        lab.layernorm(x, w, eps=0.0)
    with pytest.raises(ValueError, match="together"):
        lab.based_layernorm_fwd(x, w, None, x, residual=x)
    q, f = gen(1, (1, 2, 4, 64), "bf16"), lab.rotary_freqs(64)
    with pytest.raises(TypeError, match="freqs"):
        lab.rotary(q, None, f.float())
    with pytest.raises(ValueError, match="layout"):
        lab.rotary(q, None, f, layout="other")
    with pytest.raises(ValueError, match="k:"):
        lab.rotary(q, gen(1, (1, 2, 5, 64), "bf16"), f)
    with pytest.raises(TypeError, match="k"):
        lab.rotary(q, q.float(), f)
    with pytest.raises(TypeError, match="pos"):
        lab.rotary(q, None, f, torch.tensor([0], dtype=torch.int32, device="cuda"))
    with pytest.raises(lab.BasedError):
        lab.rotary(q, None, lab.rotary_freqs(66))
    with pytest.raises(TypeError):
        lab.rotary_grad(q, None, f)
    a = gen(1, (2, 5, 64), "bf16")
    with pytest.raises(TypeError, match="g"):
        lab.gatedrec(a, a.float())
    with pytest.raises(ValueError, match="h0"):
        lab.gatedrec(a, a, gen(1, (1, 64)))
    with pytest.raises(ValueError, match="lengths"):
        lab.gatedrec(a, a, lengths=torch.tensor([5], device="cuda"))
    with pytest.raises(TypeError, match="h:"):
        lab.gatedrec_step(a[:, 0].contiguous(), a[:, 1].contiguous(), a[:, 2].contiguous())


def test_calls_on_two_streams_and_in_a_graph():
    """The same calls on two side streams at once, then captured and replayed on new
    inputs: the bits of the plain calls."""
    w, freqs = gen(1, (1024,)), lab.rotary_freqs(64)
    sets = []
    for i in range(3):
        x, g = gen(10 + i, (2, 300, 1024), "bf16"), gen(20 + i, (2, 300, 1024), "bf16")
        q, h = gen(30 + i, (2, 4, 300, 64), "bf16"), gen(40 + i, (2, 1024))
        sets.append((x, g, q, h))

    def calls(x, g, q, h, stream=None):
        y, r, mean, rstd = lab.layernorm(x, w, residual=g, return_stats=True, stream=stream)
        dx, dw, db = lab.layernorm_grad(x, r, w, mean, rstd, stream=stream)
        qo, ko = lab.rotary(q, q, freqs, 5, stream=stream)
        a, last, chunks = lab.gatedrec(y, g, h, return_state=True, for_grad=True, stream=stream)
        d = lab.gatedrec_grad(y, g, x, chunks, h, stream=stream)
        return [y, r, mean, rstd, dx, dw, db, qo, ko, a, last, chunks, *d]

    plain = [[t.clone() for t in calls(*s)] for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [calls(*s, stream=st) for s, st in zip(sets, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, plain):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    held = [t.clone() for t in sets[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(*held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls(*held)
    for k in (1, 2, 0, 2):
        for dst, src in zip(held, sets[k]):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(outs, plain[k]))
    assert lab.based_get_device_error() == 0


def test_a_layer_and_its_gradient():
    """norm -> projections -> rotary -> window attention, and norm -> projections ->
    gated recurrence, with the gradients of both mixers down to their inputs; each
    step is compared with the oracle on the step's own inputs.  The bounds of the
    projections and of the attention are those of their own tests."""
    B, L, C, H, W = 2, 150, 256, 4, 64
    x, res = gen(1, (B, L, C), "bf16"), gen(2, (B, L, C), "bf16")
    w, b = gen(3, (C,), scale=0.2, shift=1.0), gen(4, (C,), scale=0.2)
    y, r, mean, rstd = lab.layernorm(x, w, b, residual=res, return_stats=True)
    ref, _, s = layer.layernorm(f64(r), f64(w), f64(b), 1e-5)
    within(y, ref, STEP["bf16"] * np.abs(ref) + 16 * U * (1 + np.abs(ref)), "norm")
    wq = gen(5, (3 * H * 64, C), "bf16", scale=0.05)
    q, k, v = lab.proj_heads_multi(y, wq, H, (64, 64, 64))
    freqs = lab.rotary_freqs(64)
    qr, kr = lab.rotary(q, k, freqs)
    f = f64(freqs)
    for got, src in ((qr, f64(q)), (kr, f64(k))):
        want = layer.rotary(src, f, 0, "half")
        within(got, want, rotary_bound(src, want, f, 0, L, "half", 1.0, "bf16"), "rotary")
    out = lab.window_attn(qr, kr, v, W)
    want = np.asarray(oracle.window_attn(f64(qr), f64(kr), f64(v), W))
    assert np.linalg.norm(f64(out) - want) <= 5e-3 * np.linalg.norm(want)
    dout = gen(6, out.shape, "bf16")
    dqr, dkr, dv = lab.window_grad(qr, kr, v, dout, W)
    dq, dk = lab.rotary_grad(dqr, dkr, freqs)
    gq, gk, gv = grad.window_grad(f64(qr), f64(kr), f64(v), f64(dout), W)
    for got, g_ref in ((dq, gq), (dk, gk)):
        want = layer.rotary(g_ref, f, 0, "half", inverse=True)
        assert np.linalg.norm(f64(got) - want) <= 1e-2 * np.linalg.norm(want)
    # the recurrence beside it: the projection with one "head" gives [B, 1, L, C]
    wg = gen(7, (2 * C, C), "bf16", scale=0.1)
    xi, gi = (t.view(B, L, C) for t in lab.proj_heads_multi(y, wg, 1, (C, C)))
    hy, last, chunks = lab.gatedrec(xi, gi, return_state=True, for_grad=True)
    ry, rl, _ = layer.gatedrec(f64(xi), f64(gi))
    by, bl, _ = rec_bounds(f64(xi), f64(gi), None)
    within(hy, ry, STEP["bf16"] * np.abs(ry) + 1.01 * by, "recurrence")
    within(last, rl, bl, "state")
    dhy = gen(8, hy.shape, "bf16")
    dxi, dgi, _ = lab.gatedrec_grad(xi, gi, dhy, chunks)
    want = layer.gatedrec_grad(f64(xi), f64(gi), f64(dhy))
    bx, bg, _ = rec_bounds(f64(xi), f64(gi), None, f64(dhy))
    within(dxi, want[0], bx + 2.0 ** -24 * np.abs(want[0]), "dx")
    within(dgi, want[1], bg + 2.0 ** -24 * np.abs(want[1]), "dg")
    # through the projections (torch products) and back through the norm
    dy = torch.cat([dxi, dgi], -1).bfloat16().reshape(B * L, 2 * C) @ wg
    dy = dy.view(B, L, C)
    dres = gen(9, (B, L, C))
    dr, dw, db = lab.layernorm_grad(dy, r, w, mean, rstd, dres)
    want = layer.layernorm_grad(f64(dy), f64(r), f64(w), 1e-5, f64(dres))
    for got, ref in zip((dr, dw, db), want):
        assert np.linalg.norm(f64(got) - ref) <= 2.0 ** -15 * np.linalg.norm(ref)
    assert lab.based_get_device_error() == 0


def test_offsets_past_32_bits():
    """Tensors of over 2^31 elements: what lies at their ends is what a call on the
    ends alone gives, bit for bit."""
    def fill(shape, seed, dtype=torch.bfloat16):
        g = torch.Generator(device="cuda").manual_seed(seed)
        t = torch.empty(shape, dtype=dtype, device="cuda")
        flat = t.view(-1)
        flat[:1 << 20].normal_(generator=g)
        flat[-(1 << 28):].normal_(generator=g)
        flat[1 << 20:-(1 << 28)] = 0.5
        return t

    rows, D = (1 << 21) + 5, 1024
    x, w = fill((rows, D), 1), gen(2, (D,))
    y, mean, rstd = lab.layernorm(x, w, return_stats=True)
    for part in (slice(0, 64), slice(rows - 64, rows)):
        want = lab.layernorm(x[part].contiguous(), w, return_stats=True)
        assert all(torch.equal(a, b) for a, b in zip((y[part], mean[part], rstd[part]), want))
    del y
    dx, _, _ = lab.layernorm_grad(x, x, w, mean, rstd)
    tail = slice(rows - 64, rows)
    want = lab.layernorm_grad(x[tail].contiguous(), x[tail].contiguous(), w,
                              mean[tail].clone(), rstd[tail].clone())[0]
    assert torch.equal(dx[tail], want)
    del x, dx
    freqs, L = lab.rotary_freqs(128), (1 << 20) + 8
    q = fill((1, 17, L, 128), 3)
    out = lab.rotary(q, None, freqs, 7)[0]
    assert torch.equal(out[:, -1:], lab.rotary(q[:, -1:].contiguous(), None, freqs, 7)[0])
    del q, out
    L, D, last = (1 << 20) + (1 << 14), 2048, 1 << 16
    x, g = fill((1, L, D), 4), fill((1, L, D), 5)
    y, h, chunks = lab.gatedrec(x, g, return_state=True, for_grad=True)
    cut = L - last
    tail = [t[:, cut:].contiguous() for t in (x, g)]
    yt, ht, ct = lab.gatedrec(*tail, chunks[:, cut // 64].contiguous(), return_state=True,
                              for_grad=True)
    assert torch.equal(y[:, cut:], yt) and torch.equal(h, ht)
    assert torch.equal(chunks[:, cut // 64:], ct)
    del yt, y
    dx, dg, _ = lab.gatedrec_grad(x, g, x, chunks)
    del g
    want = lab.gatedrec_grad(*tail, tail[0], ct)
    assert torch.equal(dx[:, cut:], want[0]) and torch.equal(dg[:, cut:], want[1])
    assert lab.based_get_device_error() == 0


def test_raw_stream_handles_and_workspaces():
    """A stream given by its handle, and a workspace of the caller's, give the same bits."""
    x, w = gen(1, (300, 1000), "bf16"), gen(2, (1000,))
    _, mean, rstd = lab.layernorm(x, w, return_stats=True)
    want = lab.layernorm_grad(x, x, w, mean, rstd)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    nbytes = lab.based_layernorm_bwd_workspace_bytes(300, 1000)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(t) for t in want]
    lab.based_layernorm_bwd(x, x, w, mean, rstd, *outs, workspace=ws, stream=side.cuda_stream)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    with pytest.raises(lab.BasedError):
        lab.based_layernorm_bwd(x, x, w, mean, rstd, *outs, workspace=ws[:nbytes - 16])
