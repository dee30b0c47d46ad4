"""The layer operators where their kernels take other paths than at the common sizes: odd
widths of the recurrence over many rounds, every cut of a sequence, the layer norm in place
at each of its row layouts.  Bounds and inputs are those of ``test_gpu_layer``."""
import pytest
import torch
from test_gpu_layer import DT, STEP, Out, f64, gen, masked, rec_bounds, rec_inputs, within

import linear_attention_lm_b200 as lab
from linear_attention_lm_b200 import build as lab_build
from oracle import layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lab_build.build()
    lab.load_library()
    torch.cuda.set_device(0)


# more rounds than the ring has slots: one CTA per sequence and channel block (the first two
# and the fourth, which has the widest blocks), clusters, and odd widths of each
REC_PATHS = [(8, 800, 1024), (8, 801, 999), (1, 9000, 333), (20, 600, 999), (2, 2500, 151)]


@pytest.mark.parametrize("B,L,D", REC_PATHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ragged", [False, True])
def test_gatedrec_over_many_rounds(B, L, D, dtype, ragged):
    x, g, n = rec_inputs(B, L, D, dtype, ragged)
    dy, h0, dh = gen(3, (B, L, D), dtype), gen(5, (B, D)), gen(6, (B, D))
    if ragged:
        for b in range(B):
            dy[b, int(n[b]):] = float("nan")
    out = Out()
    y, last = out((B, L, D), DT[dtype]), out((B, D), torch.float32)
    chunks = out((B, -(-L // 64), D), torch.float32)
    lab.based_gatedrec_fwd(x, g, y, h0, last, chunks, n)
    dx, dg = out((B, L, D), torch.float32), out((B, L, D), torch.float32)
    dh0 = out((B, D), torch.float32)
    lab.based_gatedrec_bwd(x, g, dy, chunks, dx, dg, dh, dh0, n)
    out.check()
    lens = None if n is None else n.tolist()
    a = [masked(t, n) for t in (x, g, dy)]
    ry, rl, rb = layer.gatedrec(a[0], a[1], f64(h0), lens)
    by, bl, bb = rec_bounds(a[0], a[1], f64(h0), lengths=lens)
    within(y, ry, STEP[dtype] * abs(ry) + 1.01 * by, "y")
    within(last, rl, bl, "h_last")
    within(chunks, rb[:, ::64], bb[:, ::64], "h_chunks")
    want = layer.gatedrec_grad(*a, f64(h0), f64(dh), lens)
    bx, bg, b0 = rec_bounds(a[0], a[1], f64(h0), a[2], f64(dh), lens)
    within(dx, want[0], bx + 2.0 ** -24 * abs(want[0]), "dx")
    within(dg, want[1], bg + 2.0 ** -24 * abs(want[1]), "dg")
    within(dh0, want[2], b0, "dh0")


# several rows to a warp, to a CTA and to each of several CTAs; rows that are whole vectors
# and rows that are not; the widest rows, which are not copied ahead
@pytest.mark.parametrize("rows,D", [(700, 1), (5000, 17), (3000, 100), (700, 999), (400, 1024),
                                    (200, 4100), (190, 8191), (190, 16383), (160, 16384)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layernorm_in_place_and_left_out(rows, D, dtype):
    """In place as documented, and with dbias or dresid left out: the bits of the calls
    that write elsewhere and ask for everything."""
    x, res, w = gen(1, (rows, D), dtype), gen(2, (rows, D), dtype, scale=2.0), gen(3, (D,), shift=1.0)
    y, r, mean, rstd = lab.layernorm(x, w, residual=res, return_stats=True)
    a, b = x.clone(), res.clone()
    lab.based_layernorm_fwd(a, w, None, a, residual=b, resid_out=b)
    assert torch.equal(a, y) and torch.equal(b, r)
    a, b = x.clone(), res.clone()
    lab.based_layernorm_fwd(a, w, None, b, residual=b, resid_out=a)
    assert torch.equal(b, y) and torch.equal(a, r)
    a = r.clone()
    lab.based_layernorm_fwd(a, w, None, a)
    assert torch.equal(a, y)
    dres = gen(4, (rows, D))
    dx, dw, db = lab.layernorm_grad(x, r, w, mean, rstd, dres)
    held = dres.clone()
    got = lab.based_layernorm_bwd(x, r, w, mean, rstd, held, torch.empty_like(dw), None, held)
    assert torch.equal(held, dx) and torch.equal(got[1], dw) and got[2] is None
    dx, dw, db = lab.layernorm_grad(x, r, w, mean, rstd)
    assert torch.equal(got[1], dw)
    plain = lab.based_layernorm_bwd(x, r, w, mean, rstd, torch.empty_like(dx), torch.empty_like(dw), None)
    assert torch.equal(plain[0], dx) and torch.equal(plain[1], dw)
    assert lab.based_get_device_error() == 0


def test_layernorm_odd_width_past_32_bits():
    """More than 2^31 elements in rows that start at any element: the last rows are what a
    call on them alone gives, bit for bit."""
    rows, D = (1 << 21) + (1 << 13) + 5, 1021
    x = torch.full((rows, D), 0.5, dtype=torch.bfloat16, device="cuda")
    tail = slice(rows - 64, rows)
    x[:64], x[tail] = gen(1, (64, D), "bf16"), gen(2, (64, D), "bf16")
    w = gen(3, (D,))
    y, mean, rstd = lab.layernorm(x, w, return_stats=True)
    for part in (slice(0, 64), tail):
        want = lab.layernorm(x[part].clone(), w, return_stats=True)
        assert all(torch.equal(a, b) for a, b in zip((y[part], mean[part], rstd[part]), want))
    del y
    dx, _, _ = lab.layernorm_grad(x, x, w, mean, rstd)
    for part in (slice(0, 64), tail):
        want = lab.layernorm_grad(x[part].clone(), x[part].clone(), w, mean[part].clone(), rstd[part].clone())
        assert torch.equal(dx[part], want[0])
    assert lab.based_get_device_error() == 0
