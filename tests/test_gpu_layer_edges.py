"""Edges of the layer operators on the GPU: values that are not finite, gates close to 1,
and widths and paths that only some sizes reach."""
import numpy as np
import pytest
import torch

import linear_attention_lm_b200 as lab
from linear_attention_lm_b200 import build as lab_build

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lab_build.build()
    lab.load_library()
    torch.cuda.set_device(0)


def normal(seed, shape, dtype="f32", scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(DT[dtype])


def spread_lengths(B, L):
    """Lengths of a padded batch, none of them a whole number of tiles but the first."""
    return torch.tensor([L] + [(L * (2 * b + 1) // (2 * B)) | 1 for b in range(1, B)], device="cuda")


# one thread per two channels (the first three), tiles with one and several rounds, odd
# widths, several CTAs per sequence
REC_SHAPES = [(4, 14, 64), (5, 9, 33), (128, 40, 256), (4, 130, 256), (3, 700, 33), (2, 3000, 24),
              (8, 1500, 1024)]


@pytest.mark.parametrize("B,L,D", REC_SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_gatedrec_gradient_padding_is_zero_beside_a_bad_final_gradient(B, L, D, dtype, bad):
    """dx and dg are zero past a sequence's length also where dh_last is not finite, and
    the other channels have the bits that they have without it."""
    x, g, dy = (normal(i, (B, L, D), dtype) for i in range(3))
    dh, n = normal(4, (B, D)), spread_lengths(B, L)
    _, chunks = lab.gatedrec(x, g, None, n, for_grad=True)
    want = lab.gatedrec_grad(x, g, dy, chunks, dh, n)
    dh2 = dh.clone()
    dh2[:, 1::7] = bad
    dx, dg, dh0 = lab.gatedrec_grad(x, g, dy, chunks, dh2, n)
    past = torch.arange(L, device="cuda")[None, :] >= n[:, None]
    assert not dx[past].any() and not dg[past].any()
    clean = torch.ones(D, dtype=torch.bool, device="cuda")
    clean[1::7] = False
    for a, b in zip((dx, dg, dh0), want):
        assert torch.equal(a[..., clean], b[..., clean])
    assert lab.based_get_device_error() == 0


# ------------------------------------------------------------------ slow decays

def slow_gates(D, dtype):
    """Logits of 11 to 17.  In fp32 the first half lies where 1 - a is halfway between two
    multiples of 2^-24, the spacing of fp32 below 1: a rounded a is worst there."""
    k = np.arange(D // 2)
    n = (k % 90 + 1.5) * 2.0 ** -24
    g = np.concatenate([np.log1p(-n) - np.log(n), np.linspace(11.0, 17.0, D - D // 2)])
    return torch.from_numpy(g.astype(np.float32)).to(DT[dtype])


def rates(g):
    """1 - a in fp64, and the kernels' relative error of it: 2^x to 2^-22, its argument's
    rounding |g| 2^-23, a division to 2^-22."""
    g = g.double().cpu().numpy()
    return np.exp(-g) / (1 + np.exp(-g)), 2.0 ** -20 + np.abs(g) * 2.0 ** -22


SLOW = [(1, 16384, 64), (8, 4096, 1024), (2, 5000, 33), (1, 9000, 333), (60, 512, 1024)]


@pytest.mark.parametrize("B,L,D", SLOW)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gatedrec_slow_decay_keeps_its_rate(B, L, D, dtype):
    """From a state of 1, with x = 0 the state decays to (1 - n)^L, with x = 1 it stays 1;
    and a final gradient of 1 decays to (1 - n)^L.

    The state stays in (1/2, 1], where an fp32 rounding is at most 2^-25.  A lane of S
    tokens (32 bytes of x forward, 16 backward) rounds its product of gates once, joins
    maps once and rounds the state once for each warp or lane group: 2^-25 twice per S
    tokens.  What a product leaves out is summed to S 2^-24 of itself, and the tokens of
    the last lane are walked with a rounding of a and of the state each."""
    size = 2 if dtype == "bf16" else 4
    gates = slow_gates(D, dtype)
    n, tau = rates(gates)
    g = gates.cuda().expand(B, L, D).contiguous()
    zero, one = torch.zeros(B, L, D, dtype=DT[dtype], device="cuda"), torch.ones(B, D, device="cuda")
    want = np.exp(L * np.log1p(-n))

    def bound(S, rate_error=True):
        steps = L * 2.0 ** -24 / S + L * n * S * 2.0 ** -24 + 2 * S * 2.0 ** -24
        return steps + (L * n * tau if rate_error else 0.0)

    _, last, chunks = lab.gatedrec(zero, g, one, return_state=True, for_grad=True)
    off = np.abs(last.double().cpu().numpy() - want) - bound(32 // size)
    assert off.max() <= 0, off.max()
    _, last = lab.gatedrec(torch.ones_like(zero), g, one, return_state=True)
    off = np.abs(last.double().cpu().numpy() - 1.0) - bound(32 // size, False)
    assert off.max() <= 0, off.max()
    _, _, dh0 = lab.gatedrec_grad(zero, g, zero, chunks, one)
    off = np.abs(dh0.double().cpu().numpy() - want) - bound(16 // size)
    assert off.max() <= 0, off.max()


@pytest.mark.parametrize("B,L,D", [(128, 48, 1024), (3, 16, 333), (4, 15, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gatedrec_slow_decay_keeps_its_rate_in_short_sequences(B, L, D, dtype):
    """The same where a thread walks the tokens: one rounding of the state per token, of at
    most 2^-25 as it lies in (1/2, 1], and what is added to it first is rounded to 2^-24
    of n."""
    gates = slow_gates(D, dtype)
    n, tau = rates(gates)
    g = gates.cuda().expand(B, L, D).contiguous()
    zero = torch.zeros(B, L, D, dtype=DT[dtype], device="cuda")
    start = 0.6 + 0.39 * torch.rand(B, D, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    bound = L * (2.0 ** -25 + n * (tau + 2.0 ** -23))
    want = start.double().cpu().numpy() * np.exp(L * np.log1p(-n))
    _, last, chunks = lab.gatedrec(zero, g, start, return_state=True, for_grad=True)
    off = np.abs(last.double().cpu().numpy() - want) - bound
    assert off.max() <= 0, off.max()
    _, _, dh0 = lab.gatedrec_grad(zero, g, zero, chunks, start)
    off = np.abs(dh0.double().cpu().numpy() - want) - bound
    assert off.max() <= 0, off.max()


@pytest.mark.parametrize("B,D", [(64, 1024), (5, 33)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gatedrec_step_rounds_once(B, D, dtype):
    """The new state is the exact one, rounded once: half a step of fp32 at its size, and
    n (|h| + |x|) times the gate's error and the roundings of n x and of what is added."""
    gates = slow_gates(D, dtype)
    n, tau = rates(gates)
    h = 1 + torch.rand(B, D, generator=torch.Generator("cuda").manual_seed(2), device="cuda")
    x, g = normal(3, (B, D), dtype), gates.cuda().expand(B, D).contiguous()
    h64, x64 = h.double().cpu().numpy(), x.double().cpu().numpy()
    lab.gatedrec_step(x, g, h)
    want = h64 + n * (x64 - h64)
    bound = np.spacing(np.float32(want) * np.float32(1 + 2.0 ** -20)) / 2 + n * (np.abs(h64) + np.abs(x64)) * (tau + 2.0 ** -22)
    off = np.abs(h.double().cpu().numpy() - want) - bound
    assert off.max() <= 0, off.max()


# ------------------------------------------------------------------ values that are not finite

@pytest.mark.parametrize("B,L,D", REC_SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gatedrec_bad_values_stay_in_their_channel(B, L, D, dtype):
    """An infinite or NaN x, a NaN logit and an infinite first state: other channels and
    sequences, the tokens before, and the padding keep their bits."""
    x, g, dy = (normal(i, (B, L, D), dtype) for i in range(3))
    h0, n = normal(4, (B, D)), spread_lengths(B, L)
    y, last, chunks = lab.gatedrec(x, g, h0, n, return_state=True, for_grad=True)
    grads = lab.gatedrec_grad(x, g, dy, chunks, None, n)
    t = int(n[1]) // 2  # inside the first two sequences
    x2, g2, h2 = x.clone(), g.clone(), h0.clone()
    x2[0, t, 0::5], g2[1, t, 2::5], h2[1, 4::5] = float("inf"), float("nan"), float("inf")
    x2[1, t, 0::5] = float("nan")
    y2, last2, chunks2 = lab.gatedrec(x2, g2, h2, n, return_state=True, for_grad=True)
    more = lab.gatedrec_grad(x2, g2, dy, chunks2, None, n)
    past = torch.arange(L, device="cuda")[None, :] >= n[:, None]
    bad = torch.zeros(B, 1, D, dtype=torch.bool, device="cuda")
    bad[:2, :, 0::5] = bad[1, :, 2::5] = bad[1, :, 4::5] = True
    before = torch.arange(L, device="cuda")[None, :, None] < t
    before = before.expand(B, L, D).clone()
    before[1, :, 4::5] = False  # a bad first state
    same = ~bad | before | past[..., None]
    assert torch.equal(y2[same], y[same])
    assert torch.equal(last2[~bad[:, 0]], last[~bad[:, 0]])
    assert torch.equal(chunks2[~bad.expand_as(chunks)], chunks[~bad.expand_as(chunks)])
    for a, b in zip(more[:2], grads[:2]):
        assert torch.equal(a[(~bad | past[..., None])], b[(~bad | past[..., None])])
    assert torch.equal(more[2][~bad[:, 0]], grads[2][~bad[:, 0]])
    assert not y2[past].any() and not more[0][past].any() and not more[1][past].any()
    assert lab.based_get_device_error() == 0


def test_layernorm_largest_values():
    """|r| of 7e16 at the widest rows: the squares' sum stays below fp32's largest.  A row
    of ones and minus ones scaled by it gives the row's own norm, up to the roundings of
    two sums of at most 80 steps (as in the parity test) on either side."""
    for D in (64, 999, 16384):
        x = torch.ones(3, D, device="cuda")
        x[:, ::2] = -1.0
        w, b = torch.ones(D, device="cuda"), torch.zeros(D, device="cuda")
        want = lab.layernorm(x, w, b, eps=1e-12)
        got = lab.layernorm(x * 7e16, w, b, eps=1e-12)
        assert float((got - want).abs().max()) <= 4 * 80 * 2.0 ** -24
