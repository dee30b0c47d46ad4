"""Host-only checks of the layer norm, rotary and gated recurrence entry points:
what the C ABI refuses before any launch, and what the binding refuses.  No
kernel is launched here."""
import ctypes

import numpy as np
import pytest
import torch

import linear_attention_lm_b200 as lab
from linear_attention_lm_b200 import build as lab_build
from oracle import layer

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 5
FAKE = 1 << 20  # a 16-byte-aligned non-null address; never dereferenced here
N = None


@pytest.fixture(scope="module")
def lib():
    lab_build.build()
    return lab.load_library()


def ln(lib, x=FAKE, res=N, w=FAKE, b=N, y=FAKE, r=N, mean=N, rstd=N, rows=4, D=64, dt=1, eps=1e-5):
    return lib.based_layernorm_fwd(x, res, w, b, y, r, mean, rstd, rows, D, dt, eps, N)


def test_layernorm_refusals(lib):
    assert ln(lib, rows=-1) == INVALID
    assert ln(lib, D=0) == INVALID
    assert ln(lib, dt=3) == INVALID
    assert ln(lib, D=16385) == UNSUPPORTED
    for eps in (0.0, -1e-5, float("nan"), float("inf")):
        assert ln(lib, eps=eps) == INVALID
    for name in ("x", "w", "y"):
        assert ln(lib, **{name: N}) == INVALID
    for name in ("x", "w", "b", "y", "mean", "rstd"):
        assert ln(lib, **{name: FAKE + 4}) == INVALID
    assert ln(lib, res=FAKE) == INVALID       # no place for the stream
    assert ln(lib, r=FAKE) == INVALID         # a stream without a residual
    assert ln(lib, res=FAKE, r=FAKE + 8) == INVALID
    assert ln(lib, x=N, w=N, y=N, rows=0) == OK


def lnb(lib, dy=FAKE, x=FAKE, w=FAKE, mean=FAKE, rstd=FAKE, dres=N, dx=FAKE, dw=FAKE, db=FAKE,
        rows=4, D=64, dt=1, ws=FAKE, nbytes=1 << 40):
    return lib.based_layernorm_bwd(dy, x, w, mean, rstd, dres, dx, dw, db, rows, D, dt, ws, nbytes, N)


def test_layernorm_gradient_refusals(lib):
    assert lnb(lib, rows=-1) == INVALID
    assert lnb(lib, D=0) == INVALID
    assert lnb(lib, dt=-1) == INVALID
    assert lnb(lib, D=20000) == UNSUPPORTED
    for name in ("dy", "x", "w", "mean", "rstd", "dx", "dw"):
        assert lnb(lib, **{name: N}) == INVALID
    for name in ("dy", "x", "w", "mean", "rstd", "dres", "dx", "dw", "db", "ws"):
        assert lnb(lib, **{name: FAKE + 4}) == INVALID
    need = lib.based_layernorm_bwd_workspace_bytes(4, 64)
    assert 0 < need <= 4 * 2 * 64 * 4
    assert lnb(lib, ws=N) == WORKSPACE
    assert lnb(lib, nbytes=need - 1) == WORKSPACE


def test_layernorm_workspace(lib):
    bad = ctypes.c_size_t(-1).value
    f = lib.based_layernorm_bwd_workspace_bytes
    assert f(-1, 64) == bad and f(4, 0) == bad and f(4, 16385) == bad
    assert f(0, 64) == 0
    # at most 512 parts of two rows of D sums, however many rows
    assert 0 < f(1 << 40, 16384) <= 512 * 2 * 16384 * 4
    with pytest.raises(lab.BasedError):
        lab.based_layernorm_bwd_workspace_bytes(-1, 64)


def rot(lib, q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, f=FAKE, pos=N, pos0=0, B=1, Hq=2, Hk=2, L=8, D=64,
        rot=64, layout=0, m=1.0, dt=1):
    return lib.based_rotary_fwd(q, k, qo, ko, f, pos, pos0, B, Hq, Hk, L, D, rot, layout, m, dt, N)


def test_rotary_refusals(lib):
    for kw in (dict(B=-1), dict(Hq=-1), dict(Hk=-1), dict(L=-1), dict(D=0), dict(rot=0),
               dict(rot=66), dict(rot=63), dict(layout=2), dict(dt=2), dict(m=float("nan")),
               dict(m=float("inf")), dict(pos0=-1), dict(q=N), dict(k=N), dict(qo=N), dict(ko=N),
               dict(f=N), dict(q=FAKE + 2), dict(ko=FAKE + 8), dict(f=FAKE + 4),
               dict(pos=FAKE + 4)):
        assert rot(lib, **kw) == INVALID, kw
    for kw in (dict(pos0=(1 << 31) - 7), dict(D=65538), dict(Hq=1 << 19), dict(B=1 << 21, L=1 << 21),
               dict(Hq=(1 << 31) - 1, Hk=(1 << 31) - 1)):
        assert rot(lib, **kw) == UNSUPPORTED, kw
    assert rot(lib, q=N, k=N, qo=N, ko=N, f=N, L=0) == OK
    assert rot(lib, q=N, k=N, qo=N, ko=N, f=N, Hq=0, Hk=0) == OK
    f = lib.based_rotary_bwd
    assert f(FAKE, FAKE, FAKE, N, FAKE, N, 0, 1, 2, 2, 8, 64, 64, 0, 1.0, N) == INVALID
    assert f(FAKE, FAKE, FAKE, FAKE, FAKE, N, -5, 1, 2, 2, 8, 64, 64, 0, 1.0, N) == INVALID


@pytest.mark.parametrize("rot_dim", [2, 64, 90, 128])
@pytest.mark.parametrize("kw", [dict(), dict(base=500000.0), dict(scaling="linear", factor=4.0),
                                dict(scaling="by_parts", factor=8.0, original_len=2048,
                                     low_turns=1.0, high_turns=4.0),
                                dict(scaling="by_parts", factor=32.0, original_len=8192,
                                     low_turns=0.5, high_turns=30.0)])
def test_rotary_frequencies(lib, rot_dim, kw):
    """pow against exp of a logarithm: a few steps of 2^-53 times the exponent's
    size, at most log(base) (13.2)."""
    got = lab.based_rotary_freqs(rot_dim, **kw).numpy()
    names = {"low_turns": "low", "high_turns": "high"}
    want = layer.rotary_freqs(rot_dim, **{names.get(n, n): v for n, v in kw.items()})
    assert np.max(np.abs(got / want - 1)) <= 64 * 2.0 ** -53


def test_rotary_frequency_refusals(lib):
    for kw in (dict(rot_dim=0), dict(rot_dim=7), dict(base=0.0), dict(base=float("inf")),
               dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=float("nan")),
               dict(scaling="by_parts", factor=2.0, original_len=0),
               dict(scaling="by_parts", factor=2.0, original_len=9, low_turns=4.0, high_turns=4.0)):
        with pytest.raises(lab.BasedError):
            lab.based_rotary_freqs(**{"rot_dim": 8, **kw})
    with pytest.raises(ValueError):
        lab.based_rotary_freqs(8, scaling="other")
    # a factor that the scaling does not use is not looked at
    assert lab.based_rotary_freqs(8, factor=0.0).shape == (4,)


def rec(lib, x=FAKE, g=FAKE, y=FAKE, h0=N, hl=N, hc=N, n=N, B=2, L=8, D=64, dt=1):
    return lib.based_gatedrec_fwd(x, g, y, h0, hl, hc, n, B, L, D, dt, N)


def recb(lib, x=FAKE, g=FAKE, dy=FAKE, hc=FAKE, dhl=N, dx=FAKE, dg=FAKE, dh0=N, n=N, B=2, L=8, D=64,
         dt=1):
    return lib.based_gatedrec_bwd(x, g, dy, hc, dhl, dx, dg, dh0, n, B, L, D, dt, N)


def test_gatedrec_refusals(lib):
    for f in (rec, recb):
        for kw in (dict(B=-1), dict(L=-1), dict(D=0), dict(dt=9), dict(x=N), dict(g=N),
                   dict(x=FAKE + 2), dict(n=FAKE + 4)):
            assert f(lib, **kw) == INVALID, kw
        assert f(lib, x=N, g=N, L=0, **({"y": N} if f is rec else
                                        dict(dy=N, hc=N, dx=N, dg=N))) == OK
        assert f(lib, B=1 << 30, L=0, D=1 << 20) == UNSUPPORTED
        assert f(lib, D=(1 << 20) + 1) == UNSUPPORTED
    for kw in (dict(y=N), dict(h0=FAKE + 4), dict(hl=FAKE + 4), dict(hc=FAKE + 4)):
        assert rec(lib, **kw) == INVALID, kw
    for kw in (dict(dy=N), dict(hc=N), dict(dx=N), dict(dg=N), dict(dhl=FAKE + 4),
               dict(dh0=FAKE + 4), dict(hc=FAKE + 4)):
        assert recb(lib, **kw) == INVALID, kw


def test_gatedrec_step_refusals(lib):
    f = lib.based_gatedrec_step
    assert f(FAKE, FAKE, FAKE, FAKE, -1, 64, 1, N) == INVALID
    assert f(FAKE, FAKE, FAKE, FAKE, 1, 0, 1, N) == INVALID
    assert f(FAKE, FAKE, FAKE, FAKE, 1, 64, 4, N) == INVALID
    assert f(FAKE, FAKE, N, FAKE, 1, 64, 1, N) == INVALID
    assert f(FAKE, FAKE, FAKE + 4, FAKE, 1, 64, 1, N) == INVALID
    assert f(N, N, N, N, 0, 64, 1, N) == OK


def test_binding_refuses_cpu_tensors():
    x, w, f = torch.zeros(2, 4, 8), torch.zeros(8), torch.zeros(4, dtype=torch.float64)
    h, x4 = torch.zeros(2, 8), torch.zeros(1, 2, 4, 8)
    for call in (lambda: lab.layernorm(x, w), lambda: lab.layernorm_grad(x, x, w, h, h),
                 lambda: lab.rotary(x4, x4, f), lambda: lab.rotary_grad(x4, None, f),
                 lambda: lab.gatedrec(x, x), lambda: lab.gatedrec_grad(x, x, x, x),
                 lambda: lab.gatedrec_step(h, h, h)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        lab.layernorm(None, w)
    with pytest.raises(TypeError):
        lab.rotary(None, None, f)
