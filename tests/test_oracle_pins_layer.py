"""Pins of the fp64 layer norm, rotary positions and gated recurrence of
``oracle/layer.py`` (CPU): torch's fp64 functions, finite differences, closed
forms.

Difference quotients: a central difference of step h = 1e-5 of a smooth function
of values of size 1 is off by about h^2 |f'''| / 6 + 2^-52 |f| / h, some 1e-10;
5e-8 of the largest gradient leaves room for the derivatives of 1 / sqrt."""
import math

import numpy as np
import pytest
import torch

from oracle import layer


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def numeric(f, a, h=1e-5):
    """Gradient of the scalar f() with respect to the array a, changed in place."""
    out = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + h
        up = f()
        a[i] = keep - h
        out[i] = (up - f()) / (2 * h)
        a[i] = keep
    return out


def close(got, want, tol=5e-8):
    assert np.max(np.abs(got - want)) <= tol * max(1.0, np.max(np.abs(want)))


@pytest.mark.parametrize("rows,D", [(1, 1), (3, 7), (5, 64)])
def test_layernorm_is_torchs(rows, D):
    r = rng(rows)
    x, w, b = r.standard_normal((rows, D)), r.standard_normal(D), r.standard_normal(D)
    y, mean, rstd = layer.layernorm(x, w, b, 1e-5)
    want = torch.nn.functional.layer_norm(torch.tensor(x), (D,), torch.tensor(w), torch.tensor(b),
                                          1e-5).numpy()
    assert np.max(np.abs(y - want)) <= 1e-13 * max(1.0, np.max(np.abs(want)))
    assert np.allclose(mean, x.mean(1)) and np.allclose(rstd, (x.var(1) + 1e-5) ** -0.5)


def test_layernorm_gradient_is_its_differences():
    r = rng(3)
    x, w, b, dy = (r.standard_normal(s) for s in ((4, 9), (9,), (9,), (4, 9)))
    dres = r.standard_normal((4, 9))
    f = lambda: float((layer.layernorm(x, w, b, 1e-3)[0] * dy).sum() + (dres * x).sum())  # noqa: E731
    dx, dw, db = layer.layernorm_grad(dy, x, w, 1e-3, dres)
    close(dx, numeric(f, x))
    close(dw, numeric(f, w))
    close(db, numeric(f, b))


def test_rotary_closed_forms():
    freqs = layer.rotary_freqs(4)
    assert np.allclose(freqs * 2 * math.pi, [1.0, 0.01], rtol=1e-15)
    x = np.zeros((1, 1, 3, 6))
    x[..., 0], x[..., 1], x[..., 4], x[..., 5] = 1.0, 1.0, 7.0, 8.0
    y = layer.rotary(x, freqs, 5, "half")       # pairs (0, 2), (1, 3)
    z = layer.rotary(x, freqs, 5, "interleaved")  # pairs (0, 1), (2, 3)
    for t in range(3):
        p = 5 + t
        assert np.allclose(y[0, 0, t], [math.cos(p), math.cos(0.01 * p), math.sin(p),
                                        math.sin(0.01 * p), 7, 8], atol=1e-13)
        assert np.allclose(z[0, 0, t], [math.cos(p) - math.sin(p), math.sin(p) + math.cos(p),
                                        0, 0, 7, 8], atol=1e-13)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_depends_on_distance_and_inverts(layout):
    r = rng(5)
    q, k = r.standard_normal((2, 2, 1, 3, 8))
    freqs = layer.rotary_freqs(8)
    dots = [np.sum(layer.rotary(q, freqs, [p, p + 1], layout) *
                   layer.rotary(k, freqs, [p - 3, p + 4], layout), -1) for p in (3, 40000)]
    assert np.max(np.abs(dots[0] - dots[1])) <= 1e-10  # 40000 turns of a 2^-53 table
    back = layer.rotary(layer.rotary(q, freqs, 9, layout, 1.5), freqs, 9, layout, 1.5, inverse=True)
    assert np.max(np.abs(back - 2.25 * q)) <= 1e-13
    dy = r.standard_normal(q.shape)  # the inverse is the gradient: <dy, R q> = <R^T dy, q>
    assert abs(np.sum(dy * layer.rotary(q, freqs, 9, layout, 1.5)) -
               np.sum(layer.rotary(dy, freqs, 9, layout, 1.5, inverse=True) * q)) <= 1e-12


def test_rotary_scalings():
    plain = layer.rotary_freqs(64)
    assert np.allclose(layer.rotary_freqs(64, scaling="linear", factor=8.0), plain / 8, rtol=1e-15)
    parts = layer.rotary_freqs(64, scaling="by_parts", factor=8.0, original_len=2048)
    n = plain * 2048
    assert np.array_equal(parts[n >= 4], plain[n >= 4])
    assert np.allclose(parts[n <= 1], plain[n <= 1] / 8, rtol=1e-15)
    mid = (n > 1) & (n < 4)
    assert mid.any() and np.all(parts[mid] < plain[mid]) and np.all(parts[mid] > plain[mid] / 8)


def test_gatedrec_closed_forms():
    x = rng(7).standard_normal((2, 6, 3))
    h0 = rng(8).standard_normal((2, 3))
    inf = np.full_like(x, np.inf)
    assert np.array_equal(layer.gatedrec(x, -inf, h0)[0], x)
    y, last, before = layer.gatedrec(x, inf, h0)
    assert np.array_equal(y, np.repeat(h0[:, None], 6, 1)) and np.array_equal(last, h0)
    assert np.array_equal(before, y)
    # a = 1/2 everywhere: h_t = sum 2^-(t-s+1) x_s + 2^-(t+1) h0
    y = layer.gatedrec(x, np.zeros_like(x), h0)[0]
    want = sum(2.0 ** -(5 - s + 1) * x[:, s] for s in range(6)) + 2.0 ** -6 * h0
    assert np.allclose(y[:, 5], want, rtol=1e-14)


def test_gatedrec_continues_and_stops_at_its_length():
    r = rng(9)
    x, g, h0 = r.standard_normal((3, 11, 4)), r.standard_normal((3, 11, 4)), r.standard_normal((3, 4))
    y, last, _ = layer.gatedrec(x, g, h0)
    y0, mid, _ = layer.gatedrec(x[:, :5], g[:, :5], h0)
    y1, end, _ = layer.gatedrec(x[:, 5:], g[:, 5:], mid)
    assert np.array_equal(np.concatenate([y0, y1], 1), y) and np.array_equal(end, last)
    x[1, 5:], g[1, 5:] = np.nan, np.nan
    yr, lr, br = layer.gatedrec(x, g, h0, [11, 5, 0])
    assert np.array_equal(yr[1, :5], y[1, :5]) and not yr[1, 5:].any() and not br[2].any()
    assert np.array_equal(lr[1], mid[1]) and np.array_equal(lr[2], h0[2])


@pytest.mark.parametrize("lengths", [None, [5, 0, 3]])
def test_gatedrec_gradient_is_its_differences(lengths):
    r = rng(11)
    x, g, dy = r.standard_normal((3, 3, 5, 2))
    h0, dh = r.standard_normal((2, 3, 2))

    def f():
        y, last, _ = layer.gatedrec(x, g, h0, lengths)
        return float((y * dy).sum() + (last * dh).sum())

    dx, dg, dh0 = layer.gatedrec_grad(x, g, dy, h0, dh, lengths)
    close(dx, numeric(f, x))
    close(dg, numeric(f, g))
    close(dh0, numeric(f, h0))
