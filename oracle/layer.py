"""fp64 layer norm, rotary positions and gated recurrence, with their gradients
-- TEST INFRASTRUCTURE ONLY.

Only ``tests/`` and ``smoke()`` import this module (it imports nothing from the
product).  Plain numpy float64 from the definitions:

  layer norm: y = (r - mean(r)) / sqrt(var(r) + eps) * w + b over the last axis;
  rotary: the pair (u, v) of a head at position p, as the number u + iv, times
  m exp(2 pi i p f);
  gated recurrence: h_t = a_t h_{t-1} + (1 - a_t) x_t, a = 1 / (1 + exp(-g)).

Pinned in ``tests/test_oracle_pins_layer.py`` by torch's fp64 functions, by
finite differences and by closed forms.
"""
from __future__ import annotations

import math

import numpy as np


def layernorm(r, w, b, eps):
    """y, mean, rstd of r [..., D]."""
    mean = r.mean(-1)
    z = r - mean[..., None]
    rstd = 1.0 / np.sqrt((z * z).mean(-1) + eps)
    y = z * rstd[..., None] * w
    return (y if b is None else y + b), mean, rstd


def layernorm_grad(dy, r, w, eps, dresid=None):
    """dx, dw, db."""
    mean = r.mean(-1, keepdims=True)
    rstd = 1.0 / np.sqrt(((r - mean) ** 2).mean(-1, keepdims=True) + eps)
    xh = (r - mean) * rstd
    t = dy * w
    dx = rstd * (t - t.mean(-1, keepdims=True) - xh * (t * xh).mean(-1, keepdims=True))
    lead = tuple(range(dy.ndim - 1))
    return (dx if dresid is None else dx + dresid), (dy * xh).sum(lead), dy.sum(lead)


def rotary_freqs(rot, base=10000.0, scaling="none", factor=1.0, original_len=1, low=1.0, high=4.0):
    """Turns per position of each pair."""
    out = []
    for i in range(rot // 2):
        f = math.exp(-2.0 * i / rot * math.log(base)) / (2.0 * math.pi)
        if scaling == "linear":
            f = f / factor
        elif scaling == "by_parts":
            n = f * original_len
            keep = 0.0 if n <= low else 1.0 if n >= high else (n - low) / (high - low)
            f = keep * f + (1.0 - keep) * (f / factor)
        out.append(f)
    return np.array(out)


def rotary(x, freqs, pos, layout, mscale=1.0, inverse=False):
    """x [B, H, L, D], pos an int or [B]."""
    B, _, L, _ = x.shape
    rot = 2 * len(freqs)
    out = x.copy()
    start = np.broadcast_to(np.asarray(pos, dtype=np.int64), (B,))
    for b in range(B):
        turns = np.outer(np.arange(L) + int(start[b]), freqs)
        z = mscale * np.exp(2j * np.pi * (turns - np.round(turns)))  # [L, rot / 2]
        if inverse:
            z = z.conj()
        if layout == "half":
            w = (x[b, :, :, :rot // 2] + 1j * x[b, :, :, rot // 2:rot]) * z
            out[b, :, :, :rot // 2], out[b, :, :, rot // 2:rot] = w.real, w.imag
        else:
            w = (x[b, :, :, 0:rot:2] + 1j * x[b, :, :, 1:rot:2]) * z
            out[b, :, :, 0:rot:2], out[b, :, :, 1:rot:2] = w.real, w.imag
    return out


def _gates(g):
    """sigmoid(g) and sigmoid(-g), each to full relative precision."""
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g)), 1.0 / (1.0 + np.exp(g))


def gatedrec(x, g, h0=None, lengths=None):
    """y [B, L, D] (zero past the lengths), the final state [B, D], and the
    states that enter each token [B, L, D] (zero past the lengths)."""
    B, L, D = x.shape
    y, before = np.zeros((B, L, D)), np.zeros((B, L, D))
    last = np.zeros((B, D))
    for b in range(B):
        h = np.zeros(D) if h0 is None else h0[b].copy()
        for t in range(L if lengths is None else int(lengths[b])):
            a, n = _gates(g[b, t])
            before[b, t] = h
            h = a * h + n * x[b, t]
            y[b, t] = h
        last[b] = h
    return y, last, before


def gatedrec_grad(x, g, dy, h0=None, dh_last=None, lengths=None):
    """dx, dg [B, L, D] (zero past the lengths) and dh0 [B, D]."""
    B, L, D = x.shape
    _, _, before = gatedrec(x, g, h0, lengths)
    dx, dg, dh0 = np.zeros((B, L, D)), np.zeros((B, L, D)), np.zeros((B, D))
    for b in range(B):
        carry = np.zeros(D) if dh_last is None else dh_last[b].copy()
        for t in range((L if lengths is None else int(lengths[b])) - 1, -1, -1):
            a, n = _gates(g[b, t])
            l = dy[b, t] + carry
            dx[b, t] = n * l
            dg[b, t] = l * (before[b, t] - x[b, t]) * a * n
            carry = a * l
        dh0[b] = carry
    return dx, dg, dh0
