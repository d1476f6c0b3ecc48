"""Plain oracle of what stands between a decoder layer's projections: the
gated feed-forward product and rotary positions, in fp64 from their formulas,
with no code of the library.

    silu(g) = g / (1 + e^-g)
    H = silu(G) * U
    dG = dH U s (1 + G (1 - s)),  dU = dH G s,   s = 1 / (1 + e^-G)

Rotary positions take pair (a, b) of a head at position t by the angle
w = t f to (a cos w - b sin w, b cos w + a sin w).
"""
from __future__ import annotations

import numpy as np

from . import linear


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-np.asarray(g, dtype=np.float64)))


def gate(g, u):
    """silu(g) * u."""
    return np.asarray(g, dtype=np.float64) * sigmoid(g) * u


def gate_backward(dh, g, u):
    """(dg, du) of h = silu(g) * u."""
    s = sigmoid(g)
    return dh * u * s * (1.0 + g * (1.0 - s)), dh * g * s


def pair_rows(gate_rows, up_rows):
    """Rows of two matrices [N, ...] as one [2 N, ...]: eight of each in turn (N a multiple of 8)."""
    out = []
    for j in range(0, len(gate_rows), 8):
        out += [gate_rows[j:j + 8], up_rows[j:j + 8]]
    return np.concatenate(out)


def split_pair(y):
    """The products [M, 2 N] with a pair's rows: those of the gate and of the other weight, [M, N] each."""
    gate_cols = [c for c in range(y.shape[1]) if c % 16 < 8]
    up_cols = [c for c in range(y.shape[1]) if c % 16 >= 8]
    return y[:, gate_cols], y[:, up_cols]


def feed_forward(x, wg, wu, adapters=None, scale=0.0):
    """(h, g, u): adapters (ag, bg, au, bu) or None."""
    ag, bg, au, bu = adapters if adapters is not None else (None,) * 4
    g, u = linear.forward(x, wg, ag, bg, scale), linear.forward(x, wu, au, bu, scale)
    return gate(g, u), g, u


def feed_forward_backward(dh, x, wg, wu, adapters=None, scale=0.0):
    """(dx, dag, dbg, dau, dbu), the last four None without adapters."""
    ag, bg, au, bu = adapters if adapters is not None else (None,) * 4
    _, g, u = feed_forward(x, wg, wu, adapters, scale)
    dg, du = gate_backward(np.asarray(dh, dtype=np.float64), g, u)
    xg, dag, dbg = linear.backward(dg, x, wg, ag, bg, scale)
    xu, dau, dbu = linear.backward(du, x, wu, au, bu, scale)
    return xg + xu, dag, dbg, dau, dbu


def rope_freqs(rot, base=10000.0, scaling="plain", factor=1.0, trained=4096, low=1.0, high=32.0):
    """(radians a position of each of rot / 2 pairs, amplitude)."""
    amplitude = 1.0
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2.0))
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f = f / factor
        if scaling == "parts":
            turns = trained * f / (2.0 * np.pi)
            keep = (turns - low) / (high - low)
            keep = 0.0 if keep < 0.0 else 1.0 if keep > 1.0 else keep
            f = keep * f + (1.0 - keep) * f / factor
            amplitude = 0.1 * np.log(factor) + 1.0
        out.append(f)
    return np.array(out), amplitude


def rope(x, positions, freqs, amplitude=1.0, interleaved=False, backward=False):
    """x [rows, heads, dim] rotated by positions [rows]; backward: the gradient of x from that of the result."""
    out = np.array(x, dtype=np.float64)
    half = len(freqs)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        w = np.asarray(positions, dtype=np.float64) * freqs[i]
        c, s = (amplitude * np.cos(w))[:, None], (amplitude * np.sin(w))[:, None]
        if backward:
            s = -s
        out[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        out[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return out
