"""Plain oracle of the microscaled formats, RMSNorm and the microscaled
products: NumPy in fp64, written from the definitions (OCP Microscaling
Formats specification 1.0 for the formats), with no code of the library.

A microscaled matrix here is (codes, scales): codes uint8 [rows, cols], one
element per entry (not packed), scales uint8 [rows, cols / 32]. `pack` and
`unpack` convert to and from the stored layout.
"""
from __future__ import annotations

import numpy as np

FP4, FP8 = 0, 1
BLOCK = 32
# mantissa bits, exponent bias, exponent of the largest power of two, codes of the positive finite values
_TYPES = {FP4: (1, 1, 2, 8), FP8: (3, 7, 8, 127)}


def element_values(mx: int) -> np.ndarray:
    """fp64 value of every code (NaN where the code is one)."""
    mbits, bias, _, positive = _TYPES[mx]
    half = 8 if mx == FP4 else 128
    v = np.full(2 * half, np.nan)
    for c in range(positive):
        e, m = c >> mbits, c & ((1 << mbits) - 1)
        frac = m / (1 << mbits)
        v[c] = frac * 2.0 ** (1 - bias) if e == 0 else (1.0 + frac) * 2.0 ** (e - bias)
        v[half + c] = -v[c]
    return v


def nearest_codes(x: np.ndarray, mx: int) -> np.ndarray:
    """Code of the element nearest to each finite x: ties to the even code,
    magnitudes past the largest saturate, the sign bit is x's."""
    positive = _TYPES[mx][3]
    table = element_values(mx)[:positive]
    mids = (table[1:] + table[:-1]) / 2          # exact in fp64
    a = np.abs(x)
    low = np.searchsorted(mids, a, side="left")   # a tie goes down ...
    high = np.searchsorted(mids, a, side="right")  # ... or up
    code = np.where(low % 2 == 0, low, high)
    return (code + np.where(np.signbit(x), 8 if mx == FP4 else 128, 0)).astype(np.uint8)


def quantize(x: np.ndarray, mx: int):
    """(codes, scales) of x [rows, cols]. Blocks with a NaN or an Inf: scale 255, codes 0."""
    with np.errstate(invalid="ignore"):           # signalling NaN among every bf16 pattern
        x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    b = x.reshape(rows, cols // BLOCK, BLOCK)
    bad = ~np.isfinite(b).all(-1)
    amax = np.where(bad, 1.0, np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1))
    _, e = np.frexp(amax)                        # amax = m 2^e, m in [1/2, 1): floor(log2 amax) = e - 1
    s = np.where(amax > 0, np.maximum(e - 1 - _TYPES[mx][2], -127), -127)
    codes = nearest_codes(np.ldexp(np.where(bad[..., None], 0.0, b), -s[..., None]), mx)
    scales = np.where(bad, 255, s + 127).astype(np.uint8)
    return codes.reshape(rows, cols), scales


def dequantize(codes: np.ndarray, scales: np.ndarray, mx: int) -> np.ndarray:
    rows, cols = codes.shape
    v = element_values(mx)[codes].reshape(rows, cols // BLOCK, BLOCK)
    f = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (v * f[..., None]).reshape(rows, cols)


def pitch(cols: int) -> int:
    return 16 * -(-cols // 512)


def pack(codes: np.ndarray, scales: np.ndarray, mx: int):
    """The stored codes and scale rows."""
    rows, cols = codes.shape
    padded = np.zeros((rows, pitch(cols)), np.uint8)
    padded[:, :cols // BLOCK] = scales
    if mx == FP8:
        return codes, padded
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8), padded


def unpack(stored: np.ndarray, padded: np.ndarray, cols: int, mx: int):
    scales = padded[:, :cols // BLOCK]
    if mx == FP8:
        return stored, scales
    codes = np.empty((stored.shape[0], cols), np.uint8)
    codes[:, 0::2], codes[:, 1::2] = stored & 15, stored >> 4
    return codes, scales


def round_bf16(x: np.ndarray) -> np.ndarray:
    """fp64 rounded once to bf16 (nearest even, within the normal range), as fp64."""
    m, e = np.frexp(np.asarray(x, dtype=np.float64))
    return np.ldexp(np.rint(np.ldexp(m, 8)), e - 8)


def rmsnorm(x, weight, eps, residual=None):
    """(y, h, rstd) in fp64: h is the rounded bf16 sum, y is not rounded."""
    h = np.asarray(x, np.float64) if residual is None else round_bf16(np.asarray(x, np.float64) + residual)
    rstd = 1.0 / np.sqrt((h * h).mean(-1) + eps)
    return h * rstd[:, None] * np.asarray(weight, np.float64), h, rstd


def rmsnorm_backward(dy, h, weight, eps, dh=None):
    """(dx, dw) in fp64 of y = h rstd weight with dh arriving at h directly."""
    rstd = (1.0 / np.sqrt((h * h).mean(-1) + eps))[:, None]
    u, g = h * rstd, dy * weight
    dx = rstd * (g - u * (g * u).mean(-1, keepdims=True))
    return (dx if dh is None else dx + dh), (dy * u).sum(0)


def linear(x: np.ndarray, w: np.ndarray):
    """(x w^T, sum |x| |w|): the product and what bounds the error of its sums."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def grouped(x: np.ndarray, w: np.ndarray, offsets):
    """Row i of the product by expert (w [experts, N, K]); NaN where no expert has the row. And the bound's sums."""
    y = np.full((x.shape[0], w.shape[1]), np.nan)
    size = np.full_like(y, np.nan)
    for e in range(w.shape[0]):
        a, b = (min(max(int(o), 0), x.shape[0]) for o in offsets[e:e + 2])
        if a < b:
            y[a:b], size[a:b] = linear(x[a:b], w[e])
    return y, size
