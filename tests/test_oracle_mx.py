"""Pins of the microscaled and RMSNorm oracle from outside itself: the
element tables of the format specification, nearest codes by exact rational
arithmetic, gradients by central differences, the layout by hand, and planted
mistakes that each pin has to catch."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import mx


def test_element_tables():
    assert list(mx.element_values(mx.FP4)[:8]) == [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    v = mx.element_values(mx.FP8)
    assert v[0x7e] == 448.0 and np.isnan(v[0x7f]) and np.isnan(v[0xff]) and v[0x01] == 2.0 ** -9
    assert v[0x38] == 1.0 and v[0x08] == 2.0 ** -6 and v[0xb8] == -1.0
    for t in (mx.FP4, mx.FP8):
        pos = mx.element_values(t)[:mx._TYPES[t][3]]
        assert (np.diff(pos) > 0).all()


def _brute(x, t):
    table = mx.element_values(t)[:mx._TYPES[t][3]]
    a = abs(Fraction(float(x)))
    return min(range(len(table)), key=lambda c: (abs(Fraction(table[c]) - a), c % 2))


@pytest.mark.parametrize("t", [mx.FP4, mx.FP8])
def test_nearest_codes_by_rationals(t):
    rng = np.random.default_rng(3)
    table = mx.element_values(t)[:mx._TYPES[t][3]]
    mids = (table[1:] + table[:-1]) / 2
    near = np.concatenate([mids, np.nextafter(mids, 0), np.nextafter(mids, 1e9), table])
    x = np.concatenate([near, rng.normal(size=200) * table[-1] / 2, [0.0, 1e-30, table[-1] * 1.5]])
    got = mx.nearest_codes(x, t) & (7 if t == mx.FP4 else 127)
    assert list(got) == [_brute(v, t) for v in x]
    # planted: ties always down, or truncation, differ at the midpoints
    assert list(np.searchsorted(mids, np.abs(x), side="left")) != list(got)
    assert list(np.searchsorted(table, np.abs(x), side="right") - 1) != list(got)
    assert mx.nearest_codes(np.array([-0.0]), t)[0] == (8 if t == mx.FP4 else 128)


@pytest.mark.parametrize("t,e", [(mx.FP4, 2), (mx.FP8, 8)])
def test_scales(t, e):
    x = np.zeros((1, 32 * 7))
    for i, a in enumerate([1.0, 1.9999, 2.0, 0.0, 2.0 ** -140, 3e38]):
        x[0, 32 * i + 5] = -a
    x[0, 32 * 6] = np.inf
    _, s = mx.quantize(x, t)
    assert list(s[0]) == [127 - e, 127 - e, 128 - e, 0, 0, 254 - e, 255]


@pytest.mark.parametrize("t", [mx.FP4, mx.FP8])
def test_round_trip_and_layout(t):
    rng = np.random.default_rng(5)
    x = rng.normal(size=(3, 96))
    codes, scales = mx.quantize(x, t)
    v = mx.dequantize(codes, scales, t)
    top = np.abs(x.reshape(3, 3, 32)).max(-1, keepdims=True)
    # the largest error is saturation's, over the top binade's power of two: (8 - 6) / 4, (512 - 448) / 256
    worst = 2.0 ** (np.floor(np.log2(top))) * (0.5 if t == mx.FP4 else 0.25)
    assert (np.abs(v - x).reshape(3, 3, 32) <= worst).all()
    again, s2 = mx.quantize(v, t)
    assert np.array_equal(mx.dequantize(again, s2, t), v)
    stored, padded = mx.pack(codes, scales, t)
    assert padded.shape == (3, 16) and (padded[:, 3:] == 0).all()
    back, s3 = mx.unpack(stored, padded, 96, t)
    assert np.array_equal(back, codes) and np.array_equal(s3, scales)
    if t == mx.FP4:
        assert stored[0, 0] & 15 == codes[0, 0] and stored[0, 0] >> 4 == codes[0, 1]


def test_round_bf16():
    one = 1.0 + 2.0 ** -8                     # halfway between 1 and 1 + 2^-7
    x = np.array([one, one + 2.0 ** -40, one + 2.0 ** -7, -one, 0.0])
    assert list(mx.round_bf16(x)) == [1.0, 1.0 + 2.0 ** -7, 1.0 + 2.0 ** -6, -1.0, 0.0]


def test_rmsnorm_gradients_by_differences():
    rng = np.random.default_rng(7)
    h, w, dy, dh = rng.normal(size=(3, 32)), rng.normal(size=32), rng.normal(size=(3, 32)), rng.normal(size=(3, 32))
    eps, d = 1e-3, 1e-5

    def loss(h_, w_):
        y = mx.rmsnorm(h_, w_, eps)[0]
        return (y * dy).sum() + (h_ * dh).sum()

    dx, dw = mx.rmsnorm_backward(dy, h, w, eps, dh)
    for i, j in [(0, 0), (1, 7), (2, 31)]:
        p = np.zeros_like(h)
        p[i, j] = d
        num = (loss(h + p, w) - loss(h - p, w)) / (2 * d)
        assert abs(num - dx[i, j]) < 1e-6     # the differences' own error, about d^2
        # planted: without the mean's term
        assert abs(num - (dy * w / np.sqrt((h * h).mean(-1, keepdims=True) + eps) + dh)[i, j]) > 1e-4
    q = np.zeros_like(w)
    q[9] = d
    assert abs((loss(h, w + q) - loss(h, w - q)) / (2 * d) - dw[9]) < 1e-6


def test_grouped_rows():
    rng = np.random.default_rng(9)
    x, w = rng.normal(size=(6, 32)), rng.normal(size=(3, 4, 32))
    y, _ = mx.grouped(x, w, [1, 3, 3, 5])
    assert np.isnan(y[0]).all() and np.isnan(y[5]).all()
    assert np.allclose(y[2], w[0] @ x[2]) and np.allclose(y[4], w[2] @ x[4])
