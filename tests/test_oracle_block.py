"""Pins of the oracle of the gated product and of rotary positions from
outside itself: known values, central differences, complex multiplication,
rotations of far positions in exact rational turns, and planted mistakes that
each pin has to catch."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import block


def test_gate_known_values():
    assert block.gate(0.0, 5.0) == 0.0
    assert abs(block.gate(1.0, 2.0) - 2.0 * np.e / (1.0 + np.e)) < 1e-15
    assert abs(block.gate(30.0, 1.0) - 30.0) < 1e-11 and block.gate(-800.0, 1.0) == 0.0
    g = np.linspace(-6, 6, 25)
    assert np.allclose(block.gate(g, 1.0) + block.gate(-g, 1.0) * -1, g)   # silu(g) - silu(-g) = g


def test_gate_backward_by_differences():
    rng = np.random.default_rng(1)
    dh, g, u = rng.normal(size=(3, 200)) * 2
    dg, du = block.gate_backward(dh, g, u)
    e = 1e-6
    assert np.allclose(dg, dh * (block.gate(g + e, u) - block.gate(g - e, u)) / (2 * e), atol=1e-8)
    assert np.allclose(du, dh * (block.gate(g, u + e) - block.gate(g, u - e)) / (2 * e), atol=1e-8)
    wrong = dh * u * block.sigmoid(g)   # planted: the sigmoid taken for a constant
    assert not np.allclose(wrong, dg, atol=1e-3)


def test_feed_forward_backward_by_differences():
    rng = np.random.default_rng(2)
    x, wg, wu = rng.normal(size=(3, 5)), rng.normal(size=(4, 5)), rng.normal(size=(4, 5))
    ad = [rng.normal(size=s) for s in ((2, 5), (4, 2), (2, 5), (4, 2))]
    dh = rng.normal(size=(3, 4))
    grads = block.feed_forward_backward(dh, x, wg, wu, ad, 0.7)

    def loss():
        return (dh * block.feed_forward(x, wg, wu, ad, 0.7)[0]).sum()
    for t, d in zip([x] + ad, grads):
        for _ in range(6):
            i = tuple(rng.integers(0, n) for n in t.shape)
            keep, e = t[i], 1e-6
            t[i] = keep + e
            up = loss()
            t[i] = keep - e
            down = loss()
            t[i] = keep
            assert abs((up - down) / (2 * e) - d[i]) < 1e-7 * max(1.0, abs(d[i]))


def test_pair_rows_by_hand():
    g, u = np.arange(16)[:, None], 100 + np.arange(16)[:, None]
    want = list(range(8)) + list(range(100, 108)) + list(range(8, 16)) + list(range(108, 116))
    assert list(block.pair_rows(g, u)[:, 0]) == want
    a, b = block.split_pair(np.array([want]))
    assert list(a[0]) == list(range(16)) and list(b[0]) == list(range(100, 116))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_complex_multiplication(interleaved):
    rng = np.random.default_rng(3)
    x, pos = rng.normal(size=(5, 2, 10)), np.array([0, 1, 7, 100, 5])
    f, _ = block.rope_freqs(6)
    y = block.rope(x, pos, f, 1.5, interleaved)
    a, b = (x[..., 0:6:2], x[..., 1:6:2]) if interleaved else (x[..., :3], x[..., 3:6])
    z = (a + 1j * b) * 1.5 * np.exp(1j * pos[:, None] * f)[:, None, :]
    got = y[..., 0:6:2] + 1j * y[..., 1:6:2] if interleaved else y[..., :3] + 1j * y[..., 3:6]
    assert np.allclose(got, z) and np.array_equal(y[..., 6:], x[..., 6:])
    assert np.allclose(y[0, ..., :6], 1.5 * x[0, ..., :6])
    other = block.rope(x, pos, f, 1.5, not interleaved)   # planted: the other layout
    assert not np.allclose(other, y)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_backward_is_the_transpose(interleaved):
    rng = np.random.default_rng(4)
    x, dy, pos = rng.normal(size=(4, 3, 8)), rng.normal(size=(4, 3, 8)), np.array([3, 900, 0, 12])
    f, _ = block.rope_freqs(8)
    left = (dy * block.rope(x, pos, f, 0.8, interleaved)).sum()
    dx = block.rope(dy, pos, f, 0.8, interleaved, backward=True)
    assert np.isclose(left, (dx * x).sum())
    assert not np.isclose(left, (block.rope(dy, pos, f, 0.8, interleaved) * x).sum())   # planted: the same way round


def test_rope_depends_on_distances_only():
    rng = np.random.default_rng(5)
    q, k = rng.normal(size=(2, 1, 1, 16))
    f, _ = block.rope_freqs(16)
    dots = [(block.rope(q, [9 + s], f) * block.rope(k, [4 + s], f)).sum() for s in (0, 1, 50)]
    assert np.allclose(dots, dots[0])


def test_rope_freqs():
    f, amp = block.rope_freqs(128)
    assert f[0] == 1.0 and np.isclose(f[63], 10000.0 ** (-126 / 128)) and amp == 1.0
    lin, _ = block.rope_freqs(128, scaling="linear", factor=4.0)
    assert np.allclose(lin, f / 4)
    ntk, _ = block.rope_freqs(128, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0 and np.isclose(ntk[63], f[63] / 4)   # the ends are those of plain and linear
    parts, amp = block.rope_freqs(128, scaling="parts", factor=4.0, trained=2048, low=1.0, high=32.0)
    turns = [Fraction(2048) * Fraction(x) / Fraction(2 * np.pi) for x in f]
    for p, t, x in zip(parts, turns, f):
        assert np.isclose(p, x if t >= 32 else x / 4 if t <= 1 else x / 4 + (x - x / 4) * float(t - 1) / 31)
    assert np.isclose(amp, 1 + 0.1 * np.log(4))


def test_turns_of_far_positions():
    """The rotation forms an angle's turns in fp64 as t (f / (2 pi)): three roundings, 2^-23 turns at 2^31, as
    qlora_block.h states, and more than the 2^-25 of one rounding with a rounded constant left out."""
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510")
    rng = np.random.default_rng(6)
    worst = 0
    for f in [1.0, *rng.uniform(0.5, 1.0, 60)]:
        for t in rng.integers(2 ** 31 - 2 ** 20, 2 ** 31, 60):
            got = float(t) * (f * 0.15915494309189533577)
            worst = max(worst, abs(Fraction(got) - int(t) * Fraction(f) / two_pi))
    assert Fraction(1, 2 ** 25) < worst < Fraction(1, 2 ** 23)
