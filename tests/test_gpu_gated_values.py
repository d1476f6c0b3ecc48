"""Values of the gated block with adapters that random inputs do not reach, at each of its kernels: infinities, a
padded rank, inputs that have a mean.

Infinities: a sum with one of them is that one by the sign of its factor, with two of different signs NaN, whatever
the order; what no infinite term reaches keeps its bits. The formula is taken in fp64 term by term, so that it adds
nothing of its own (no padding, no blocks)."""
import numpy as np
import pytest

from oracle import block
from tests import gpu_util as gu
from tests.test_gpu_gated import GRADS, Data, f64, near, qb  # noqa: F401

pytestmark = pytest.mark.gpu

# one row in registers; one that is not; a few in LDS; up to 16, too long for LDS, up to 32; tiles, whole and with split low products
PATHS = [(1, 64, 256), (1, 64, 320), (3, 128, 320), (9, 64, 192), (4, 64, 8192), (20, 128, 128), (32, 64, 64), (40, 128, 192), (40, 64, 1024),
         (300, 128, 128)]


def product(x, w):
    """x w^T, one sum over the products of each element."""
    with np.errstate(invalid="ignore"):
        return np.stack([(row * w).sum(-1) for row in x])


def same_kind(got, want, label):
    """Infinite with the sign, NaN and finite in the same places."""
    g = f64(got)
    assert np.array_equal(np.isnan(g), np.isnan(want)), f"{label}: NaN in {np.isnan(g).sum()} places, not {np.isnan(want).sum()}"
    assert np.array_equal(np.where(np.isinf(g), g, 0), np.where(np.isinf(want), want, 0)), f"{label}: infinities"


def equal_rows(a, b, rows):
    import torch
    keep = torch.ones(a.shape[0], dtype=torch.bool, device="cuda")
    keep[rows] = False
    return torch.equal(a[keep], b[keep])


@pytest.mark.parametrize("r", [0, 1, 8, 70])
@pytest.mark.parametrize("M,N,K", PATHS)
def test_infinite_inputs(qb, M, N, K, r):  # noqa: F811
    gu.announce(f"gated infinite X {M}x{N}x{K} r={r}")
    d = Data(qb, M, N, K, r)
    clean = qb.qlora_gated_fwd_save(d.X, *d.args)
    rows = sorted({0, M // 2, M - 1})
    X = d.X.clone()
    for i, m in enumerate(rows):
        X[m, (37 * i + 5) % K] = (-1) ** i * float("inf")
    H, G, U, Hs = qb.qlora_gated_fwd_save(X, *d.args)
    x, sums = f64(X)[rows], []
    with np.errstate(invalid="ignore"):
        for i, w in enumerate((d.gate, d.up)):
            y = product(x, f64(qb.qlora_nf4_dequantize(w)))
            if r:
                a, b, cols = f64(d.factors[2 * i]), f64(d.factors[2 * i + 1]), Hs.shape[1] // 2
                low = d.scale * product(x, a)
                same_kind(Hs[rows, i * cols:i * cols + r], low, "Hs")
                assert not Hs[:, i * cols + r:(i + 1) * cols].any(), "the columns behind the rank"
                y = y + product(low, b)
            sums.append(y)
        h = block.gate(*sums)
    for got, want, before, label in ((G, sums[0], clean[1], "G"), (U, sums[1], clean[2], "U"), (H, h, clean[0], "H")):
        same_kind(got[rows], want, label)
        assert equal_rows(got, before, rows), label


@pytest.mark.parametrize("r", [0, 1, 3, 8, 70])
@pytest.mark.parametrize("M,N,K", PATHS)
def test_infinite_gradients(qb, M, N, K, r):  # noqa: F811
    gu.announce(f"gated infinite dH {M}x{N}x{K} r={r}")
    d = Data(qb, M, N, K, r)
    kept = qb.qlora_gated_fwd_save(d.X, *d.args)[1:]
    clean = qb.qlora_gated_bwd(d.dH, d.X, *kept, *d.args)
    rows = sorted({0, M - 1})
    dH = d.dH.clone()
    for i, m in enumerate(rows):
        dH[m, (29 * i + 3) % N] = (-1) ** i * float("inf")
    out = qb.qlora_gated_bwd(dH, d.X, *kept, *d.args)
    with np.errstate(invalid="ignore"):
        sides = block.gate_backward(f64(dH), f64(kept[0]), f64(kept[1]))
        dx = 0.0
        for i, (dd, w) in enumerate(zip(sides, (d.gate, d.up))):
            dx = dx + product(dd[rows], f64(qb.qlora_nf4_dequantize(w)).T)
            if r:
                a, b, cols = f64(d.factors[2 * i]), f64(d.factors[2 * i + 1]), kept[2].shape[1] // 2
                low = d.scale * product(dd, b.T)
                dx = dx + product(low[rows], a.T)
                same_kind(out[1 + 2 * i], product(low.T, f64(d.X).T), GRADS[1 + 2 * i])
                same_kind(out[2 + 2 * i], product(dd.T, f64(kept[2])[:, i * cols:i * cols + r].T), GRADS[2 + 2 * i])
    same_kind(out[0][rows], dx, "dX")
    assert equal_rows(out[0], clean[0], rows)


@pytest.mark.parametrize("side", [0, 1])
@pytest.mark.parametrize("M,N,K", PATHS)
def test_overflow_of_one_adapter(qb, M, N, K, side):  # noqa: F811
    """One weight's adapter activations overflow: the other weight's sums keep their bits."""
    import torch
    gu.announce(f"gated overflow {M}x{N}x{K} side {side}")
    d = Data(qb, M, N, K, 8)
    d.X.abs_().add_(0.5)
    clean = qb.qlora_gated_fwd_save(d.X, *d.args)
    d.factors[2 * side].fill_(3e38)
    H, G, U, Hs = qb.qlora_gated_fwd_save(d.X, *d.args)
    cols = Hs.shape[1] // 2
    assert torch.isinf(Hs[:, side * cols:side * cols + 8]).all() and not torch.isfinite((G, U)[side]).any()
    assert torch.equal((U, G)[side], clean[2 - side])


@pytest.mark.parametrize("fmt", [0, 1, 2, 3])
@pytest.mark.parametrize("mean", [1.0, -4.0])
@pytest.mark.parametrize("M,N,K", [(1, 1088, 4096), (1, 1088, 4160), (1, 320, 16384), (4, 1088, 4096), (4, 576, 8192), (16, 1088, 4096), (32, 1088, 4096),
                                   (33, 1088, 4096)])
def test_inputs_with_a_mean(qb, M, N, K, mean, fmt):  # noqa: F811
    """A mean of X adds up the mean error of the weights, which is far below the error of one weight: G and U stay
    within the bar of test_gpu_gated.py, two roundings of 2.26e-3, one a weight's and one the sum's own."""
    import torch
    gu.announce(f"gated mean {mean} {M}x{N}x{K} format {fmt}")
    d = Data(qb, M, N, K, 0, fmt=fmt)
    d.X.copy_((d.X.float() + mean).to(torch.bfloat16))
    _, g, u, _ = d.oracle()
    _, G, U, _ = qb.qlora_gated_fwd_save(d.X, *d.args)
    near(G, g, 4.5e-3, "G")
    near(U, u, 4.5e-3, "U")
