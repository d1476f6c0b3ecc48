"""GPU parity of rotary positions against the fp64 oracle (oracle/block.py).

Bar. The angle is off by 2^-53 of its turns three times over (the frequency in
turns, the product, and the oracle's own product) and by the rounding of a turn
of at most one half (as 2 r) to fp32: 2^-25 half turns. Sine and cosine are
within 2 ulp of their values, 2^-22, the amplitude's product and the rotation's
two products and sum round by 2^-24 each: together less than 2^-20 of the
pair's length, and 2 pi t f 2^-51. The result is rounded once: half a step of
its type, 2^-8 or 2^-24 of it.
"""
import numpy as np
import pytest

from oracle import block
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qb():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_nf4_quantized_03_amd as m
    return m


def dtype_of(name):
    import torch
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def host64(t):
    return t.detach().cpu().double().numpy()


def check(got, x, pos, f, amp, interleaved, backward, label):
    xv, half = host64(x), len(f)
    want = block.rope(xv, pos, f, amp, interleaved, backward)
    a, b = (xv[..., 0:2 * half:2], xv[..., 1:2 * half:2]) if interleaved else (xv[..., :half], xv[..., half:2 * half])
    size = np.hypot(a, b) * abs(amp)
    off = size * (2.0 ** -20 + 2 * np.pi * 2.0 ** -51 * np.abs(np.asarray(pos, dtype=np.float64))[:, None, None] * f)
    bound = np.zeros_like(want)
    if interleaved:
        bound[..., 0:2 * half:2] = bound[..., 1:2 * half:2] = off
    else:
        bound[..., :half] = bound[..., half:2 * half] = off
    step = 2.0 ** -8 if str(x.dtype) == "torch.bfloat16" else 2.0 ** -24
    bound[..., :2 * half] += step * (np.abs(want[..., :2 * half]) + bound[..., :2 * half]) + 1e-38
    g = host64(got)
    err = np.abs(g - want)
    assert (err <= bound).all(), f"{label}: worst {np.max(err[..., :2 * half] / bound[..., :2 * half])} of the bound"
    assert np.array_equal(g[..., 2 * half:], xv[..., 2 * half:]), f"{label}: what passes through"


def positions(rng, rows, far):
    p = rng.integers(0, far + 1, rows)
    p[0] = 0
    p[-1] = far
    return p


CASES = [(1, 1, 1, 2, 2), (1, 32, 32, 128, 128), (1, 1, 1, 1024, 1024), (2, 3, 1, 6, 4), (3, 40, 8, 128, 128), (5, 7, 2, 80, 80),
         (7, 8, 8, 96, 32), (33, 12, 4, 64, 20), (64, 32, 8, 128, 64), (129, 5, 5, 256, 256), (700, 32, 8, 128, 128), (1000, 9, 1, 72, 66),
         (2, 200, 3, 130, 130), (4, 300, 300, 16, 16), (9000, 4, 4, 64, 64)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("name", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,nq,nk,dim,rot", CASES)
def test_rope(qb, rows, nq, nk, dim, rot, name, interleaved):
    import torch
    gu.announce(f"rope {rows} rows {nq}+{nk} heads {dim}/{rot} {name} {interleaved}")
    rng = np.random.default_rng(rows + dim + rot)
    dt = dtype_of(name)
    q, k = (torch.from_numpy(rng.normal(size=(rows, n, dim))).to(dt).cuda() for n in (nq, nk))
    f, _ = qb.qlora_rope_freqs(rot, device="cuda")
    pos = positions(rng, rows, 5000)
    p = torch.from_numpy(pos).cuda()
    for fn, back in ((qb.qlora_rope_fwd, False), (qb.qlora_rope_bwd, True)):
        a, b = fn(q, k, p, f, 1.25, interleaved)
        assert a.is_contiguous() and a.dtype is dt and b.shape == k.shape
        check(a, q, pos, host64(f), 1.25, interleaved, back, "q")
        check(b, k, pos, host64(f), 1.25, interleaved, back, "k")
        # int32 positions, one tensor alone, in place: the same bits
        c, none = fn(q, None, p.int(), f, 1.25, interleaved)
        assert none is None and torch.equal(c, a)
        q2, k2 = q.clone(), k.clone()
        out = fn(q2, k2, p, f, 1.25, interleaved, outs=(q2, k2))
        assert out[0] is q2 and torch.equal(q2, a) and torch.equal(k2, b)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("name", ["bf16", "fp32"])
@pytest.mark.parametrize("offset", [0, 8, 1])
def test_strides_and_alignment(qb, name, interleaved, offset):
    """Queries and keys out of one fused projection, heads in front of rows, views that begin anywhere, and outputs with gaps."""
    import torch
    gu.announce(f"rope strides {name} {interleaved} {offset}")
    dt, rows, nq, nk, dim = dtype_of(name), 37, 6, 2, 64
    rng = np.random.default_rng(offset)
    f, _ = qb.qlora_rope_freqs(32, device="cuda")
    pos = positions(rng, rows, 100)
    p = torch.from_numpy(pos).cuda()
    flat = torch.from_numpy(rng.normal(size=rows * (nq + 2 * nk) * dim + offset)).to(dt).cuda()
    both = flat[offset:].view(rows, nq + 2 * nk, dim)
    before = both.clone()
    q, k = both[:, :nq], both[:, nq:nq + nk]
    a, b = qb.qlora_rope_fwd(q, k, p, f, interleaved=interleaved)
    check(a, q, pos, host64(f), 1.0, interleaved, False, "q")
    check(b, k, pos, host64(f), 1.0, interleaved, False, "k")
    t = q.transpose(0, 1).contiguous().transpose(0, 1)   # heads in front of rows
    assert t.stride(0) == dim and torch.equal(qb.qlora_rope_fwd(t, k, p, f, interleaved=interleaved)[0], a)
    wide = torch.full((rows, nq, dim + 6), 5.0, dtype=dt, device="cuda")
    out = torch.full((nk, rows, dim), 5.0, dtype=dt, device="cuda").transpose(0, 1)
    qb.qlora_rope_fwd(q, k, p, f, interleaved=interleaved, outs=(wide[..., :dim], out))
    assert torch.equal(wide[..., :dim], a) and (wide[..., dim:] == 5.0).all() and torch.equal(out, b)
    # in place in the fused projection: values stay as they were
    assert torch.equal(both, before)
    qb.qlora_rope_fwd(q, k, p, f, interleaved=interleaved, outs=(q, k))
    assert torch.equal(q, a) and torch.equal(k, b) and torch.equal(both[:, nq + nk:], before[:, nq + nk:])
    # one query for all rows
    one = torch.from_numpy(rng.normal(size=(1, nq, dim))).to(dt).cuda()
    assert torch.equal(qb.qlora_rope_fwd(one.expand(rows, nq, dim), None, p, f)[0], qb.qlora_rope_fwd(one.repeat(rows, 1, 1), None, p, f)[0])


@pytest.mark.parametrize("scaling,factor", [(0, 1.0), (1, 16.0), (2, 16.0), (3, 16.0)])
def test_far_positions(qb, scaling, factor):
    """Positions up to 2^31 - 1, and negative ones, with each scaling."""
    import torch
    gu.announce(f"rope far {scaling}")
    rng = np.random.default_rng(scaling)
    f, amp = qb.qlora_rope_freqs(128, scaling=scaling, factor=factor, device="cuda")
    pos = np.array([2 ** 31 - 1, 131071, 1000003, 1 << 24, (1 << 24) + 1, -1, -77777, 12345678, 2 ** 31 - 2])
    x = torch.from_numpy(rng.normal(size=(len(pos), 3, 128))).float().cuda()
    for p in (torch.from_numpy(pos).cuda(), torch.from_numpy(pos).int().cuda()):
        y, _ = qb.qlora_rope_fwd(x, None, p, f, amp)
        check(y, x, pos, host64(f), amp, False, False, "far")


def test_special_values(qb):
    """NaN and Inf stay in their pair; position 0 with amplitude 1 leaves the values as they are."""
    import torch
    gu.announce("rope special values")
    f, _ = qb.qlora_rope_freqs(16, device="cuda")
    for dt in (torch.bfloat16, torch.float32):
        for interleaved in (False, True):
            x = torch.randn(4, 2, 24, device="cuda").to(dt)
            p = torch.tensor([0, 3, 9, 0], device="cuda")
            clean, _ = qb.qlora_rope_fwd(x, None, p, f, interleaved=interleaved)
            assert torch.equal(clean[0], x[0]) and torch.equal(clean[3], x[3])
            bad = x.clone()
            bad[1, 0, 2], bad[2, 1, 5], bad[1, 1, 20] = float("nan"), float("inf"), float("nan")
            y, _ = qb.qlora_rope_fwd(bad, None, p, f, interleaved=interleaved)
            hit = torch.zeros_like(x, dtype=torch.bool)
            for at, i in (((1, 0), 2), ((2, 1), 5)):
                hit[at + (i,)] = True
                hit[at + ((i ^ 1) if interleaved else (i + 8) % 16,)] = True
            hit[1, 1, 20] = True
            assert not torch.isfinite(y[hit]).any() and torch.equal(y[~hit], clean[~hit])


def test_backward_by_differences(qb):
    """The gradient against differences of the forward pass, which is linear."""
    import torch
    gu.announce("rope differences")
    rng = np.random.default_rng(9)
    f, amp = qb.qlora_rope_freqs(12, scaling=3, factor=2.0, device="cuda")
    p = torch.tensor([5, 0, 70], device="cuda")
    for interleaved in (False, True):
        x, dy = (torch.from_numpy(rng.normal(size=(3, 2, 16))).float().cuda() for _ in range(2))
        dx, _ = qb.qlora_rope_bwd(dy, None, p, f, amp, interleaved)
        base = qb.qlora_rope_fwd(x, None, p, f, amp, interleaved)[0].double()
        for i in rng.choice(x.numel(), 40, replace=False):
            moved = x.clone()
            moved.view(-1)[i] += 1.0
            step = (moved.view(-1)[i].double() - x.view(-1)[i].double()).item()
            diff = ((qb.qlora_rope_fwd(moved, None, p, f, amp, interleaved)[0].double() - base) * dy.double()).sum().item() / step
            # both differences of outputs of a few units, rounded to 2^-24 of them, times gradients of a few units
            assert abs(diff - dx.view(-1)[i].item()) < 1e-5


def test_many_rows_and_past_32_bits(qb):
    """More workgroups than one launch takes, and elements behind 2^32: the last rows against the same rows on their own."""
    import torch
    gu.announce("rope past 32 bits")
    f, _ = qb.qlora_rope_freqs(128, device="cuda")
    rows, n = (1 << 21) + 3, 17
    x = torch.zeros(rows, n, 128, dtype=torch.bfloat16, device="cuda")
    x[-5:] = torch.randn(5, n, 128, device="cuda")
    p = torch.arange(rows, device="cuda")
    y, _ = qb.qlora_rope_fwd(x, None, p, f)
    assert torch.equal(y[-5:], qb.qlora_rope_fwd(x[-5:].contiguous(), None, p[-5:].contiguous(), f)[0]) and not y[rows // 2].any()
    del x, y
    rows = 3 * (1 << 21) + 1
    x = torch.zeros(rows, 1, 1024, dtype=torch.bfloat16, device="cuda")
    x[-2:] = torch.randn(2, 1, 1024, device="cuda")
    f, _ = qb.qlora_rope_freqs(1024, device="cuda")
    p = torch.arange(rows, device="cuda")
    qb.qlora_rope_fwd(x, None, p, f, outs=(x, None))
    assert not x[:-2].any() and x[-2:].any()


def test_captured_and_two_streams(qb):
    """Captured with its positions and replayed with others; two streams at once."""
    import torch
    gu.announce("rope captured")
    f, amp = qb.qlora_rope_freqs(64, scaling=1, factor=4.0, device="cuda")
    q, k = torch.randn(9, 8, 64, device="cuda").bfloat16(), torch.randn(9, 2, 64, device="cuda").bfloat16()
    p = torch.arange(9, device="cuda")
    call = lambda: qb.qlora_rope_fwd(q, k, p, f, amp) + qb.qlora_rope_bwd(q, k, p, f, amp)  # noqa: E731
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            outs = call()
    for i in range(4):
        p += 1000
        q.copy_(torch.randn_like(q))
        graph.replay()
        torch.cuda.synchronize()
        kept = [o.clone() for o in outs]
        assert all(torch.equal(a, b) for a, b in zip(kept, call())), f"replay {i}"
    want = call()
    torch.cuda.synchronize()
    other, got = torch.cuda.Stream(), []
    for _ in range(6):
        for st in (stream, other):
            with torch.cuda.stream(st):
                got.append(call())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for outs in got for a, b in zip(outs, want))


def test_refusals_with_tensors(qb):
    import torch
    gu.announce("rope refusals")
    f, _ = qb.qlora_rope_freqs(32, device="cuda")
    q, p = torch.randn(3, 2, 64, device="cuda"), torch.arange(3, device="cuda")
    for args, error in (((q.half(), None, p, f), TypeError), ((q[0], None, p, f), ValueError), ((q.cpu(), None, p, f), TypeError),
                        ((q, q.bfloat16(), p, f), TypeError), ((q, q[:2], p, f), ValueError), ((q, q[..., :62], p, f), ValueError),
                        ((q, None, p.float(), f), TypeError), ((q, None, p[:2], f), ValueError), ((q, None, p, f.float()), TypeError),
                        ((q, None, p, f.cpu()), TypeError), ((q.transpose(1, 2), None, p, f), ValueError),
                        ((q, None, p, torch.ones(33, dtype=torch.float64, device="cuda")), qb.QloraError),
                        ((q, None, torch.arange(6, device="cuda")[::2], f), ValueError)):
        with pytest.raises(error):
            qb.qlora_rope_fwd(*args)
    with pytest.raises(qb.QloraError, match="overlap"):
        qb.qlora_rope_fwd(q, None, p, f, outs=(torch.empty(1, 2, 64, device="cuda").expand(3, 2, 64), None))
    with pytest.raises(ValueError):
        qb.qlora_rope_fwd(q, None, p, f, outs=(torch.empty_like(q), torch.empty_like(q)))
    with pytest.raises(ValueError):
        qb.qlora_rope_fwd(q, None, p, f, outs=(torch.empty(3, 3, 64, device="cuda"), None))


@pytest.mark.parametrize("interleaved", [False, True])
def test_more_workgroups_than_one_launch_takes(qb, interleaved):
    """Heads of 1024 elements that begin at an odd one have a workgroup to a token: 2^21 of them to a launch, three
    launches here, and elements behind 2^32. The rows at the launches' ends are bit for bit what they are in a call of
    their own, with other outputs and in place, and the others stay zero."""
    import torch
    gu.announce(f"rope in three launches {interleaved}")
    f, _ = qb.qlora_rope_freqs(1024, device="cuda")
    rows, at = 2 * (1 << 21) + 3, torch.tensor([0, (1 << 21) - 1, 1 << 21, (1 << 22) - 1, 1 << 22, (1 << 22) + 2], device="cuda")
    flat = torch.zeros(rows * 1024 + 1, dtype=torch.bfloat16, device="cuda")
    x = flat[1:].view(rows, 1, 1024)
    x[at] = torch.randn(len(at), 1, 1024, device="cuda").bfloat16()
    p = torch.arange(rows, device="cuda")
    few = torch.zeros(len(at) * 1024 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(len(at), 1, 1024)
    few.copy_(x[at])
    want = qb.qlora_rope_fwd(few, None, p[at].contiguous(), f, interleaved=interleaved)[0]
    check(want, few, p[at].cpu().numpy(), host64(f), 1.0, interleaved, False, "few")
    y, _ = qb.qlora_rope_fwd(x, None, p, f, interleaved=interleaved)
    qb.qlora_rope_fwd(x, None, p, f, interleaved=interleaved, outs=(x, None))
    for t in (y, x):
        assert torch.equal(t[at], want)
        t[at] = 0
        assert not t.any()
