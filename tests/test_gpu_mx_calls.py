"""The microscaled and norm calls in the ways a program makes them: without the
host accelerator, captured and replayed with other contents, through autograd."""
import numpy as np
import pytest

from tests import gpu_util as gu
from tests.test_gpu_mx import qb  # noqa: F401  (qb: the fixture)

pytestmark = pytest.mark.gpu


def test_calls_without_fastcall(qb, monkeypatch):  # noqa: F811
    """Every call with new outputs gives the same bits without _fastcall.so."""
    import torch
    import bit_nf4_quantized_03_amd.mx as binding
    assert binding._fast is not None, "_fastcall.so is not built"
    x, res, dy, dh = (torch.randn(70, 544, device="cuda").bfloat16() for _ in range(4))
    g = torch.rand(544, device="cuda") + 0.5
    w = qb.qlora_mx_quantize(torch.randn(96, 544, device="cuda"))

    def tensors(out):
        if isinstance(out, qb.MXMatrix):
            return [out.codes, out.scales]
        return [t for o in out for t in tensors(o)] if isinstance(out, tuple) else [out]

    def calls():
        q = qb.qlora_mx_quantize(x, qb.QLORA_MX_FP8)
        y, h, rstd = qb.qlora_rmsnorm_fwd(x, g, 1e-6, residual=res)
        outs = (q, qb.qlora_mx_dequantize(q, torch.bfloat16), qb.qlora_mx_dequantize(w), (y, h, rstd),
                qb.qlora_rmsnorm_mx(x, g, 1e-6, residual=res), qb.qlora_rmsnorm_mx(x, g, 1e-6, mx=qb.QLORA_MX_FP4)[0],
                qb.qlora_rmsnorm_bwd(dy, h, g, rstd, dH=dh), qb.qlora_mx_linear(q, w))
        return tensors(outs)
    gu.announce("mx calls with _fastcall")
    with_it = calls()
    gu.announce("mx calls without _fastcall")
    monkeypatch.setattr(binding, "_fast", None)
    without = calls()
    assert len(with_it) == len(without) and all(torch.equal(a, b) for a, b in zip(with_it, without))


# Offsets to replay a capture with: the rows of all experts move, M and the experts stay.
def _offsets(M, E):
    yield np.linspace(0, M, E + 1).astype(int)                 # evenly
    yield np.array([0] + [M] * E)                              # the first expert has every row
    yield np.array([0] * E + [M])                              # the last one
    yield np.array([0] * (E // 2 + 1) + [M] * (E - E // 2))    # one in the middle
    yield np.full(E + 1, M // 2)                               # no expert has a row
    front, end = M // 5, M - M // 3
    yield np.concatenate([[front], np.sort(np.random.default_rng(M).integers(front, end + 1, E - 1)), [end]])   # rows without one


@pytest.mark.parametrize("t", [0, 1])
@pytest.mark.parametrize("M,E,N,K", [(40, 8, 100, 544), (128, 16, 64, 1056),                     # the stream of few rows
                                     (200, 8, 100, 544), (600, 4, 264, 1056), (2000, 3, 512, 288)])   # tiles
def test_capture_replayed_with_other_offsets(qb, M, E, N, K, t):  # noqa: F811
    """One capture of the product by expert serves whatever the offsets hold when it is replayed."""
    import torch
    torch.manual_seed(M)
    X = qb.qlora_mx_quantize(torch.randn(M, K, device="cuda"), t)
    W = qb.qlora_mx_quantize(torch.randn(E * N, K, device="cuda"))
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")

    def both():
        qb.qlora_mx_linear_grouped(X, W, off, out=out)
        return qb.qlora_mx_linear_grouped(X, W, off)
    gu.announce(f"mx grouped captured M={M} E={E} N={N} K={K} type {t}")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        new = both()
    every = qb.MXMatrix(N * E, K, W.codes, W.scales, W.mx)
    for i, at in enumerate(_offsets(M, E)):
        gu.announce(f"  replay {i}: {at[:12].tolist()}")
        off.copy_(torch.tensor(at, dtype=torch.int32))
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        got, got_new = out.clone(), new.clone()
        out.fill_(9.0)
        want_new = both()
        assert torch.equal(got, out) and torch.equal(got_new, want_new), f"replay {i}"
        # and it is the product: each row against its expert's columns of the product with all weights
        wide = qb.qlora_mx_linear(X, every).float().view(M, E, N)
        mag = (qb.qlora_mx_dequantize(X).abs() @ qb.qlora_mx_dequantize(W).abs().t()).view(M, E, N)
        for e in range(E):
            a, b = int(at[e]), int(at[e + 1])
            # two results, each within product_bound (K additions, the instruction's cut, half a step) of the exact
            # sum; a twentieth more because the bound is taken from the rounded one
            bound = 2.0 ** -8 * wide[a:b, e].abs() + (K * 2.0 ** -23 + (7 * 2.0 ** -12 if t else 0.0)) * mag[a:b, e]
            assert ((got[a:b].float() - wide[a:b, e]).abs() <= 2.1 * bound).all(), (i, e)
        none = torch.ones(M, dtype=torch.bool)
        none[int(at[0]):int(at[-1])] = False
        assert (got[none.cuda()] == 9.0).all() and (got_new[none.cuda()] == 0.0).all()


def test_autograd_norm_captured(qb):  # noqa: F811
    """The forward and backward of autograd.rmsnorm in one capture, replayed with new inputs and gradients in the
    captured buffers and checked against the raw calls. (No eager graph of these leaves is alive.)"""
    import torch
    from bit_nf4_quantized_03_amd.autograd import rmsnorm
    gu.announce("autograd norm captured")
    x, r = (torch.randn(300, 1024, device="cuda").bfloat16().requires_grad_(True) for _ in range(2))
    g = (torch.rand(1024, device="cuda") + 0.5).requires_grad_(True)
    dy, dh = (torch.randn(300, 1024, device="cuda").bfloat16() for _ in range(2))

    def step():
        y, h = rmsnorm(x, g, r)
        return (y.detach(), h.detach(), *torch.autograd.grad((y, h), (x, r, g), (dy, dh)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(3):
        gu.announce(f"  replay {i}")
        with torch.no_grad():
            for t in (x, r, dy, dh):
                t.copy_(torch.randn(300, 1024, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        y, h, rstd = qb.qlora_rmsnorm_fwd(x.detach(), g.detach(), 1e-6, residual=r.detach())
        dx, dw = qb.qlora_rmsnorm_bwd(dy, h, g.detach(), rstd, dH=dh)
        for a, b in zip(outs, (y, h, dx, dx, dw)):
            assert torch.equal(a, b), f"replay {i}"


def test_autograd_norm_of_views(qb):  # noqa: F811
    """Inputs and gradients that begin 2 bytes behind a 16-byte border, or lie transposed."""
    import torch
    from bit_nf4_quantized_03_amd.autograd import rmsnorm
    gu.announce("autograd norm of views")
    x, r, dy, dh = (torch.randn(40, 160, device="cuda").bfloat16() for _ in range(4))
    g = torch.rand(160, device="cuda") + 0.5

    def run(turn):
        a, b = (turn(t).requires_grad_(True) for t in (x, r))
        torch.autograd.backward(rmsnorm(a, g, b), [turn(dy), turn(dh)])
        return a.grad, b.grad
    want = run(lambda t: t.clone())
    shifted = run(lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(40, 160))
    turned = run(lambda t: t.t().contiguous().t())
    for got in (shifted, turned):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_norm_over_its_input_has_no_h(qb):  # noqa: F811
    """Without a residual H is X; where the output takes X's place there is none, and the backward refuses that."""
    import torch
    gu.announce("rmsnorm over its input")
    x, g = torch.randn(5, 96, device="cuda").bfloat16(), torch.rand(96, device="cuda") + 0.5
    y, h, rstd = qb.qlora_rmsnorm_fwd(x, g)
    assert h is x
    z = x.clone()
    y2, h2, rstd2 = qb.qlora_rmsnorm_fwd(z, g, out=z)
    assert y2 is z and torch.equal(y2, y) and torch.equal(rstd2, rstd) and h2 is None
    with pytest.raises(TypeError):
        qb.qlora_rmsnorm_bwd(y, h2, g, rstd2)
    y3, h3, _ = qb.qlora_rmsnorm_fwd(x, g, out=torch.empty_like(x))
    assert h3 is x and torch.equal(y3, y)


_WAITING = """
import sys, threading, time, torch
import bit_nf4_quantized_03_amd as qb
import bit_nf4_quantized_03_amd.mx as binding
assert binding._fast is not None
x, res, dy = (torch.randn(64, 512, device="cuda").bfloat16() for _ in range(3))
g = torch.ones(512, device="cuda")
q = qb.qlora_mx_quantize(x)
y, h, rstd = qb.qlora_rmsnorm_fwd(x, g, residual=res)
calls = {
    "quantize": lambda: qb.qlora_mx_quantize(x), "dequantize": lambda: qb.qlora_mx_dequantize(q), "linear": lambda: qb.qlora_mx_linear(q, q),
    "norm": lambda: qb.qlora_rmsnorm_fwd(x, g, residual=res), "norm mx": lambda: qb.qlora_rmsnorm_mx(x, g, residual=res),
    "backward": lambda: qb.qlora_rmsnorm_bwd(dy, h, g, rstd)}
for f in calls.values():
    f()
torch.cuda.synchronize()
a = time.perf_counter()
torch.cuda._sleep(1 << 22)
torch.cuda.synchronize()
cycles = int((1 << 22) * 0.2 / (time.perf_counter() - a))   # of a fifth of a second at the most
print(f"{cycles} cycles", flush=True)
ticks = []
def count():
    while True:
        ticks.append(time.perf_counter())
        time.sleep(0.0005)
threading.Thread(target=count, daemon=True).start()
for name, f in calls.items():
    busy = threading.Thread(target=torch.cuda._sleep, args=(cycles,), daemon=True)   # on this thread's stream, the default one
    busy.start()
    time.sleep(0.02)
    a = time.perf_counter()
    f()
    b = time.perf_counter()
    busy.join()
    torch.cuda.synchronize()
    inside = [a] + [v for v in ticks if a < v < b] + [b]
    gap = max(q - p for p, q in zip(inside, inside[1:]))
    print(f"{name}: waited {(b - a) * 1e3:.1f} ms, the other thread at most {gap * 1e3:.1f}", flush=True)
    assert b - a > 0.02, "the call does not wait"
    assert gap < 0.5 * (b - a), name
print("all fine", flush=True)
"""


def test_other_threads_run_while_a_call_waits(qb):  # noqa: F811
    """Where launches wait for their kernel (a process with AMD_SERIALIZE_KERNEL=3) and a thread keeps the stream busy,
    a third thread of the program goes on while a call waits."""
    import os
    import subprocess
    import sys
    gu.announce("calls that wait, in a process of their own")
    r = subprocess.run([sys.executable, "-u", "-c", _WAITING], cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       env=dict(os.environ, AMD_SERIALIZE_KERNEL="3"), capture_output=True, text=True, timeout=40)
    print(r.stdout)
    assert r.returncode == 0 and "all fine" in r.stdout, r.stdout + r.stderr
