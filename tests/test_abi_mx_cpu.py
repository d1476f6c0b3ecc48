"""C-ABI checks of include/qlora_mx.h that need no GPU: exports, sizes, and
invalid arguments rejected on the host with a message before anything is
launched."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qlora_mx.h")

qb = pytest.importorskip("bit_nf4_quantized_03_amd")
from bit_nf4_quantized_03_amd import mx as binding  # noqa: E402

lib = qb.lib
ref = ctypes.byref
# never dereferenced: every call below fails before a launch
FAKE = 1 << 20
BF16, F32, FP4, FP8 = qb.QLORA_BF16, qb.QLORA_F32, qb.QLORA_MX_FP4, qb.QLORA_MX_FP8


def M(rows=64, cols=64, codes=FAKE, scales=FAKE, type=FP4):
    return binding._MX(rows, cols, codes, scales, type)


def test_every_declared_symbol_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(qlora_[a-z0-9_]+)\s*\(", text)))
    assert sorted(qb.MX_EXPORTED_SYMBOLS) == names
    for name in names:
        assert hasattr(lib, name), name
        assert name in qb.__all__ and hasattr(qb, name), name


def test_sizes():
    assert [qb.qlora_mx_scale_pitch(c) for c in (32, 512, 544, 4096, 11008, 1 << 22)] == [16, 16, 32, 128, 352, 131072]
    assert [qb.qlora_mx_scale_pitch(c) for c in (0, -32, 33, (1 << 22) + 32)] == [0, 0, 0, 0]
    assert qb.qlora_mx_storage_bytes(3, 64, FP4) == 3 * (32 + 16)
    assert qb.qlora_mx_storage_bytes(3, 64, FP8) == 3 * (64 + 16)
    assert qb.qlora_mx_storage_bytes(3, 64, 2) == qb.qlora_mx_storage_bytes(0, 64, 0) == qb.qlora_mx_storage_bytes(3, 65, 0) == 0
    assert qb.qlora_mx_storage_bytes(1 << 40, 64, 0) == 0
    assert qb.qlora_rmsnorm_bwd_workspace_bytes(1, 32) == 0 and qb.qlora_rmsnorm_bwd_workspace_bytes(100, 64) >= 512
    assert qb.qlora_rmsnorm_bwd_workspace_bytes(1, 32800) == qb.qlora_rmsnorm_bwd_workspace_bytes(0, 64) == 0
    assert qb.qlora_rmsnorm_bwd_workspace_bytes(1 << 35, 64) == 0


def test_quantize_rejects():
    q = lib.qlora_mx_quantize
    assert q(None, BF16, 64, 64, ref(M()), None) == -1
    assert q(FAKE, 5, 64, 64, ref(M()), None) == -3
    assert q(FAKE, F32, 64, 64, None, None) == -1
    assert q(FAKE, F32, 64, 32, ref(M()), None) == -2
    assert q(FAKE, F32, 64, 48, ref(M(cols=48)), None) == -2
    assert q(FAKE, F32, 0, 64, ref(M(rows=0)), None) == -2
    assert q(FAKE, F32, 64, 64, ref(M(type=2)), None) == -7
    assert q(FAKE, F32, 64, 64, ref(M(codes=0)), None) == -1
    assert q(FAKE, F32, 64, 64, ref(M(scales=0)), None) == -1
    assert q(FAKE, F32, 64, 64, ref(M(scales=FAKE + 8)), None) == -6
    assert q(FAKE + 2, BF16, 64, 64, ref(M()), None) == -6
    assert "16-byte aligned" in qb.qlora_last_error()


def test_dequantize_rejects():
    d = lib.qlora_mx_dequantize
    assert d(None, FAKE, F32, None) == -1
    assert d(ref(M()), None, F32, None) == -1
    assert d(ref(M()), FAKE, 2, None) == -3
    assert d(ref(M()), FAKE + 4, F32, None) == -6
    assert d(ref(M(cols=1 << 23)), FAKE, F32, None) == -2


def test_norm_rejects():
    f = lib.qlora_rmsnorm_fwd
    ok = dict(X=FAKE, res=FAKE, w=FAKE, wt=F32, rows=4, cols=64, eps=1e-6, Y=2 * FAKE, H=FAKE, rstd=FAKE)

    def call(**kw):
        a = dict(ok, **kw)
        return f(a["X"], a["res"], a["w"], a["wt"], a["rows"], a["cols"], a["eps"], a["Y"], a["H"], a["rstd"], None)
    assert call(X=None) == call(w=None) == call(Y=None) == call(H=None) == -1
    assert call(res=None) == -2                     # H without a residual
    assert call(wt=3) == -3
    assert call(rows=0) == call(cols=0) == call(cols=40) == call(cols=32800) == call(rows=1 << 35) == -2
    assert call(eps=-1e-9) == call(eps=float("inf")) == call(eps=float("nan")) == -2
    assert call(Y=FAKE) == -2                       # Y is H
    for name in ("X", "res", "w", "Y", "H", "rstd"):
        assert call(**{name: 3 * FAKE + 4}) == -6, name
    g = lib.qlora_rmsnorm_mx
    assert g(FAKE, FAKE, FAKE, F32, 4, 64, 1e-6, None, FAKE, None) == -1
    assert g(FAKE, FAKE, FAKE, F32, 4, 64, 1e-6, ref(M(4, 96)), FAKE, None) == -2
    assert g(FAKE, FAKE, FAKE, F32, 4, 64, 1e-6, ref(M(4, 64, type=9)), FAKE, None) == -7
    assert g(FAKE, None, FAKE, F32, 4, 64, 1e-6, ref(M(4, 64)), FAKE, None) == -2
    b = lib.qlora_rmsnorm_bwd
    need = qb.qlora_rmsnorm_bwd_workspace_bytes(100, 64)
    args = [FAKE, FAKE, FAKE, F32, FAKE, None, 100, 64, 2 * FAKE, FAKE, FAKE, need, None]
    for i in (0, 1, 2, 4, 8, 9):
        bad = list(args)
        bad[i] = None
        assert b(*bad) == -1, i
    for i in (0, 1, 2, 4, 5, 8, 9, 10):
        bad = list(args)
        bad[i] = 3 * FAKE + 8
        assert b(*bad) == -6, i
    bad = list(args)
    bad[8] = FAKE                                   # dX is H
    assert b(*bad) == -2
    bad = list(args)
    bad[11] = need - 1
    assert b(*bad) == -4
    bad = list(args)
    bad[10] = None
    assert b(*bad) == -4


def test_products_reject():
    f = lib.qlora_mx_linear
    x = M(4, 64, type=FP8)
    assert f(None, ref(M()), FAKE, None) == f(ref(x), None, FAKE, None) == f(ref(x), ref(M()), None, None) == -1
    assert f(ref(x), ref(M(type=FP8)), FAKE, None) == -7
    assert f(ref(x), ref(M(cols=96)), FAKE, None) == -2
    assert f(ref(x), ref(M()), FAKE + 8, None) == -6
    for m, n in ((1 << 25, 1), (1, 1 << 25), (1 << 19, 1 << 19)):
        assert f(ref(M(m, 64, type=FP8)), ref(M(n, 64)), FAKE, None) == -2
    g = lib.qlora_mx_linear_grouped
    assert g(ref(x), ref(M()), None, 2, FAKE, None) == -1
    for e in (0, -1, 3, 1025):
        assert g(ref(x), ref(M()), FAKE, e, FAKE, None) == -2, e
    assert g(ref(x), ref(M()), FAKE + 2, 2, FAKE, None) == -6
    assert g(ref(M(1 << 25, 64, type=FP8)), ref(M()), FAKE, 2, FAKE, None) == -2
    assert g(ref(x), ref(M(1 << 29, 64)), FAKE, 1024, FAKE, None) == -2
    assert g(ref(x), ref(M(type=FP8)), FAKE, 2, FAKE, None) == -7


def test_binding_refuses_host_tensors():
    import torch
    t = torch.zeros(4, 64)
    with pytest.raises(TypeError):
        qb.qlora_mx_quantize(t)
    with pytest.raises(TypeError):
        qb.qlora_rmsnorm_fwd(t.to(torch.bfloat16), torch.ones(64))
    host = qb.MXMatrix.empty(4, 64, "cpu")
    with pytest.raises(TypeError):
        qb.qlora_mx_dequantize(host)
    with pytest.raises(TypeError):
        qb.qlora_mx_linear(host, host)
    for bad in ((0, 64), (4, 40), (4, 0)):
        with pytest.raises(ValueError):
            qb.MXMatrix.empty(*bad, "cpu")
    with pytest.raises(ValueError):
        qb.MXMatrix.empty(4, 64, "cpu", 5)
