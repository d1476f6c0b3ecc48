"""Python binding of what stands between a decoder layer's projections
(include/qlora_block.h): the gated feed-forward product and rotary positions.

As in the package itself, the functions carry the names of the C entry points
and only marshal arguments: torch supplies device memory and the current
stream of the tensors' device. They are re-exported by the package.
"""
from __future__ import annotations

import ctypes
from ctypes import byref
from typing import Optional, Tuple

import torch

from . import NF4Weight, QloraError, _Weight, format_has_dq, lib, qlora_last_error
from .mx import _DTYPES, _MX, MXMatrix, QLORA_MX_FP8, _empty, _empty_1d, _entry, _fast, _fast_on, _tensor

__all__ = [
    "BLOCK_EXPORTED_SYMBOLS", "QLORA_ROPE_PLAIN", "QLORA_ROPE_LINEAR", "QLORA_ROPE_NTK", "QLORA_ROPE_PARTS",
    "qlora_mx_pair", "qlora_mx_gated", "qlora_mx_gated_grouped", "qlora_gated_saved_cols",
    "qlora_gated_workspace_bytes", "qlora_gated_fwd", "qlora_gated_fwd_save", "qlora_gated_bwd", "qlora_rope_freqs",
    "qlora_rope_fwd", "qlora_rope_bwd",
]

BLOCK_EXPORTED_SYMBOLS = (
    "qlora_mx_pair", "qlora_mx_gated", "qlora_mx_gated_grouped", "qlora_gated_saved_cols",
    "qlora_gated_workspace_bytes", "qlora_gated_fwd", "qlora_gated_bwd", "qlora_rope_freqs", "qlora_rope_fwd",
    "qlora_rope_bwd",
)

QLORA_ROPE_PLAIN = 0    # the frequencies as they are
QLORA_ROPE_LINEAR = 1   # positions pressed together
QLORA_ROPE_NTK = 2      # a larger base
QLORA_ROPE_PARTS = 3    # by parts: fast pairs as they are, slow ones pressed together


class _Adapters(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in ("gate_A", "gate_B", "up_A", "up_B")] + \
        [("r", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class _Grads(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in ("gate_A", "gate_B", "up_A", "up_B")]


class _Heads(ctypes.Structure):
    _fields_ = [("inp", ctypes.c_void_p), ("out", ctypes.c_void_p)] + \
        [(name, ctypes.c_int64) for name in ("heads", "in_row", "in_head", "out_row", "out_head")]


def _declare():
    i64, vp, i32, f64, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32, ctypes.c_double, ctypes.c_int
    mp, hp, dp = ctypes.POINTER(_MX), ctypes.POINTER(_Heads), ctypes.POINTER(ctypes.c_double)
    wp, ap, gp, sz = ctypes.POINTER(_Weight), ctypes.POINTER(_Adapters), ctypes.POINTER(_Grads), ctypes.c_size_t
    rope = [hp, hp, ci, i64, i32, i32, vp, i32, vp, f64, i32, vp]
    sigs = {
        "qlora_mx_pair": (ci, [mp, mp, mp, vp]),
        "qlora_mx_gated": (ci, [mp, mp, vp, mp, vp]),
        "qlora_mx_gated_grouped": (ci, [mp, mp, vp, i32, vp, mp, i32, vp]),
        "qlora_gated_saved_cols": (i64, [i32]),
        "qlora_gated_workspace_bytes": (sz, [i64, i64, i64, i32, i32]),
        "qlora_gated_fwd": (ci, [vp, i64, wp, wp, ap, vp, vp, vp, vp, vp, sz, vp]),
        "qlora_gated_bwd": (ci, [vp, vp, vp, vp, vp, i64, wp, wp, ap, vp, gp, vp, sz, vp]),
        "qlora_rope_freqs": (ci, [i32, f64, i32, f64, i64, f64, f64, dp, dp]),
        "qlora_rope_fwd": (ci, rope),
        "qlora_rope_bwd": (ci, rope),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args


_declare()

_pair, _gated, _gated_grouped = _entry("qlora_mx_pair"), _entry("qlora_mx_gated"), _entry("qlora_mx_gated_grouped")
_block_fwd, _block_bwd = _entry("qlora_gated_fwd"), _entry("qlora_gated_bwd")
_rope_fwd, _rope_bwd = _entry("qlora_rope_fwd"), _entry("qlora_rope_bwd")


def qlora_mx_pair(gate: MXMatrix, up: MXMatrix, out: Optional[MXMatrix] = None) -> MXMatrix:
    """The pair [2 N, K] of two 4-bit weights [N, K], N a multiple of 8, that
    qlora_mx_gated reads: eight rows of each in turn."""
    sg = gate.c_struct("gate")
    index = gate.codes.get_device()
    su = up.c_struct("up", index)
    if out is None:
        out = MXMatrix.empty(2 * gate.rows, gate.cols, gate.codes.device, gate.mx)
    _pair(index, byref(sg), byref(su), byref(out.c_struct("out", index)))
    return out


def _gated_out(X, index, N, mx, out):
    """H and how the entry point takes it: (result, address of a bf16 H, struct of a microscaled one). A given ``out``
    decides, whatever ``mx`` is."""
    if N % 32:
        raise ValueError(f"H would have {N} columns: a pair has a multiple of 64 rows")
    if out is None:
        if mx is None:
            out = _empty(X.rows, N, torch.bfloat16, X.codes.device)
        else:
            out = MXMatrix.empty(X.rows, N, X.codes.device, mx)
    if isinstance(out, MXMatrix):
        return out, None, byref(out.c_struct("out", index))
    return out, _tensor("out", out, torch.bfloat16, (X.rows, N), index), None


def qlora_mx_gated(X: MXMatrix, W: MXMatrix, mx: Optional[int] = QLORA_MX_FP8, out=None):
    """H = silu(X Wg^T) * (X Wu^T), W the pair [2 N, K] of both weights (N a
    multiple of 32): a new matrix in microscaled floats of type ``mx`` (what the
    down projection takes), a new bf16 tensor [M, N] with ``mx`` None, or
    ``out``, which is one or the other and decides."""
    if out is None and (at := _fast_on(X.codes)):
        new = _fast.gated(*at, X.codes, X.scales, X.rows, X.cols, X.mx, W.codes, W.scales, W.rows, W.cols, W.mx, mx)
        if new is not None:
            return new if mx is None else MXMatrix(X.rows, W.rows // 2, *new, mx)
    sx = X.c_struct("X")
    index = X.codes.get_device()
    sw = W.c_struct("W", index)
    out, h, hq = _gated_out(X, index, W.rows // 2, mx, out)
    _gated(index, byref(sx), byref(sw), h, hq)
    return out


def qlora_mx_gated_grouped(X: MXMatrix, W: MXMatrix, offsets, mx: Optional[int] = QLORA_MX_FP8, out=None):
    """qlora_mx_gated by expert: X [M, K] with its rows sorted by expert, W
    [experts * 2 N, K] the experts' pairs one below the other, offsets int32
    [experts + 1] on the device. Rows that no expert has are left as they were
    (zero in a new H)."""
    if out is None and (at := _fast_on(X.codes)):
        new = _fast.gated(*at, X.codes, X.scales, X.rows, X.cols, X.mx, W.codes, W.scales, W.rows, W.cols, W.mx, mx, offsets)
        if new is not None:
            return new if mx is None else MXMatrix(X.rows, W.rows // 2 // (offsets.shape[0] - 1), *new, mx)
    sx = X.c_struct("X")
    index = X.codes.get_device()
    sw = W.c_struct("W", index)
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets must be a tensor [experts + 1]")
    off = _tensor("offsets", offsets, torch.int32, offsets.shape, index)
    experts = offsets.shape[0] - 1
    if W.rows % (2 * experts):
        raise ValueError(f"W has {W.rows} rows, not a multiple of two for each of {experts} experts")
    clear = out is None
    out, h, hq = _gated_out(X, index, W.rows // experts // 2, mx, out)
    _gated_grouped(index, byref(sx), byref(sw), off, experts, h, hq, clear)
    return out


def qlora_gated_saved_cols(r: int) -> int:
    """Columns of the kept adapter activations of adapters of rank ``r``."""
    return int(lib.qlora_gated_saved_cols(r))


def qlora_gated_workspace_bytes(M: int, N: int, K: int, r: int, backward: bool) -> int:
    return int(lib.qlora_gated_workspace_bytes(M, N, K, r, bool(backward)))


def _weight(name, W: NF4Weight, index):
    """The C struct of a weight, after checking its buffers against its shape and format."""
    n = W.rows * W.cols
    blocks = -(-n // 64)
    if format_has_dq(W.fmt):
        parts = (("absmax_q", torch.int8, blocks), ("dq_scale", torch.float32, -(-blocks // 256)), ("dq_mean", torch.float32, 1))
    else:
        parts = (("absmax", torch.float32, blocks),)
    for part, dtype, count in (("codes", torch.uint8, (n + 1) // 2),) + parts:
        _tensor(f"{name}.{part}", getattr(W, part), dtype, (count,), index)
    return W.c_struct()


def _block_args(X, gate, up, Ag, Bg, Au, Bu, scale):
    """(M, N, K, r, device index, the two weights' structs, the adapters' struct or None, their type)"""
    if not isinstance(X, torch.Tensor) or not X.is_cuda:
        raise TypeError("X must be a CUDA (HIP) tensor")
    index, N, K = X.get_device(), gate.rows, gate.cols
    if X.dim() != 2 or X.shape[0] < 1:
        raise ValueError(f"X must be [M, {K}] with M >= 1, got {tuple(X.shape)}")
    M = X.shape[0]
    _tensor("X", X, torch.bfloat16, (M, K), index)
    sg, su = _weight("gate", gate, index), _weight("up", up, index)
    factors = (Ag, Bg, Au, Bu)
    if all(t is None for t in factors):
        return M, N, K, 0, index, sg, su, None, None
    if any(t is None for t in factors):
        raise ValueError("Ag, Bg, Au and Bu must all be given or all be None")
    if not isinstance(Ag, torch.Tensor) or Ag.dim() != 2 or Ag.shape[0] < 1:
        raise ValueError(f"Ag must be a tensor [r, {K}] with r >= 1")
    r, dtype = Ag.shape[0], Ag.dtype
    if dtype not in _DTYPES:
        raise TypeError(f"the adapters must be float32 or bfloat16, got {dtype}")
    at = [_tensor(name, t, dtype, shape, index)
          for name, t, shape in zip(("Ag", "Bg", "Au", "Bu"), factors, ((r, K), (N, r), (r, K), (N, r)))]
    return M, N, K, r, index, sg, su, _Adapters(*at, r, _DTYPES[dtype], float(scale)), dtype


def _block_ws(ws, M, N, K, r, backward, index, device):
    """(address, bytes, tensor) of the workspace; nothing of it is expected or kept."""
    if ws is None:
        ws = _empty_1d(lib.qlora_gated_workspace_bytes(M, N, K, r, backward), torch.uint8, device)
    else:
        _tensor("ws", ws, None, ws.shape, index)
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


def _given(t, name, shape, dtype, index, device):
    """``t`` after its checks, or a new tensor."""
    if t is None:
        return _empty(*shape, dtype, device)
    _tensor(name, t, dtype, shape, index)
    return t


def _parts(W: NF4Weight):
    return W.rows, W.cols, W.codes, W.absmax_q, W.dq_scale, W.dq_mean, W.absmax, W.fmt


def qlora_gated_fwd(X, gate: NF4Weight, up: NF4Weight, Ag=None, Bg=None, Au=None, Bu=None, scale: float = 0.0, ws=None, out=None):
    """H = silu(G) * U, G = X Wg^T + scale (X Ag^T) Bg^T and U likewise: X bf16
    [M, K], two frozen 4-bit weights [N, K] of one format, adapters A [r, K] and
    B [N, r] in fp32 or bf16 (all four or none). H bf16 [M, N]."""
    if ws is None and out is None and (at := _fast_on(X)):
        new = _fast.block(*at, X, *_parts(gate), *_parts(up), Ag, Bg, Au, Bu, scale, False)
        if new is not None:
            return new
    M, N, K, r, index, sg, su, ad, _ = _block_args(X, gate, up, Ag, Bg, Au, Bu, scale)
    out = _given(out, "out", (M, N), torch.bfloat16, index, X.device)
    at, size, ws = _block_ws(ws, M, N, K, r, False, index, X.device)
    _block_fwd(index, X.data_ptr(), M, byref(sg), byref(su), ad and byref(ad), out.data_ptr(), None, None, None, at, size)
    return out


def qlora_gated_fwd_save(X, gate: NF4Weight, up: NF4Weight, Ag=None, Bg=None, Au=None, Bu=None, scale: float = 0.0, ws=None,
                         outs: Optional[Tuple] = None):
    """(H, G, U, Hs): qlora_gated_fwd's H and what qlora_gated_bwd takes: G and U
    in bf16 and the adapter activations Hs bf16 [M, qlora_gated_saved_cols(r)]
    (None without adapters)."""
    if ws is None and outs is None and (at := _fast_on(X)):
        new = _fast.block(*at, X, *_parts(gate), *_parts(up), Ag, Bg, Au, Bu, scale, True)
        if new is not None:
            return new
    M, N, K, r, index, sg, su, ad, _ = _block_args(X, gate, up, Ag, Bg, Au, Bu, scale)
    H, G, U, Hs = (None,) * 4 if outs is None else outs
    H, G, U = (_given(t, name, (M, N), torch.bfloat16, index, X.device) for name, t in (("H", H), ("G", G), ("U", U)))
    if r:
        Hs = _given(Hs, "Hs", (M, lib.qlora_gated_saved_cols(r)), torch.bfloat16, index, X.device)
    elif Hs is not None:
        raise ValueError("without adapters Hs must be None")
    at, size, ws = _block_ws(ws, M, N, K, r, False, index, X.device)
    _block_fwd(index, X.data_ptr(), M, byref(sg), byref(su), ad and byref(ad), H.data_ptr(), G.data_ptr(), U.data_ptr(),
               Hs.data_ptr() if r else None, at, size)
    return H, G, U, Hs


def qlora_gated_bwd(dH, X, G, U, Hs, gate: NF4Weight, up: NF4Weight, Ag=None, Bg=None, Au=None, Bu=None, scale: float = 0.0,
                    ws=None, outs: Optional[Tuple] = None):
    """(dX, dAg, dBg, dAu, dBu) from the gradient of H and what
    qlora_gated_fwd_save kept, with its arguments: dX bf16, the others in the
    adapters' type (None without adapters). The weights get no gradient."""
    if ws is None and outs is None and (at := _fast_on(X)):
        new = _fast.block_bwd(*at, dH, X, G, U, Hs, *_parts(gate), *_parts(up), Ag, Bg, Au, Bu, scale)
        if new is not None:
            return new
    M, N, K, r, index, sg, su, ad, dtype = _block_args(X, gate, up, Ag, Bg, Au, Bu, scale)
    ins = [_tensor(name, t, torch.bfloat16, (M, N), index) for name, t in (("dH", dH), ("G", G), ("U", U))]
    dX, *grads = (None,) * 5 if outs is None else outs
    dX = _given(dX, "dX", (M, K), torch.bfloat16, index, X.device)
    hs = sgr = None
    if r:
        hs = _tensor("Hs", Hs, torch.bfloat16, (M, lib.qlora_gated_saved_cols(r)), index)
        grads = [_given(t, name, shape, dtype, index, X.device)
                 for t, name, shape in zip(grads, ("dAg", "dBg", "dAu", "dBu"), ((r, K), (N, r), (r, K), (N, r)))]
        sgr = _Grads(*(t.data_ptr() for t in grads))
    elif Hs is not None or any(t is not None for t in grads):
        raise ValueError("without adapters Hs and their gradients must be None")
    at, size, ws = _block_ws(ws, M, N, K, r, True, index, X.device)
    _block_bwd(index, ins[0], X.data_ptr(), ins[1], ins[2], hs, M, byref(sg), byref(su), ad and byref(ad), dX.data_ptr(),
               sgr and byref(sgr), at, size)
    return (dX, *grads)


def qlora_rope_freqs(rot: int, base: float = 10000.0, scaling: int = QLORA_ROPE_PLAIN, factor: float = 1.0,
                     trained: int = 4096, low: float = 1.0, high: float = 32.0, device=None):
    """(freqs, amplitude): fp64 [rot / 2], radians a position of each pair, and
    the factor of the rotated values, for a context ``factor`` times as long as
    the ``trained`` positions. Formed once and kept with the model."""
    if rot < 2 or rot % 2:
        raise ValueError(f"rot must be even and at least 2, got {rot}")
    freqs, amplitude = (ctypes.c_double * (rot // 2))(), ctypes.c_double()
    status = lib.qlora_rope_freqs(rot, float(base), scaling, float(factor), int(trained), float(low), float(high), freqs, byref(amplitude))
    if status != 0:
        raise QloraError("qlora_rope_freqs", status, qlora_last_error())
    return torch.tensor(list(freqs), dtype=torch.float64, device=device), amplitude.value


def _heads(name, t, out, dtype, shape, index):
    """The C struct of heads [rows, heads, dim] and of their output, the elements of a head next to each other."""
    for what, x in ((name, t), (f"out {name}", out)):
        if not isinstance(x, torch.Tensor) or not x.is_cuda:
            raise TypeError(f"{what} must be a CUDA (HIP) tensor")
        if x.dtype is not dtype:
            raise TypeError(f"{what} must be {dtype}, got {x.dtype}")
        if x.dim() != 3 or x.numel() == 0 or (x.shape[0], x.shape[2]) != shape or x.shape[1] != t.shape[1]:
            raise ValueError(f"{what} must be [{shape[0]}, heads, {shape[1]}], got {tuple(x.shape)}")
        if x.stride(2) != 1:
            raise ValueError(f"the elements of a head of {what} must lie next to each other")
        if x.get_device() != index:
            raise ValueError(f"{what} is on {x.device}, expected cuda:{index}")
    return _Heads(t.data_ptr(), out.data_ptr(), t.shape[1], t.stride(0), t.stride(1), out.stride(0), out.stride(1))


def _rope(backward, Q, K, positions, freqs, amplitude, interleaved, outs):
    if outs is None and (at := _fast_on(Q)):
        new = _fast.rope(*at, Q, K, positions, freqs, amplitude, bool(interleaved), backward)
        if new is not None:
            return new
    if not isinstance(Q, torch.Tensor) or not Q.is_cuda:
        raise TypeError("the heads must be CUDA (HIP) tensors")
    if Q.dim() != 3:
        raise ValueError(f"the heads must be [rows, heads, dim], got {tuple(Q.shape)}")
    if Q.dtype not in _DTYPES:
        raise TypeError(f"the heads must be float32 or bfloat16, got {Q.dtype}")
    index, rows, dim = Q.get_device(), Q.shape[0], Q.shape[2]
    if not isinstance(positions, torch.Tensor) or positions.dtype not in (torch.int32, torch.int64):
        raise TypeError("positions must be an int32 or int64 tensor")
    pos = _tensor("positions", positions, None, (rows,), index)
    if not isinstance(freqs, torch.Tensor) or freqs.dim() != 1:
        raise ValueError("freqs must be a tensor [rot / 2]")
    f = _tensor("freqs", freqs, torch.float64, freqs.shape, index)
    if outs is None:
        q, k = torch.empty(Q.shape, dtype=Q.dtype, device=Q.device), None
        if K is not None:
            k = torch.empty(K.shape, dtype=Q.dtype, device=Q.device) if isinstance(K, torch.Tensor) else K
    else:
        q, k = outs
        if (K is None) != (k is None):
            raise ValueError("outs must have what there are heads for")
    sq = _heads("Q", Q, q, Q.dtype, (rows, dim), index)
    sk = None if K is None else _heads("K", K, k, Q.dtype, (rows, dim), index)
    entry = _rope_bwd if backward else _rope_fwd
    entry(index, byref(sq), None if sk is None else byref(sk), _DTYPES[Q.dtype], rows, dim, 2 * freqs.shape[0], pos,
          positions.dtype is torch.int64, f, float(amplitude), bool(interleaved))
    return q, k


def qlora_rope_fwd(Q, K, positions, freqs, amplitude: float = 1.0, interleaved: bool = False,
                   outs: Optional[Tuple] = None):
    """(Q', K'): the heads [rows, heads, dim] (fp32 or bf16, any strides of rows
    and heads) rotated by their positions [rows] (int32 or int64). The first 2
    len(freqs) elements of a head are rotated, element i with i + len(freqs) or,
    ``interleaved``, 2 i with 2 i + 1; the others pass through. K may be None.
    ``outs`` may be (Q, K) themselves."""
    return _rope(False, Q, K, positions, freqs, amplitude, interleaved, outs)


def qlora_rope_bwd(dQ, dK, positions, freqs, amplitude: float = 1.0, interleaved: bool = False,
                   outs: Optional[Tuple] = None):
    """(gradients of Q and K) of qlora_rope_fwd from those of its outputs; with the same arguments as it."""
    return _rope(True, dQ, dK, positions, freqs, amplitude, interleaved, outs)
