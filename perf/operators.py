"""Cases and plain forms of the microscaled serving path and of the RMSNorm around it.

Four operators, each in a plain form of elementary torch operations (``own`` false) and as a
user calls it from this package (``own`` true):

* quantize:   a matrix to microscaled 4- or 8-bit floats (blocks of 32 along a row, one power of
              two per block) and back to the bf16 values that it stands for;
* norm:       RMSNorm with the residual's addition, its output in microscaled floats;
* norm_train: the same norm with a bf16 output, forward and backward;
* linear:     Y = X W^T, X in microscaled 8- or 4-bit floats, W in microscaled 4-bit floats;
* grouped:    the same product with one W per expert, the rows of X sorted by expert.

Layout of a microscaled matrix [rows, cols], cols a multiple of 32: codes row-major, 4-bit
elements two to a byte (the even one in the low half), 8-bit ones (e4m3) one to a byte; scales one
byte s per block, standing for 2^(s - 127), in rows of 16 ceil(cols / 512) bytes (zero padded).
A block's exponent is floor(log2 of its largest magnitude) minus that of the element type's
largest power of two (2 for 4 bits, 8 for 8 bits); elements round to nearest, ties to even, and
saturate.
"""
import math

import torch

own = False

EPS = 1e-6
# element type: bits of mantissa, exponent of the largest power of two, smallest normal exponent, largest value
TYPES = {"fp4": (1, 2, 0, 6.0), "fp8": (3, 8, -6, 448.0)}
FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # a 65B-width MLP weight brought to 4 bits when a model is loaded
        {"name": "quantize weight 22016x8192", "op": "quantize", "rows": 22016, "cols": 8192, "dtype": "bf16", "mx": "fp4"},
        # a ragged batch of MLP activations on their way into the down projection
        {"name": "quantize activations 37x11008", "op": "quantize", "rows": 37, "cols": 11008, "dtype": "bf16", "mx": "fp8"},
        # one token's residual stream before a projection: latency counts
        {"name": "norm 1x4096", "op": "norm", "rows": 1, "cols": 4096, "mx": "fp8", "residual": True, "weight": "bf16"},
        # a prompt of 4096 tokens at 7B width
        {"name": "norm 4096x4096", "op": "norm", "rows": 4096, "cols": 4096, "mx": "fp8", "residual": True, "weight": "fp32"},
        # an odd number of tokens at 65B width, first norm of a stack (no residual yet), forward and backward
        {"name": "norm train 777x8192", "op": "norm_train", "rows": 777, "cols": 8192, "residual": False, "weight": "bf16"},
        # a training step's norm at 7B width, forward and backward
        {"name": "norm train 4096x4096", "op": "norm_train", "rows": 4096, "cols": 4096, "residual": True, "weight": "fp32"},
        # the smallest decode product: one token, 7B gate / up projection
        {"name": "linear 1x11008x4096", "op": "linear", "M": 1, "N": 11008, "K": 4096, "mx": "fp8"},
        # a ragged prompt, between decode and training sizes, into the down projection
        {"name": "linear 301x4096x11008", "op": "linear", "M": 301, "N": 4096, "K": 11008, "mx": "fp8"},
        # a prompt of 4096 tokens through a 7B attention projection
        {"name": "linear 4096x4096x4096", "op": "linear", "M": 4096, "N": 4096, "K": 4096, "mx": "fp8"},
        # the largest: 65B up projection, activations in 4 bits too
        {"name": "linear 2048x22016x8192 fp4", "op": "linear", "M": 2048, "N": 22016, "K": 8192, "mx": "fp4"},
        # a decode batch over eight experts, some without a token, spare rows at the end of the buffers
        {"name": "grouped 8 experts 33 rows", "op": "grouped", "E": 8, "M": 33, "N": 11008, "K": 4096, "mx": "fp8", "skew": 1.0, "spare": 3},
        # a prompt over eight experts, unevenly spread
        {"name": "grouped 8 experts 4096 rows", "op": "grouped", "E": 8, "M": 4096, "N": 4096, "K": 4096, "mx": "fp8", "skew": 0.5, "spare": 0},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["quantize", "norm", "norm_train", "linear", "grouped"])
    mx = rng.choice(["fp4", "fp8", "fp8"])
    weight = rng.choice(["bf16", "fp32"])
    if op == "quantize":
        cols = 32 * _spread(rng, 1, 688)
        rows = _spread(rng, 1, min(22016, 22016 * 8192 // cols))
        return {"op": op, "rows": rows, "cols": cols, "dtype": weight, "mx": mx}
    if op in ("norm", "norm_train"):
        cols = 32 * _spread(rng, 4, 512)
        rows = _spread(rng, 1, min(8192, 4096 * 4096 // cols))
        case = {"op": op, "rows": rows, "cols": cols, "residual": rng.random() < 0.7, "weight": weight}
        return case if op == "norm_train" else dict(case, mx=mx)
    if op == "linear":
        K = 32 * _spread(rng, 4, 688)
        N = _spread(rng, 16, min(22016, 22016 * 8192 // K))
        M = _spread(rng, 1, 4096)
        M = min(M, 2048 * 22016 * 8192 // (N * K))
        return {"op": op, "M": M, "N": N, "K": K, "mx": mx}
    E = rng.randint(2, 24)
    K = 32 * _spread(rng, 8, 344)
    N = _spread(rng, 64, min(11008, 8 * 11008 * 4096 // (E * K)))
    M = _spread(rng, 1, 4096)
    return {"op": op, "E": E, "M": M, "N": N, "K": K, "mx": mx, "skew": round(rng.uniform(0.0, 1.5), 2), "spare": rng.choice([0, 0, 1, 5])}


# ------------------------------------------------------------------ plain forms

def _pow2(e, dtype):
    """2^e for whole e within the type's normal range."""
    if dtype == torch.float64:
        return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _plain_quantize(v, mx):
    """v [rows, cols] fp32 or fp64: the elements (in units of their block's power of two) and the block exponents."""
    mantissa, top, low, most = TYPES[mx]
    b = v.reshape(v.shape[0], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    exponent = (torch.frexp(amax)[1] - 1 - top).clamp(-126, 127)
    scaled = b * _pow2(-exponent, v.dtype)
    step = _pow2((torch.frexp(scaled)[1] - 1).clamp(min=low) - mantissa, v.dtype)
    return (torch.round(scaled / step) * step).clamp(-most, most), exponent


def _plain_values(v, mx):
    q, exponent = _plain_quantize(v, mx)
    return (q * _pow2(exponent, v.dtype)).reshape(v.shape).to(torch.bfloat16)


def _plain_scales(scales, blocks):
    s = scales[:, :blocks].to(torch.int32)
    return torch.where(s == 0, torch.full_like(s, 0x00400000), s << 23).view(torch.float32)


def _plain_matrix(codes, scales, cols, mx):
    """The fp32 values of a microscaled matrix."""
    if mx == "fp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(FP4 + tuple(-x for x in FP4), device=codes.device)
        v = table[torch.stack([codes & 15, codes >> 4], -1).to(torch.int32)]
    v = v.reshape(codes.shape[0], cols // 32, 32)
    return (v * _plain_scales(scales, cols // 32)[:, :, None]).reshape(codes.shape[0], cols)


def _plain_norm(x, residual, weight, dtype):
    h = x if residual is None else (x.float() + residual.float()).to(torch.bfloat16)
    d = h.to(dtype)
    rstd = 1.0 / torch.sqrt((d * d).mean(-1, keepdim=True) + EPS)
    return h, d, rstd, weight.to(dtype)


def _plain_run(s):
    c = s["case"]
    op = c["op"]
    if op == "quantize":
        return _plain_values(s["x"].float(), c["mx"])
    if op == "norm":
        # the rounding to 8 or 4 bits needs the value next to a border: 64 bits
        h, d, rstd, w = _plain_norm(s["x"], s["residual"], s["weight"], torch.float64)
        return {"h": h, "values": _plain_values(d * rstd * w, c["mx"])}
    if op == "norm_train":
        h, d, rstd, w = _plain_norm(s["x"], s["residual"], s["weight"], torch.float32)
        unit = d * rstd
        dy = s["dy"].float()
        g = dy * w
        dx = rstd * (g - unit * (g * unit).mean(-1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"y": (unit * w).to(torch.bfloat16), "h": h, "dx": dx.to(torch.bfloat16), "dw": (dy * unit).sum(0)}
    x = _plain_matrix(s["x_codes"], s["x_scales"], c["K"], c["mx"])
    w = _plain_matrix(s["w_codes"], s["w_scales"], c["K"], "fp4")
    if op == "linear":
        return torch.matmul(x, w.t()).to(torch.bfloat16)
    offsets = s["offsets"].to(torch.int64)
    row = torch.arange(c["M"], device=x.device)
    expert = torch.searchsorted(offsets[1:], row, right=True)
    place = row - offsets[expert]
    padded = torch.zeros(c["E"], c["K"], s["most"], device=x.device)
    padded[expert, :, place] = x[: c["M"]]
    y = torch.bmm(w.view(c["E"], c["N"], c["K"]), padded)
    s["out"][: c["M"]] = y[expert, :, place].to(torch.bfloat16)
    return s["out"]


# --------------------------------------------------------------- the framework's

def _own_run(s):
    import bit_nf4_quantized_03_amd as qb
    c = s["case"]
    op = c["op"]
    types = {"fp4": qb.QLORA_MX_FP4, "fp8": qb.QLORA_MX_FP8}
    if op == "quantize":
        q = qb.qlora_mx_quantize(s["x"], types[c["mx"]])
        return qb.qlora_mx_dequantize(q, torch.bfloat16)
    if op == "norm":
        q, h = qb.qlora_rmsnorm_mx(s["x"], s["weight"], EPS, residual=s["residual"], mx=types[c["mx"]])
        return {"h": h, "values": qb.qlora_mx_dequantize(q, torch.bfloat16)}
    if op == "norm_train":
        y, h, rstd = qb.qlora_rmsnorm_fwd(s["x"], s["weight"], EPS, residual=s["residual"])
        dx, dw = qb.qlora_rmsnorm_bwd(s["dy"], h, s["weight"], rstd, dH=s["dh"])
        return {"y": y, "h": h, "dx": dx, "dw": dw}
    x = qb.MXMatrix(s["x_codes"].shape[0], c["K"], s["x_codes"], s["x_scales"], types[c["mx"]])
    w = qb.MXMatrix(s["w_codes"].shape[0], c["K"], s["w_codes"], s["w_scales"], qb.QLORA_MX_FP4)
    if op == "linear":
        return qb.qlora_mx_linear(x, w)
    return qb.qlora_mx_linear_grouped(x, w, s["offsets"], out=s["out"])


def run(state):
    if own:
        return _own_run(state)
    return _plain_run(state)


# ------------------------------------------------------------------------ inputs

def _normal(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda") * std


def _activations(g, rows, cols):
    """Normal values, one column in 64 ten times as large, as the streams of trained models have them."""
    loud = torch.where(torch.rand(cols, generator=g, device="cuda") < 1 / 64, 10.0, 1.0)
    return (_normal(g, (rows, cols)) * loud).to(torch.bfloat16)


def _packed(v, mx):
    """(codes, scales) of fp32 values in the layout above."""
    rows, cols = v.shape
    q, exponent = _plain_quantize(v, mx)
    scales = torch.zeros(rows, 16 * (-(-cols // 512)), dtype=torch.uint8, device=v.device)
    scales[:, : cols // 32] = (exponent.view(rows, -1) + 127).to(torch.uint8)
    q = q.reshape(rows, cols)
    if mx == "fp8":
        return q.to(torch.float8_e4m3fn).view(torch.uint8), scales
    index = torch.bucketize(q.abs(), torch.tensor(FP4, device=v.device)).to(torch.uint8) | (torch.signbit(q).to(torch.uint8) << 3)
    return index[:, 0::2] | (index[:, 1::2] << 4), scales


def _packed_rows(g, rows, cols, mx, std):
    """A microscaled matrix of normal values, made in strips of rows."""
    parts = [_packed(_normal(g, (min(8192, rows - r), cols), std), mx) for r in range(0, rows, 8192)]
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}
    if op == "quantize":
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        if case["mx"] == "fp8":
            s["x"] = _activations(g, case["rows"], case["cols"]).to(dtype)
        else:
            s["x"] = torch.empty(case["rows"], case["cols"], dtype=dtype, device="cuda")
            for r in range(0, case["rows"], 4096):
                part = s["x"][r: r + 4096]
                part.copy_(_normal(g, part.shape, 0.02))
        return s
    if op in ("norm", "norm_train"):
        shape = (case["rows"], case["cols"])
        s["x"] = _activations(g, *shape)
        s["residual"] = (4.0 * _activations(g, *shape).float()).to(torch.bfloat16) if case["residual"] else None
        s["weight"] = (1.0 + _normal(g, (case["cols"],), 0.1)).to(torch.bfloat16 if case["weight"] == "bf16" else torch.float32)
        if op == "norm_train":
            s["dy"] = _normal(g, shape, 0.01).to(torch.bfloat16)
            s["dh"] = _normal(g, shape, 0.01).to(torch.bfloat16) if case["residual"] else None
        return s
    rows = case["M"] + case.get("spare", 0)
    x = _activations(g, rows, case["K"]).float()
    s["x_codes"], s["x_scales"] = _packed(x, case["mx"])
    s["w_codes"], s["w_scales"] = _packed_rows(g, case["N"] * case.get("E", 1), case["K"], "fp4", 0.02)
    if op == "grouped":
        # each row picks an expert, the popular ones more often; rows are sorted by expert
        share = torch.exp(case["skew"] * _normal(g, (case["E"],)))
        pick = torch.multinomial(share, case["M"], replacement=True, generator=g)
        counts = torch.bincount(pick, minlength=case["E"])
        s["offsets"] = torch.zeros(case["E"] + 1, dtype=torch.int32, device="cuda")
        s["offsets"][1:] = torch.cumsum(counts, 0)
        s["most"] = int(counts.max())
        s["out"] = torch.zeros(rows, case["N"], dtype=torch.bfloat16, device="cuda")
    return s


# -------------------------------------------------------------------------- work

def _mx_bytes(rows, cols, mx):
    return rows * cols * (1.0 if mx == "fp8" else 0.5) + rows * cols / 32


def work(case):
    op = case["op"]
    if op in ("quantize", "norm", "norm_train"):
        n = case["rows"] * case["cols"]
    if op == "quantize":
        size = 2 if case["dtype"] == "bf16" else 4
        # read, written in few bits, and written again as the values of those
        return {"bytes": n * (size + 2) + _mx_bytes(case["rows"], case["cols"], case["mx"]), "flops": 4 * n}
    if op == "norm":
        moved = (6 if case["residual"] else 2) * n
        return {"bytes": moved + 2 * n + _mx_bytes(case["rows"], case["cols"], case["mx"]), "flops": 8 * n}
    if op == "norm_train":
        # x, residual, dy, dh in; y, h, dx out (h is read by the backward too, but the forward made it)
        return {"bytes": (14 if case["residual"] else 8) * n + 8 * case["cols"], "flops": 16 * n}
    M, N, K, E = case["M"], case["N"], case["K"], case.get("E", 1)
    weights = _mx_bytes(N * min(E, M), K, "fp4")
    return {"bytes": _mx_bytes(M, K, case["mx"]) + weights + 2 * M * N, "flops": 2 * M * N * K}


# ----------------------------------------------------- the definition in 64 bits

def _exact_nearest(v, mx):
    """The element nearest to each |v| (ties to the even code), with v's sign."""
    mantissa, top, low, most = TYPES[mx]
    values = [m * 2.0 ** (low - mantissa) for m in range(1 << mantissa)]
    values += [(1 + m / (1 << mantissa)) * 2.0 ** e for e in range(low, top + 1) for m in range(1 << mantissa)]
    values = [x for x in values if x <= most]
    table = torch.tensor(values, dtype=torch.float64, device=v.device)
    middle = (table[1:] + table[:-1]) / 2
    below, above = torch.bucketize(v.abs(), middle), torch.bucketize(v.abs(), middle, right=True)
    code = torch.where(below % 2 == 0, below, above)
    return table[code] * torch.sign(v)


def _exact_values(v, mx):
    """The microscaled values of v [rows, cols] in 64 bits."""
    out = torch.empty_like(v)
    for r in range(0, v.shape[0], 2048):
        b = v[r: r + 2048].reshape(-1, 32)
        amax = b.abs().amax(-1, keepdim=True)
        k = torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0)))
        k = k + (torch.exp2(k + 1) <= amax) - ((torch.exp2(k) > amax) & (amax > 0)).to(k.dtype)
        scale = torch.exp2(torch.clamp(k - TYPES[mx][1], -127, 127))
        out[r: r + 2048] = (_exact_nearest(b / scale, mx) * scale).reshape(-1, v.shape[1])
    return out


def _exact_matrix(codes, scales, cols, mx):
    c = codes.to(torch.int64)
    if mx == "fp4":
        c = torch.stack([c % 16, c // 16], -1).reshape(codes.shape[0], cols)
        sign, e, m = c // 8, (c // 2) % 4, (c % 2).double()
        v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2((e - 1).double()))
    else:
        sign, e, m = c // 128, (c // 8) % 16, (c % 8).double()
        v = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2((e - 7).double()))
    block = torch.exp2(scales[:, : cols // 32].double() - 127)
    return v * (1 - 2 * sign) * block.repeat_interleave(32, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_values(s["x"].double(), case["mx"])
    if op in ("norm", "norm_train"):
        total = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
        h, w = total.to(torch.bfloat16).double(), s["weight"].double()
        root = torch.sqrt(torch.sum(h * h, 1, keepdim=True) / case["cols"] + EPS)
        y = h / root * w
        if op == "norm":
            return {"h": total, "values": _exact_values(y, case["mx"])}
        dy = s["dy"].double()
        along = torch.sum(dy * w * h, 1, keepdim=True) / case["cols"]
        dx = dy * w / root - h * along / root ** 3
        if s["dh"] is not None:
            dx = dx + s["dh"].double()
        return {"y": y, "h": total, "dx": dx, "dw": torch.sum(dy * h / root, 0)}
    x = _exact_matrix(s["x_codes"], s["x_scales"], case["K"], case["mx"])
    if op == "linear":
        parts = [_exact_matrix(s["w_codes"][r: r + 4096], s["w_scales"][r: r + 4096], case["K"], "fp4") for r in range(0, case["N"], 4096)]
        return torch.cat([x @ p.t() for p in parts], 1)
    y = torch.zeros(x.shape[0], case["N"], dtype=torch.float64, device=x.device)
    at = s["offsets"].tolist()
    for e in range(case["E"]):
        rows = slice(e * case["N"], (e + 1) * case["N"])
        y[at[e]: at[e + 1]] = x[at[e]: at[e + 1]] @ _exact_matrix(s["w_codes"][rows], s["w_scales"][rows], case["K"], "fp4").t()
    return y
