"""What is measured of the 8-bit operators: block-scaled FP8 quantization and products, and the RMS norm that feeds them.

Formats: E4M3 or E5M2 codes with one power-of-two (E8M0) scale per block of 128 elements along a row, or per
128 x 128 tile of a weight matrix.  The scale is the least power of two under which the block's largest magnitude
fits the format, 1.75 * 2^8 (E4M3) or 1.75 * 2^15 (E5M2); bytes are exponent + 127.  Products read the scales in
the tensor-core layout: rows padded to 128 and blocks to 4 with zero bytes, 128 x 4 tiles, the tile along the
blocks fastest, (row % 32) * 16 + (row / 32) * 4 + block inside a tile.
"""
import math

import torch

own = False

BLOCK = 128
FLOAT8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 8, "e5m2": 15}        # largest value: 1.75 * 2^TOP
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the norm ahead of a decoder layer's linears, one token being generated
        {"name": "norm one token", "op": "norm", "rows": 1, "cols": 4096, "residual": True, "weight": "bf16", "fmt": "e4m3"},
        # the same in a training or prefill batch
        {"name": "norm 16384x4096", "op": "norm", "rows": 16384, "cols": 4096, "residual": True, "weight": "bf16", "fmt": "e4m3"},
        # its backward pass in that batch, with the gradient that the residual path brings
        {"name": "norm backward 16384x4096", "op": "norm_bwd", "rows": 16384, "cols": 4096, "residual": True, "weight": "bf16"},
        # the final norm of a small vision model's tokens: odd row count, no residual, weights kept in fp32
        {"name": "norm backward 1379x768", "op": "norm_bwd", "rows": 1379, "cols": 768, "residual": False, "weight": "f32"},
        # a short batch of activations ahead of a linear
        {"name": "quantize 197x768", "op": "quantize", "rows": 197, "cols": 768, "axis": 1, "fmt": "e4m3"},
        # gradients along the tokens, as the weight gradient's product reads them; ragged token count
        {"name": "quantize axis 0 16301x4096", "op": "quantize", "rows": 16301, "cols": 4096, "axis": 0, "fmt": "e5m2"},
        # a weight matrix after the optimizer's step, for the forward and the data gradient's products
        {"name": "quantize tiles 11008x4096", "op": "tiles", "rows": 11008, "cols": 4096, "fmt": "e4m3"},
        # one token through an attention projection
        {"name": "gemm 1x4096x4096", "op": "gemm", "m": 1, "n": 4096, "k": 4096, "a": "e4m3", "b": "e4m3", "out": "bf16", "tiles": True},
        # a decoding batch through an up projection
        {"name": "gemm 48x11008x4096", "op": "gemm", "m": 48, "n": 11008, "k": 4096, "a": "e4m3", "b": "e4m3", "out": "bf16", "tiles": True},
        # a ragged prefill chunk through a down projection
        {"name": "gemm 1000x4096x11008", "op": "gemm", "m": 1000, "n": 4096, "k": 11008, "a": "e4m3", "b": "e4m3", "out": "bf16", "tiles": True},
        # a training batch through an up projection
        {"name": "gemm 8192x11008x4096", "op": "gemm", "m": 8192, "n": 11008, "k": 4096, "a": "e4m3", "b": "e4m3", "out": "bf16", "tiles": True},
        # the weight gradient over a ragged number of tokens: E5M2 gradients, fp32 result
        {"name": "gemm wgrad 4096x4096x8201", "op": "gemm", "m": 4096, "n": 4096, "k": 8201, "a": "e5m2", "b": "e4m3", "out": "f32", "tiles": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "quantize", "tiles", "gemm", "gemm"])
    if op == "gemm":
        while True:
            m, n, k = _log(rng, 1, 8192), _log(rng, 64, 11008), _log(rng, 64, 11008)
            if m * n * k <= 8192 * 11008 * 4096:
                break
        wgrad = rng.random() < 0.3
        return {"op": op, "m": m, "n": n, "k": k, "a": "e5m2" if wgrad else "e4m3", "b": "e4m3",
                "out": "f32" if wgrad else "bf16", "tiles": not wgrad}
    if op == "tiles":
        return {"op": op, "rows": _log(rng, 64, 11008), "cols": 8 * _log(rng, 8, 512), "fmt": "e4m3"}
    cols = 8 * _log(rng, 16, 1376)
    rows = _log(rng, 1, min(16384, 16384 * 4096 // cols))
    if op == "quantize":
        return {"op": op, "rows": rows, "cols": cols, "axis": rng.choice([0, 1]), "fmt": rng.choice(["e4m3", "e5m2"])}
    case = {"op": op, "rows": rows, "cols": cols, "residual": rng.random() < 0.7, "weight": rng.choice(["bf16", "f32"])}
    if op == "norm":
        case["fmt"] = "e4m3"
    return case


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def work(case):
    op = case["op"]
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        out = 4 if case["out"] == "f32" else 2
        return {"bytes": m * k + n * k + (m + n) * _blocks(k) + out * m * n, "flops": 2 * m * n * k}
    rows, cols = case["rows"], case["cols"]
    el = rows * cols
    if op == "quantize":
        scales = rows * _blocks(cols) if case["axis"] == 1 else cols * _blocks(rows)
        return {"bytes": 3 * el + scales, "flops": 2 * el}
    if op == "tiles":
        return {"bytes": 4 * el + rows * _blocks(cols) + cols * _blocks(rows), "flops": 2 * el}
    w = cols * (2 if case["weight"] == "bf16" else 4)
    if op == "norm":
        return {"bytes": el * (2 + (4 if case["residual"] else 0) + 1) + rows * (_blocks(cols) + 4) + w, "flops": 7 * el}
    return {"bytes": el * (6 + (2 if case["residual"] else 0)) + rows * 4 + w + 4 * cols, "flops": 12 * el}


# ----------------------------------------------------------------- inputs
def _normal(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device="cuda") * std


def _pitch(n):
    return (n + 15) // 16 * 16


def _operand(gen, rows, k, fmt, std, tiles):
    """Codes [rows, k] with 16-byte rows and their scales in the tensor-core layout, as quantization leaves them."""
    x = _normal(gen, rows, k, std=std)
    codes = torch.zeros(rows, _pitch(k), dtype=torch.uint8, device="cuda")
    if tiles:
        byte = _tile_bytes(x, fmt)
    else:
        byte = _row_bytes(x, fmt)
    codes[:, :k] = _codes(x, byte, fmt).view(torch.uint8)
    return codes[:, :k], _mma(byte)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        # activations N(0, 1) (or gradients N(0, 1e-3)) against weights N(0, 0.02) (or, for the weight
        # gradient, against activations)
        s["ac"], s["as"] = _operand(gen, m, k, case["a"], 1e-3 if case["a"] == "e5m2" else 1.0, False)
        s["bc"], s["bs"] = _operand(gen, n, k, case["b"], 0.02 if case["tiles"] else 1.0, case["tiles"])
        s["y"] = torch.empty(m, n, dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16, device="cuda")
        return s
    rows, cols = case["rows"], case["cols"]
    bf = torch.bfloat16
    if op in ("quantize", "tiles"):
        std = 1e-3 if case["fmt"] == "e5m2" else 0.02 if op == "tiles" else 1.0
        s["x"] = _normal(gen, rows, cols, std=std).to(bf)
        return s
    # a residual stream with a few large channels, as decoders have
    channel = torch.where(torch.rand(cols, generator=gen, device="cuda") < 0.005, 20.0, 1.0)
    s["w"] = (1 + _normal(gen, cols, std=0.1)).to(bf if case["weight"] == "bf16" else torch.float32)
    x = (_normal(gen, rows, cols) * channel).to(bf)
    if op == "norm":
        s["x"] = x
        s["r"] = (_normal(gen, rows, cols, std=2.0) * channel).to(bf) if case["residual"] else None
        return s
    s["h"] = x
    s["rstd"] = (x.double().square().mean(1) + EPS).rsqrt().float()
    s["dy"] = _normal(gen, rows, cols, std=1e-3).to(bf)
    s["dr"] = _normal(gen, rows, cols, std=1e-3).to(bf) if case["residual"] else None
    return s


# ------------------------------------------------------------- plain form
def _exponent_byte(amax, fmt):
    bits = amax.float().contiguous().view(torch.int32)
    up = ((bits & 0x7FFFFF) > 0x600000).int()
    return ((bits >> 23) - TOP[fmt] + up).clamp_min(0)


def _row_bytes(x, fmt):
    """Scale bytes [rows, blocks] of 1 x 128 blocks."""
    rows, cols = x.shape
    pad = torch.zeros(rows, _blocks(cols) * BLOCK, dtype=torch.float32, device=x.device)
    pad[:, :cols] = x.float().abs()
    return _exponent_byte(pad.view(rows, -1, BLOCK).amax(2), fmt)


def _tile_bytes(x, fmt):
    """Scale bytes [rows, blocks] of 128 x 128 tiles, each repeated for the tile's rows."""
    rows, cols = x.shape
    pad = torch.zeros(_blocks(rows) * BLOCK, _blocks(cols) * BLOCK, dtype=torch.float32, device=x.device)
    pad[:rows, :cols] = x.float().abs()
    byte = _exponent_byte(pad.view(_blocks(rows), BLOCK, _blocks(cols), BLOCK).amax(3).amax(1), fmt)
    return byte.repeat_interleave(BLOCK, 0)[:rows]


def _codes(x, byte, fmt):
    inv = ((254 - byte) << 23).view(torch.float32)
    return (x.float() * inv.repeat_interleave(BLOCK, 1)[:, : x.shape[1]]).to(FLOAT8[fmt])


def _mma(byte):
    rows, g = byte.shape
    pad = torch.zeros((rows + 127) // 128 * 128, (g + 3) // 4 * 4, dtype=torch.uint8, device=byte.device)
    pad[:rows, :g] = byte.to(torch.uint8)
    return pad.view(-1, 4, 32, pad.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _scale_values(flat, rows, k):
    """Scales [rows, k] (fp32) out of the tensor-core layout."""
    g4 = (_blocks(k) + 3) // 4
    byte = flat.view(-1, g4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, 4 * g4)[:rows, : _blocks(k)]
    return byte.view(torch.float8_e8m0fnu).float().repeat_interleave(BLOCK, 1)[:, :k]


def _as_e8m0(u8):
    return u8.view(torch.float8_e8m0fnu)


def _plain(s):
    op = s["op"]
    if op == "gemm":
        a = s["ac"].view(FLOAT8[s["a"]]).float() * _scale_values(s["as"], s["m"], s["k"])
        b = s["bc"].view(FLOAT8[s["b"]]).float() * _scale_values(s["bs"], s["n"], s["k"])
        return {"y": (a @ b.t()).to(s["y"].dtype)}
    if op == "quantize":
        x = s["x"] if s["axis"] == 1 else s["x"].t()
        byte = _row_bytes(x, s["fmt"])
        return {"codes": _codes(x, byte, s["fmt"]), "scales": _as_e8m0(_mma(byte))}
    if op == "tiles":
        out = {}
        for key, x in (("", s["x"]), ("_t", s["x"].t())):
            byte = _tile_bytes(x, s["fmt"])
            out["codes" + key] = _codes(x, byte, s["fmt"])
            out["scales" + key] = _as_e8m0(_mma(byte))
        return out
    w = s["w"].float()
    if op == "norm":
        x = s["x"]
        if s["r"] is not None:
            x = (x.float() + s["r"].float()).to(torch.bfloat16)    # the residual stream is a bf16 tensor
        h = x.float()
        rstd = 1.0 / (h.square().mean(1) + EPS).sqrt()
        y = h * rstd[:, None] * w
        byte = _row_bytes(y, s["fmt"])
        out = {"codes": _codes(y, byte, s["fmt"]), "scales": _as_e8m0(_mma(byte)), "rstd": rstd}
        if s["r"] is not None:
            out["h"] = x
        return out
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = s["h"].float() * rstd
    g = dy * w
    dx = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["dr"] is not None:
        dx = dx + s["dr"].float()
    return {"dx": dx.to(torch.bfloat16), "dw": (dy * xh).sum(0)}


# ------------------------------------------------------- framework's calls
def _kernels(s):
    import microscaling_fp4_quantization_mxfp4_b200 as fp8
    op = s["op"]
    if op == "gemm":
        return {"y": fp8.fp4_fp8_gemm(s["ac"], s["as"], s["bc"], s["bs"], s["a"], s["b"], out=s["y"])}
    if op == "quantize":
        q = fp8.fp4_fp8_quantize(s["x"], s["fmt"], s["axis"], "mma")
        return {"codes": q.codes.view(FLOAT8[s["fmt"]]), "scales": _as_e8m0(q.scales)}
    if op == "tiles":
        q, t = fp8.fp4_fp8_quantize_2d(s["x"], s["fmt"], "mma")
        f8 = FLOAT8[s["fmt"]]
        return {"codes": q.codes.view(f8), "scales": _as_e8m0(q.scales), "codes_t": t.codes.view(f8), "scales_t": _as_e8m0(t.scales)}
    if op == "norm":
        q = fp8.fp4_rmsnorm_fp8_quantize(s["x"], s["w"], s["r"], EPS, s["fmt"], "mma")
        out = {"codes": q.codes.view(FLOAT8[s["fmt"]]), "scales": _as_e8m0(q.scales), "rstd": q.rstd}
        if s["r"] is not None:
            out["h"] = q.residual_out
        return out
    dx, dw = fp8.fp4_rmsnorm_backward(s["dy"], s["h"], s["w"], s["rstd"], s["dr"])
    return {"dx": dx, "dw": dw}


def run(state):
    return _kernels(state) if own else _plain(state)


# ------------------------------------------------------------ 64-bit values
def _exact_quantized(y, fmt, tile):
    """Values of the codes and the scales [rows, blocks] of y (fp64), from the definition of the formats."""
    rows, cols = y.shape
    mantissa, low = {"e4m3": (3, -6), "e5m2": (2, -14)}[fmt]
    most = 1.75 * 2.0 ** TOP[fmt]
    high = rows if not tile else _blocks(rows) * BLOCK
    pad = torch.zeros(high, _blocks(cols) * BLOCK, dtype=torch.float64, device=y.device)
    pad[:rows, :cols] = y.abs()
    if tile:
        amax = pad.view(_blocks(rows), BLOCK, _blocks(cols), BLOCK).amax((1, 3)).repeat_interleave(BLOCK, 0)[:rows]
    else:
        amax = pad.view(rows, -1, BLOCK).amax(2)
    frac, ex = torch.frexp(amax / most)                     # amax <= most * 2^e for the least such e
    e = torch.where(frac == 0.5, ex - 1, ex).clamp_min(-127)
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    v = y / torch.ldexp(torch.ones_like(amax), e).repeat_interleave(BLOCK, 1)[:, :cols]
    _, ev = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (ev - 1).clamp_min(low) - mantissa)
    return torch.round(v / step) * step, e


def _exact_mma(e):
    """2^e at the places of the tensor-core layout, 2^-127 (byte 0) in the padding."""
    rows, g = e.shape
    g4 = (g + 3) // 4 * 4
    out = torch.full(((rows + 127) // 128 * 128 * g4,), 2.0 ** -127, dtype=torch.float64, device=e.device)
    r = torch.arange(rows, device=e.device)[:, None]
    c = torch.arange(g, device=e.device)[None, :]
    out[((r // 128 * (g4 // 4) + c // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + c % 4).reshape(-1)] = \
        torch.ldexp(torch.ones_like(e, dtype=torch.float64), e).reshape(-1)
    return out


def _exact_operand(codes, flat, k, fmt):
    rows = codes.shape[0]
    g = _blocks(k)
    g4 = (g + 3) // 4
    r = torch.arange(rows, device=codes.device)[:, None]
    c = torch.arange(g, device=codes.device)[None, :]
    e = flat.long()[(r // 128 * g4 + c // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + c % 4] - 127
    v = codes.view(FLOAT8[fmt]).double()
    return v * torch.ldexp(torch.ones_like(e, dtype=torch.float64), e).repeat_interleave(BLOCK, 1)[:, :k]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        a = _exact_operand(s["ac"], s["as"], s["k"], s["a"])
        b = _exact_operand(s["bc"], s["bs"], s["k"], s["b"])
        return {"y": a @ b.t()}
    if op == "quantize":
        x = s["x"].double()
        v, e = _exact_quantized(x if s["axis"] == 1 else x.t(), s["fmt"], False)
        return {"codes": v, "scales": _exact_mma(e)}
    if op == "tiles":
        x = s["x"].double()
        v, e = _exact_quantized(x, s["fmt"], True)
        vt, et = _exact_quantized(x.t(), s["fmt"], True)
        return {"codes": v, "scales": _exact_mma(e), "codes_t": vt, "scales_t": _exact_mma(et)}
    w = s["w"].double()
    if op == "norm":
        h = s["x"].double()
        if s["r"] is not None:
            h = (h + s["r"].double()).to(torch.bfloat16).double()
        rstd = (h.square().sum(1) / case["cols"] + EPS) ** -0.5
        v, e = _exact_quantized(h * rstd[:, None] * w, s["fmt"], False)
        out = {"codes": v, "scales": _exact_mma(e), "rstd": rstd}
        if s["r"] is not None:
            out["h"] = h
        return out
    dy, h, rstd = s["dy"].double(), s["h"].double(), s["rstd"].double()[:, None]
    dw = (dy * h * rstd).sum(0)
    g = dy * w
    dx = rstd * g - rstd ** 3 * h * ((g * h).sum(1, keepdim=True) / case["cols"])
    if s["dr"] is not None:
        dx = dx + s["dr"].double()
    return {"dx": dx, "dw": dw}
