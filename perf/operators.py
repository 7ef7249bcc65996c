"""Measured cases of the microscaled 4-bit operators.

``run`` computes one pass of an operator: in its plain form (elementary torch operations in
float32, rounded once at the end), or, when ``own`` is true, through the framework's calls.

  quantize  x [rows, cols] -> FP4 codes and block scales -> the values they stand for
  linear    y = X W^T of two FP4 matrices (G groups: X's column group g times W's row group g)
  proj      the grouped output projection on FP4 weights: o (bf16) encoded, each head group times
            its own matrix, z rounded to bf16 and encoded, then one dense product

Formats.  "mxfp4": E2M1 codes, one power-of-two scale per 32 elements.  "nvfp4": E2M1 codes, one
E4M3 scale per 16 elements and one float32 scale per tensor.  Codes are packed two to a byte (the
even element in the low nibble).  The scales are laid out in blocks of 128 rows x 4 scales
(512 bytes): the scale (r, b) of a block is byte (r % 32) * 16 + (r // 32) * 4 + b.

NVFP4's encoding is defined on float32 quotients, so that it is a function of the input's bits:
s = e4m3(fl(amax / fl(6 g))), T = fl(s g), code = e2m1(fl(x / T)).  With a tensor scale taken from
the data, many exact quotients lie within 2^-24 of a rounding border, so the definition has to say
on which side of it they count.
"""
import math

import torch

own = False

_MX, _NV = "mxfp4", "nvfp4"
_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_BLOCK = {_MX: 32, _NV: 16}


def _q(name, rows, cols, fmt, dtype):
    return {"name": name, "kind": "quantize", "rows": rows, "cols": cols, "fmt": fmt, "dtype": dtype}


def _l(name, M, N, K, G, fmt, out):
    return {"name": name, "kind": "linear", "M": M, "N": N, "K": K, "G": G, "fmt": fmt, "out": out}


def _p(name, T, G, K, R, d_model, fmt):
    return {"name": name, "kind": "proj", "T": T, "G": G, "K": K, "R": R, "d_model": d_model, "fmt": fmt}


def listed():
    return [
        # one decode token's 64 x 512 head outputs, encoded for the projection
        _q("quantize_nv_1", 1, 32768, _NV, "bf16"),
        # ragged rows and columns in float32 (a weight slice before its layout)
        _q("quantize_mx_777_f32", 777, 4128, _MX, "f32"),
        # the projected groups of an 8K prefill
        _q("quantize_mx_8k", 8192, 8192, _MX, "bf16"),
        # the smallest product: one token, a small layer
        _l("linear_mx_1_small", 1, 512, 512, 1, _MX, "bf16"),
        # one token, and a decode batch, through the hidden-size projection
        _l("linear_nv_1", 1, 4096, 8192, 1, _NV, "bf16"),
        _l("linear_mx_32", 32, 4096, 8192, 1, _MX, "bf16"),
        # odd sizes: a ragged chunk, float32 results, columns that fill no whole block of scales
        _l("linear_nv_333_odd", 333, 1001, 2080, 1, _NV, "f32"),
        # the head groups of a 2K chunk, each times its own matrix
        _l("linear_nv_2k_grouped", 2048, 1024, 4096, 8, _NV, "bf16"),
        # the hidden-size projection of an 8K prefill
        _l("linear_mx_8k", 8192, 4096, 8192, 1, _MX, "bf16"),
        # the whole projection: a decode batch, a ragged chunk of the small shape, an 8K prefill
        _p("proj_mx_32", 32, 8, 4096, 1024, 4096, _MX),
        _p("proj_nv_600_small", 600, 4, 512, 256, 512, _NV),
        _p("proj_mx_8k", 8192, 8, 4096, 1024, 4096, _MX),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    fmt = rng.choice((_MX, _NV))
    kind = rng.choice(("quantize", "linear", "linear", "proj"))
    if kind == "quantize":
        cols = 32 * _log(rng, 1, 1024)
        rows = max(1, min(_log(rng, 1, 16384), 8192 * 8192 // cols))
        return {"kind": kind, "rows": rows, "cols": cols, "fmt": fmt, "dtype": rng.choice(("bf16", "f32"))}
    if kind == "linear":
        G = rng.choice((1, 1, 2, 4))
        N = _log(rng, 8, 8192) if G == 1 else 128 * _log(rng, 1, 8)
        K = 32 * _log(rng, 2, 512) if G == 1 else 128 * _log(rng, 1, 32)
        M = max(1, min(_log(rng, 1, 8192), 8192 * 4096 * 8192 // (G * N * K)))
        return {"kind": kind, "M": M, "N": N, "K": K, "G": G, "fmt": fmt, "out": rng.choice(("bf16", "bf16", "f32"))}
    return {"kind": kind, "T": _log(rng, 1, 8192), "G": rng.choice((1, 2, 4, 8)), "K": 128 * _log(rng, 2, 32),
            "R": 128 * _log(rng, 1, 8), "d_model": _log(rng, 64, 4096), "fmt": fmt}


# ------------------------------------------------------------------ inputs
def _e2m1(y):
    """Codes of y: nearest of the grid, ties to the even code; the sign in bit 3 (y within +-6 or beyond: saturated)."""
    a = y.abs()
    c = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    return (c + 8 * torch.signbit(y)).to(torch.uint8)


def _encode(x, fmt, g):
    """float32 x [rows, cols] -> (codes [rows, cols], scale bytes [rows, cols / block])."""
    rows, cols = x.shape
    b = x.reshape(rows, cols // _BLOCK[fmt], _BLOCK[fmt])
    amax = b.abs().amax(-1)
    if fmt == _MX:
        frac, ex = torch.frexp(amax)  # amax = frac 2^ex, frac in [0.5, 1): least E with amax <= 0.75 2^(E + 3)
        E = torch.where(amax > 0, ex - 3 + (frac > 0.75), -127).clamp(-127, 127)
        codes = _e2m1(torch.ldexp(b, -E.unsqueeze(-1)))
        return codes.reshape(rows, cols), (E + 127).to(torch.uint8)
    s = (amax / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    T = (s.to(torch.float32) * g).unsqueeze(-1)
    y = torch.where(T > 0, b / T, torch.zeros_like(b))
    return _e2m1(y).reshape(rows, cols), s.view(torch.uint8)


def _decode(codes, scales, fmt, g):
    """The float32 values of codes [rows, cols] under scale bytes [rows, cols / block]."""
    grid = torch.tensor(_GRID + tuple(-v for v in _GRID), dtype=torch.float32, device=codes.device)
    v = grid[codes.to(torch.int32)].reshape(codes.shape[0], -1, _BLOCK[fmt])
    if fmt == _MX:
        return torch.ldexp(v, (scales.to(torch.int32) - 127).unsqueeze(-1)).reshape(codes.shape)
    return (v * (scales.view(torch.float8_e4m3fn).to(torch.float32) * g).unsqueeze(-1)).reshape(codes.shape)


def _pack(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def _unpack(packed):
    return torch.stack((packed & 15, packed >> 4), -1).reshape(packed.shape[0], -1)


def _blocked(scales):
    """Row-major scale bytes [rows, nb] in blocks of 128 rows x 4 scales, zero-padded."""
    rows, nb = scales.shape
    R, C = -(-rows // 128), -(-nb // 4)
    p = torch.zeros((R * 128, C * 4), dtype=torch.uint8, device=scales.device)
    p[:rows, :nb] = scales
    return p.reshape(R, 4, 32, C, 4).permute(0, 3, 2, 1, 4).contiguous().reshape(-1)


def _matrix(gen, rows, cols, fmt, std):
    """An FP4 matrix as a program keeps it: packed codes, scales (row-major and laid out), tensor scale."""
    x = torch.randn((rows, cols), generator=gen, device="cuda") * std
    g = (x.abs().amax() / (6.0 * 448.0)).reshape(1) if fmt == _NV else None
    codes, scales = _encode(x, fmt, g)
    return {"packed": _pack(codes), "scales": scales, "blocked": _blocked(scales), "g": g, "rows": rows, "cols": cols}


def _activations(gen, rows, cols):
    """Normal activations with a few channels that are larger, as head outputs and hidden states have."""
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    return x * torch.exp2(torch.randint(-2, 3, (1, cols), generator=gen, device="cuda").to(torch.float32))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    fmt, s = case["fmt"], dict(case)
    if case["kind"] == "quantize":
        x = _activations(gen, case["rows"], case["cols"])
        s["x"] = x.to(torch.bfloat16) if case["dtype"] == "bf16" else x
        # the tensor scale is calibrated before: the largest value maps to the largest code and scale
        s["g"] = (s["x"].float().abs().amax() / (6.0 * 448.0)).reshape(1) if fmt == _NV else None
    elif case["kind"] == "linear":
        G, K = case["G"], case["K"]
        s["x"] = _matrix(gen, case["M"], G * K, fmt, 1.0)
        s["w"] = _matrix(gen, G * case["N"], K, fmt, K ** -0.5)
    else:
        G, K, R = case["G"], case["K"], case["R"]
        s["o"] = _activations(gen, case["T"], G * K).to(torch.bfloat16)
        s["a"] = _matrix(gen, G * R, K, fmt, K ** -0.5)
        s["b"] = _matrix(gen, case["d_model"], G * R, fmt, (G * R) ** -0.5)
        # calibrated: z is a sum of unit-scale products, at most about 6 standard deviations from 0
        s["og"] = (s["o"].float().abs().amax() / (6.0 * 448.0)).reshape(1) if fmt == _NV else None
        s["zg"] = torch.full((1,), 16.0 / (6.0 * 448.0), device="cuda") if fmt == _NV else None
    return s


# ------------------------------------------------------------------ one pass
def _values(m, fmt):
    return _decode(_unpack(m["packed"]), m["scales"], fmt, m["g"])


def _group_product(x, w, G):
    """x [M, G K], w [G N, K] -> [M, G N]"""
    M, K = x.shape[0], w.shape[1]
    y = torch.matmul(x.reshape(M, G, K).transpose(0, 1), w.reshape(G, -1, K).transpose(1, 2))
    return y.transpose(0, 1).reshape(M, -1)


def run(s):
    fmt = s["fmt"]
    if own:
        from compressed_sparse_long_02_b200 import binding as B

        def mat(m):
            return B.Fp4Matrix(fmt, m["rows"], m["cols"], m["packed"], m["blocked"], m["g"])

        if s["kind"] == "quantize":
            q = B.csa_fp4_quantize(s["x"], fmt=fmt, tensor_scale=s["g"])
            return B.csa_fp4_dequantize(q)
        if s["kind"] == "linear":
            return B.csa_fp4_linear(mat(s["x"]), mat(s["w"]), groups=s["G"],
                                    out_dtype=torch.float32 if s["out"] == "f32" else torch.bfloat16)
        o = s["o"].view(s["T"], s["G"], s["K"])
        return B.csa_grouped_out_proj_fp4(o, mat(s["a"]), mat(s["b"]), groups=s["G"], o_scale=s["og"], z_scale=s["zg"])
    if s["kind"] == "quantize":
        codes, scales = _encode(s["x"].float(), fmt, s["g"])
        return _decode(codes, scales, fmt, s["g"]).to(torch.bfloat16)
    if s["kind"] == "linear":
        y = _group_product(_values(s["x"], fmt), _values(s["w"], fmt), s["G"])
        return y if s["out"] == "f32" else y.to(torch.bfloat16)
    o = _decode(*_encode(s["o"].float(), fmt, s["og"]), fmt, s["og"])
    z = _group_product(o, _values(s["a"], fmt), s["G"]).to(torch.bfloat16).float()
    z = _decode(*_encode(z, fmt, s["zg"]), fmt, s["zg"])
    return torch.matmul(z, _values(s["b"], fmt).t()).to(torch.bfloat16)


# ------------------------------------------------------------------ what a pass cannot do without
def _fp4_bytes(rows, cols, fmt):
    return rows * cols * (0.5 + 1.0 / _BLOCK[fmt])


def work(case):
    fmt = case["fmt"]
    if case["kind"] == "quantize":  # x read, the codes and scales written, their values written
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + _fp4_bytes(case["rows"], case["cols"], fmt) + 2 * n,
                "flops": 4 * n}
    if case["kind"] == "linear":
        M, N, K, G = case["M"], case["N"], case["K"], case["G"]
        return {"bytes": _fp4_bytes(M, G * K, fmt) + _fp4_bytes(G * N, K, fmt) + M * G * N * (4 if case["out"] == "f32" else 2),
                "flops": 2 * M * N * K * G}
    T, G, K, R, d = case["T"], case["G"], case["K"], case["R"], case["d_model"]
    return {"bytes": 2 * T * G * K + _fp4_bytes(G * R, K, fmt) + _fp4_bytes(d, G * R, fmt) + 2 * T * d,
            "flops": 2 * T * G * R * (K + d)}


# ------------------------------------------------------------------ the definition in 64 bits
def _near(y, bits, emin, top):
    """float64 y rounded to `bits` significant bits (least exponent emin), half to even, at most `top`."""
    a = y.abs()
    ex = torch.frexp(a)[1].to(torch.float64) - 1
    step = torch.exp2(torch.clamp(ex, min=emin) - (bits - 1))
    return torch.sign(y) * torch.clamp(torch.round(a / step) * step, max=top)


def _quantized64(x, fmt, g):
    """The values, in 64 bits, that the format holds for x."""
    n = _BLOCK[fmt]
    b = x.double().unflatten(1, (-1, n))
    amax = b.abs().amax(-1, keepdim=True)
    if fmt == _MX:
        scale = torch.exp2(torch.clamp(torch.ceil(torch.log2(torch.clamp(amax, min=1e-300) / 6.0)), -127, 127))
        scale = torch.where(amax > 6.0 * scale, 2 * scale, scale)  # log2 next to a power of two
        scale = torch.where((amax <= 3.0 * scale) & (scale > 2.0 ** -127), scale / 2, scale)
    else:
        # the roundings to 24 bits are the format's own (see above); the value is s g in full
        s = _near(_near(amax / _near(6.0 * g.double(), 24, -126, math.inf), 24, -126, math.inf), 4, -6, 448.0)
        T = _near(s * g.double(), 24, -126, math.inf)
        y = _near(torch.where(T > 0, b / T, 0.0), 24, -126, math.inf)
        return (_near(y, 2, 0, 6.0) * s * g.double()).flatten(1)
    v = _near(b / scale, 2, 0, 6.0) * scale
    return v.flatten(1)


def _held64(m, fmt):
    """The values, in 64 bits, of a packed matrix."""
    lut = [(c & 1) * 0.5 if c & 6 == 0 else (1 + 0.5 * (c & 1)) * 2.0 ** ((c >> 1 & 3) - 1) for c in range(8)]
    lut = torch.tensor(lut + [-v for v in lut], dtype=torch.float64, device=m["packed"].device)
    p = m["packed"].long()
    v = torch.empty((m["rows"], m["cols"]), dtype=torch.float64, device=p.device)
    v[:, 0::2], v[:, 1::2] = lut[p % 16], lut[p // 16]
    sb = m["scales"].double()
    if fmt == _MX:
        sc = torch.exp2(sb - 127)
    else:
        ex, frac = torch.div(sb, 8, rounding_mode="floor"), torch.remainder(sb, 8)
        sc = torch.where(ex > 0, (8 + frac) * torch.exp2(ex - 10), frac * 2.0 ** -9) * m["g"].double()
    return v * sc.repeat_interleave(_BLOCK[fmt], dim=1)


def _products64(x, w, G):
    return torch.cat([a @ b.t() for a, b in zip(x.chunk(G, 1), w.chunk(G, 0))], 1)


def exact(case, seed):
    s, fmt = prepare(case, seed), case["fmt"]
    if case["kind"] == "quantize":
        return _quantized64(s["x"], fmt, s["g"])
    if case["kind"] == "linear":
        return _products64(_held64(s["x"], fmt), _held64(s["w"], fmt), case["G"])
    z = _products64(_quantized64(s["o"], fmt, s["og"]), _held64(s["a"], fmt), case["G"])
    z = _quantized64(_near(z, 8, -126, math.inf), fmt, s["zg"])  # z is held in bf16 before it is encoded
    return z @ _held64(s["b"], fmt).t()
