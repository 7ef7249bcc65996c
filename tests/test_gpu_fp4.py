"""Microscaled 4-bit matrices on the GPU against a plain 64-bit reference.

Encoding and the scale layout must match byte for byte; decoding is exact in float32 for
values with few bits and one rounding otherwise.  A product's terms are exact (4-bit codes,
scales of at most 4 significant bits), so the error left is float32 accumulation -- one
addition of a K = 64 step's sum per step, each within 2^-23 of the running sums, all bounded by
sum |x w| -- plus the rounding of the result (half a step: 2^-8 relative in bf16, 2^-24 in
float32) and three float32 products with the tensor scales.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests import fp4_reference as R
from tests.helpers import t2np

pytestmark = pytest.mark.gpu

FMTS = ["mxfp4", "nvfp4"]


@pytest.fixture(scope="module")
def B(cuda):
    from compressed_sparse_long_02_b200 import binding
    binding.lib()
    return binding


def tensor_scale(x, dev):
    return torch.tensor([np.abs(x[np.isfinite(x)]).max() / 2688.0], dtype=torch.float32, device=dev)


def make(B, dev, rng, rows, cols, fmt, std=1.0):
    """A matrix encoded by the reference, on the device, and its float64 values."""
    x = (rng.standard_normal((rows, cols)) * std * 2.0 ** rng.integers(-3, 4, (1, cols))).astype(np.float32)
    x[rng.random((rows, cols)) < 0.02] = 0.0
    g = np.float32(np.abs(x).max() / 2688.0) if fmt == "nvfp4" else None
    codes, sb = R.encode(x, fmt, g)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    m = B.Fp4Matrix(fmt, rows, cols, up(R.pack(codes)), up(R.block_scales(sb)),
                    None if g is None else torch.tensor([g], device=dev))
    return m, R.decode(codes, sb, fmt, g)


def product(x, w, G):
    """(sum x w, sum |x w|) in float64."""
    parts = [(a @ b.T, np.abs(a) @ np.abs(b).T) for a, b in zip(np.split(x, G, 1), np.split(w, G, 0))]
    return np.concatenate([p[0] for p in parts], 1), np.concatenate([p[1] for p in parts], 1)


def assert_product(y, ref, mag, K, dtype, what=""):
    steps = -(-K // 64) + 8  # the additions of the K steps, and of up to eight split partials
    tol = (steps * 2.0 ** -23 + 4 * 2.0 ** -24) * mag + torch.finfo(dtype).eps / 2 * np.abs(ref)
    y = y.double().cpu().numpy()
    assert np.isfinite(y).all(), what
    bad = np.abs(y - ref) > tol
    assert not bad.any(), f"{what}: {bad.sum()} off, worst {np.max(np.abs(y - ref) / np.maximum(tol, 1e-300)):.2f} x the bound"


QUANT_SHAPES = [(1, 32), (1, 32768), (5, 64), (31, 96), (128, 128), (129, 160), (300, 4128), (64, 256)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", QUANT_SHAPES)
def test_encode_matches_reference(B, cuda, fmt, dtype, rows, cols):
    rng = np.random.default_rng(rows * 7 + cols)
    x = torch.from_numpy((rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-9, 9, (rows, 1))).astype(np.float32))
    x[rows // 2, : cols // 2] = 0.0  # whole zero blocks
    x = x.to(dtype).to(cuda)
    xf = x.float().cpu().numpy()
    g = tensor_scale(xf, cuda) if fmt == "nvfp4" else None
    m = B.csa_fp4_quantize(x, fmt=fmt, tensor_scale=g)
    codes, sb = R.encode(xf, fmt, None if g is None else g.item())
    assert np.array_equal(t2np(m.scales), R.block_scales(sb))
    assert np.array_equal(R.unpack(t2np(m.packed)), codes)
    # decode: exact in float32 where the value has few bits, else one rounding of code * fl(s g)
    v32 = t2np(B.csa_fp4_dequantize(m, dtype=torch.float32)).astype(np.float64)
    ref = R.decode(codes, sb, fmt, None if g is None else g.item())
    assert (np.abs(v32 - ref) <= (0.0 if fmt == "mxfp4" else 2 * 2.0 ** -24) * np.abs(ref)).all()
    assert torch.equal(B.csa_fp4_dequantize(m), torch.from_numpy(v32).float().to(torch.bfloat16).to(cuda))
    assert B.csa_get_device_error() == 0


def test_encode_agrees_with_quantize_mxfp4_and_pack_scales(B, cuda):
    x = torch.randn((77, 416), device=cuda)
    packed, scales = B.csa_quantize_mxfp4(x)
    m = B.csa_fp4_quantize(x)
    assert torch.equal(m.packed, packed)
    assert torch.equal(m.scales, B.csa_fp4_pack_scales(scales, 416))
    assert np.array_equal(t2np(m.scales), R.block_scales(t2np(scales)))


@pytest.mark.parametrize("fmt", FMTS)
def test_encode_borders_and_special_values(B, cuda, fmt):
    """Every E2M1 rounding border and its float32 neighbours under exact scales, signed zeros,
    subnormals, NaN (left out of amax, +6) and infinities."""
    edges = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.0, 4.0], np.float32)
    vals = np.concatenate([edges, np.nextafter(edges, np.float32(9)), np.nextafter(edges, np.float32(-9))])
    vals = np.concatenate([vals, -vals])
    rows = []
    for k in range(0, len(vals), 15):  # each block of 16 holds a 6, so the scale is 2^0 (and s = 1 / g exactly)
        c = vals[k:k + 15]
        rows.append(np.concatenate([[6.0], c, np.zeros(15 - len(c))]))
    x = np.stack([np.concatenate([r, r]) for r in rows]).astype(np.float32)
    special = np.zeros((5, 32), np.float32)
    special[0, :4] = [np.nan, 1.0, -2.0, -np.nan]
    special[1, :3] = [np.inf, 1.0, -3.0]
    special[2, :3] = [-np.inf, np.inf, np.nan]
    special[3, :4] = [1e-40, -1e-42, 0.0, -0.0]
    special[4, :2] = [3.0e38, -3.4e38]
    x = np.concatenate([x, special])
    g = torch.tensor([2.0 ** -3], device=cuda) if fmt == "nvfp4" else None
    m = B.csa_fp4_quantize(torch.from_numpy(x).to(cuda), fmt=fmt, tensor_scale=g)
    codes, sb = R.encode(x, fmt, None if g is None else g.item())
    assert np.array_equal(t2np(m.scales), R.block_scales(sb))
    got = R.unpack(t2np(m.packed))
    assert np.array_equal(got, codes), np.argwhere(got != codes)[:8]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_nvfp4_quotients_next_to_every_border(B, cuda, dtype):
    """x = t T and its neighbours in x's type for every border t and block scales T of many significands,
    all ones and its neighbours among them: a code is e2m1(fl(x / T)), to the bit."""
    rng = np.random.default_rng(5)
    sig = np.concatenate([[2 ** 24 - 1, 2 ** 24 - 2, 2 ** 24 - 3, 2 ** 23, 2 ** 23 + 1, 2 ** 23 + 2, 11184810, 11184811,
                           5 * 2 ** 21 + 1, 7 * 2 ** 21 - 1, 2 ** 22 * 3 - 1, 2 ** 22 * 3 + 1],
                          rng.integers(2 ** 23, 2 ** 24, 40)]).astype(np.float64)
    step = 1 if dtype is torch.float32 else 2 ** 16  # between neighbours, in float32 bits
    for s, e in zip(sig, rng.integers(-40, 20, len(sig))):
        g = np.float32(s * 2.0 ** int(e))
        rows = []
        for sc in (1.0, 1.125, 13.0, 448.0):  # the block's E4M3 scale
            T = np.float32(sc) * g
            top = np.float32(6.0) * T
            t = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32) * T
            bits = t.view(np.int32) // step * step
            x = np.concatenate([(bits + step * d).view(np.float32) for d in (-2, -1, 0, 1, 2)])
            x = np.concatenate([x, -x, [0.0, -0.0]]).astype(np.float32)
            for k in range(0, len(x), 15):
                c = x[k:k + 15]
                topb = (top.view(np.int32) // step * step).view(np.float32)
                rows.append(np.concatenate([[topb], c, np.zeros(15 - len(c), np.float32)]))
        if len(rows) % 2:
            rows.append(rows[0])
        x = np.stack(rows).astype(np.float32).reshape(len(rows) // 2, 32)
        xt = torch.from_numpy(x).to(dtype)
        assert np.array_equal(xt.float().numpy(), x)
        m = B.csa_fp4_quantize(xt.to(cuda), fmt="nvfp4", tensor_scale=torch.tensor([float(g)], device=cuda))
        codes, sb = R.encode(x, "nvfp4", g)
        assert np.array_equal(t2np(m.scales), R.block_scales(sb)), g
        got = R.unpack(t2np(m.packed))
        assert np.array_equal(got, codes), (float(g), np.argwhere(got != codes)[:4])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("g", [2.0 ** -98, 2.0 ** -60, (2.0 - 2.0 ** -23) * 2.0 ** -10, 1e-3, 2.0 ** 95])
def test_nvfp4_extreme_scales_in_whole_row_blocks(B, cuda, dtype, g):
    """Blocks whose scale is cut at 448 or underflows to 0, zero blocks and ordinary ones side by side in
    whole and ragged row blocks, under tensor scales inside and outside the range of the common path."""
    rng = np.random.default_rng(9)
    rows, cols = 300, 1056
    x = rng.standard_normal((rows, cols // 16, 16)) * 400 * g
    x *= np.array([1.0, 2.0 ** 16, 2.0 ** -20, 0.0])[rng.choice(4, (rows, cols // 16), p=[0.7, 0.1, 0.1, 0.1])][..., None]
    xt = torch.from_numpy(x.reshape(rows, cols).astype(np.float32)).to(dtype)
    m = B.csa_fp4_quantize(xt.to(cuda), fmt="nvfp4", tensor_scale=torch.tensor([g], dtype=torch.float32, device=cuda))
    codes, sb = R.encode(xt.float().numpy(), "nvfp4", g)
    assert np.array_equal(t2np(m.scales), R.block_scales(sb))
    got = R.unpack(t2np(m.packed))
    assert np.array_equal(got, codes), np.argwhere(got != codes)[:4]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_encode_strided_rows_and_reused_buffers(B, cuda, dtype):
    big = torch.randn((3, 40, 200), device=cuda).to(dtype)
    x = big[:, 4:24, 8:136]  # inner rows 200 apart; the outer step is not 20 of them
    with pytest.raises(ValueError):
        B.csa_fp4_quantize(x)
    x = big[1, :, 8:136]
    want = B.csa_fp4_quantize(x.contiguous())
    got = B.csa_fp4_quantize(x, out=B.csa_fp4_quantize(torch.zeros((40, 128), device=cuda)))
    assert torch.equal(got.packed, want.packed) and torch.equal(got.scales, want.scales)
    out = torch.full((40, 160), 7.0, dtype=dtype, device=cuda)
    B.csa_fp4_dequantize(want, out=out[:, 16:144])
    assert torch.equal(out[:, 16:144], B.csa_fp4_dequantize(want, dtype=dtype))
    assert (out[:, :16] == 7).all() and (out[:, 144:] == 7).all()


LINEAR_SHAPES = [  # M, N, K, G: every tile width, ragged rows, features and K, one to many splits
    (1, 1, 32, 1), (1, 128, 256, 1), (1, 512, 512, 1), (3, 130, 96, 1), (2, 1024, 8192, 1), (32, 257, 1056, 1),
    (33, 300, 160, 1), (64, 384, 2080, 1), (65, 129, 4096, 1), (128, 128, 288, 1), (129, 96, 64, 1), (300, 1001, 2080, 1),
    (513, 640, 544, 1), (5, 128, 128, 3), (257, 384, 640, 2), (700, 256, 384, 4), (40, 256, 4096, 8), (2000, 512, 256, 1),
    # pairs of CTAs: ragged features (the second CTA's half empty or cut), tokens and K, groups of an odd half
    (1700, 1301, 288, 1), (2400, 1153, 96, 1), (1100, 384, 384, 8), (1030, 2560, 2080, 1), (300, 9000, 32, 1),
    # many tiles of 64 and of 128 tokens
    (1000, 1500, 160, 1), (19000, 128, 64, 1), (128, 19100, 64, 1)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K,G", LINEAR_SHAPES)
def test_linear_matches_reference(B, cuda, fmt, M, N, K, G):
    rng = np.random.default_rng(M * 1000003 + N * 101 + K)
    mx, x = make(B, cuda, rng, M, G * K, fmt)
    mw, w = make(B, cuda, rng, G * N, K, fmt, K ** -0.5)
    ref, mag = product(x, w, G)
    for dtype in (torch.bfloat16, torch.float32):
        y = B.csa_fp4_linear(mx, mw, groups=G, out_dtype=dtype)
        assert B.csa_get_device_error() == 0
        assert_product(y, ref, mag, K, dtype, f"{fmt} {M}x{N}x{K} G={G} {dtype}")
        assert torch.equal(y, B.csa_fp4_linear(mx, mw, groups=G, out_dtype=dtype)), "not reproducible"


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [3, 200])
def test_linear_into_a_wider_tensor(B, cuda, fmt, M):
    """Rows of y further apart than its columns: what lies between stays as it was."""
    rng = np.random.default_rng(M)
    mx, x = make(B, cuda, rng, M, 256, fmt)
    mw, w = make(B, cuda, rng, 136, 256, fmt, 0.1)
    wide = torch.full((M, 151), 3.0, dtype=torch.bfloat16, device=cuda)
    B.csa_fp4_linear(mx, mw, out=wide[:, :136])
    assert torch.equal(wide[:, :136], B.csa_fp4_linear(mx, mw)) and (wide[:, 136:] == 3).all()


PROJ_SHAPES = [(1, 16, 128, 4, 256, 512), (37, 16, 128, 4, 256, 512), (200, 8, 64, 2, 128, 130), (300, 4, 32, 1, 384, 77),
               (1500, 16, 64, 8, 128, 1300), (2100, 8, 64, 2, 640, 96)]  # the last two: pairs of CTAs encode z


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,H,D,G,Rk,d", PROJ_SHAPES)
def test_projection_is_its_four_steps(B, cuda, fmt, T, H, D, G, Rk, d):
    """The projection equals encode, grouped product, encode, product, bit for bit; each of those is
    held to the 64-bit reference above, and its product to the reference on the encoded z here."""
    rng = np.random.default_rng(T + H)
    o = torch.from_numpy(rng.standard_normal((T, H, D)).astype(np.float32)).to(cuda).to(torch.bfloat16)
    A, _ = make(B, cuda, rng, G * Rk, H // G * D, fmt, (H // G * D) ** -0.5)
    Bm, b64 = make(B, cuda, rng, d, G * Rk, fmt, (G * Rk) ** -0.5)
    og = torch.tensor([6.0 / 2688], device=cuda) if fmt == "nvfp4" else None
    zg = torch.tensor([40.0 / 2688], device=cuda) if fmt == "nvfp4" else None
    y = B.csa_grouped_out_proj_fp4(o, A, Bm, groups=G, o_scale=og, z_scale=zg)
    z = B.csa_fp4_linear(B.csa_fp4_quantize(o.reshape(T, -1), fmt=fmt, tensor_scale=og), A, groups=G)
    zq = B.csa_fp4_quantize(z, fmt=fmt, tensor_scale=zg)
    assert torch.equal(y, B.csa_fp4_linear(zq, Bm))
    codes, sb = R.encode(z.float().cpu().numpy(), fmt, None if zg is None else zg.item())
    ref, mag = product(R.decode(codes, sb, fmt, None if zg is None else zg.item()), b64, 1)
    assert_product(y, ref, mag, G * Rk, torch.bfloat16, "projection")
    assert B.csa_get_device_error() == 0


@pytest.mark.parametrize("T,H,D,G,Rk,d", [(37, 16, 128, 4, 256, 512), (2100, 8, 64, 2, 640, 96)])
@pytest.mark.parametrize("zg", [1e-6, 2.0 ** -98, (2.0 - 2.0 ** -23) * 2.0 ** -9, 2.0 ** 30])
def test_projection_with_extreme_intermediate_scales(B, cuda, zg, T, H, D, G, Rk, d):
    """z's scales cut at 448, out of the common path's range, all ones, or all zero: the projection still
    equals its four steps, bit for bit."""
    rng = np.random.default_rng(T)
    o = torch.from_numpy(rng.standard_normal((T, H, D)).astype(np.float32)).to(cuda).to(torch.bfloat16)
    A, _ = make(B, cuda, rng, G * Rk, H // G * D, "nvfp4", (H // G * D) ** -0.5)
    Bm, _ = make(B, cuda, rng, d, G * Rk, "nvfp4", (G * Rk) ** -0.5)
    og, zg = torch.tensor([6.0 / 2688], device=cuda), torch.tensor([zg], dtype=torch.float32, device=cuda)
    y = B.csa_grouped_out_proj_fp4(o, A, Bm, groups=G, o_scale=og, z_scale=zg)
    z = B.csa_fp4_linear(B.csa_fp4_quantize(o.reshape(T, -1), fmt="nvfp4", tensor_scale=og), A, groups=G)
    zq = B.csa_fp4_quantize(z, fmt="nvfp4", tensor_scale=zg)
    codes, sb = R.encode(z.float().cpu().numpy(), "nvfp4", zg.item())
    assert np.array_equal(t2np(zq.scales), R.block_scales(sb)) and np.array_equal(R.unpack(t2np(zq.packed)), codes)
    assert torch.equal(y, B.csa_fp4_linear(zq, Bm))


def test_projection_reuses_its_workspace_on_any_stream(B, cuda):
    """Two projections with workspaces of their own on two streams at once, each repeated in one
    workspace, give what each gives alone."""
    rng = np.random.default_rng(5)
    A, _ = make(B, cuda, rng, 512, 512, "mxfp4")
    Bm, _ = make(B, cuda, rng, 256, 512, "mxfp4")
    o = [torch.randn((T, 8, 128), device=cuda).to(torch.bfloat16) for T in (150, 9)]
    want = [B.csa_grouped_out_proj_fp4(v, A, Bm, groups=2) for v in o]
    ws = [torch.empty(B.csa_grouped_out_proj_fp4_workspace("mxfp4", v.shape[0], 8, 128, 2, 256), dtype=torch.uint8, device=cuda)
          for v in o]
    streams = [torch.cuda.Stream() for _ in o]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(B.csa_grouped_out_proj_fp4(o[i], A, Bm, groups=2, workspace=ws[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(g, want[i]) for g in got[i])
    with pytest.raises(B.CsaError) as ex:
        B.csa_grouped_out_proj_fp4(o[0], A, Bm, groups=2, workspace=ws[1])
    assert ex.value.status == 4


@pytest.mark.parametrize("fmt", FMTS)
def test_captured_and_replayed(B, cuda, fmt):
    """Encoding, both products and the projection in one CUDA graph, replayed on new inputs."""
    rng = np.random.default_rng(6)
    A, _ = make(B, cuda, rng, 256, 256, fmt)
    Bm, _ = make(B, cuda, rng, 96, 256, fmt)
    g = torch.tensor([8.0 / 2688], device=cuda) if fmt == "nvfp4" else None
    zg = torch.tensor([300.0 / 2688], device=cuda) if fmt == "nvfp4" else None
    o = torch.zeros((3, 4, 128), dtype=torch.bfloat16, device=cuda)

    def step():
        q = B.csa_fp4_quantize(o.reshape(3, 512), fmt=fmt, tensor_scale=g)
        return (B.csa_fp4_dequantize(q), B.csa_fp4_linear(q, A, groups=2),
                B.csa_grouped_out_proj_fp4(o, A, Bm, groups=2, o_scale=g, z_scale=zg))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(3):
        o.copy_(torch.randn(o.shape, device=cuda) * 2)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, step()):
            assert torch.equal(a, b)
    assert B.csa_get_device_error() == 0


def test_offsets_past_32_bits(B, cuda):
    """More than 2^32 elements: the last rows of a tall matrix are encoded, decoded and multiplied as
    the same rows alone are."""
    rows, cols = 140000, 32768
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device=cuda)
    x[-130:] = torch.randn((130, cols), device=cuda)
    m = B.csa_fp4_quantize(x)
    tail = B.csa_fp4_quantize(x[-96:])  # rows - 96 is a whole number of row blocks
    assert (rows - 96) % 128 == 0
    assert torch.equal(m.packed[-96:], tail.packed)
    assert torch.equal(m.scales[-tail.scales.numel():], tail.scales)
    del x
    v = B.csa_fp4_dequantize(m)
    assert torch.equal(v[-96:], B.csa_fp4_dequantize(tail)) and not v[:1000].any()
    del v
    w = B.csa_fp4_quantize(torch.randn((160, cols), device=cuda))
    y = B.csa_fp4_linear(m, w)
    assert not y[: rows - 130].any()
    # the same rows alone take another tile width and split: float32 sums in another order
    a, b = y[-96:].double(), B.csa_fp4_linear(tail, w, out_dtype=torch.float32).double()
    mag = B.csa_fp4_dequantize(tail).abs().double() @ B.csa_fp4_dequantize(w).abs().double().t()
    assert ((a - b).abs() <= 2.0 ** -8 * b.abs() + 2 * (cols // 64 + 8) * 2.0 ** -23 * mag).all()
    assert B.csa_get_device_error() == 0


def test_empty_inputs(B, cuda):
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=cuda)
    m = B.csa_fp4_quantize(x)
    assert m.packed.shape == (0, 32) and m.scales.numel() == 0
    assert B.csa_fp4_dequantize(m).shape == (0, 64)
    w = B.csa_fp4_quantize(torch.ones((32, 64), device=cuda))
    assert B.csa_fp4_linear(m, w).shape == (0, 32)
    A = B.csa_fp4_quantize(torch.ones((128, 128), device=cuda))
    assert B.csa_grouped_out_proj_fp4(torch.empty((0, 2, 64), dtype=torch.bfloat16, device=cuda), A, A, groups=1).shape == (0, 128)


def test_nan_and_infinite_scales_reach_only_their_rows(B, cuda):
    """A NaN scale byte makes its row's products NaN and no other's; a zero row gives zeros."""
    x = torch.randn((70, 160), device=cuda)
    x[7] = 0.0
    m, w = B.csa_fp4_quantize(x), B.csa_fp4_quantize(torch.randn((150, 160), device=cuda))
    ref = B.csa_fp4_linear(m, w)
    sc = m.scales.clone()
    sc[(5 % 32) * 16 + 2] = 255  # row 5, scale 2
    y = B.csa_fp4_linear(B.Fp4Matrix("mxfp4", 70, 160, m.packed, sc), w)
    assert y[5].isnan().all() and not ref.isnan().any() and (y[7] == 0).all()
    keep = torch.arange(70, device=cuda) != 5
    assert torch.equal(y[keep], ref[keep])
    sc = w.scales.clone()
    sc[(3 % 32) * 16 + 1] = 255  # feature 3, scale 1
    y = B.csa_fp4_linear(m, B.Fp4Matrix("mxfp4", 150, 160, w.packed, sc))
    keep = torch.arange(150, device=cuda) != 3
    assert y[:, 3].isnan().all() and torch.equal(y[:, keep], ref[:, keep])


@pytest.mark.parametrize("fmt", FMTS)
def test_batch_invariant_rows(B, cuda, fmt):
    """With the switch on, a row's result is the same bits whatever the number of rows (every tile
    width, lone CTAs and pairs), in the product and in the projection."""
    rng = np.random.default_rng(8)
    M, N, K = 3000, 1536, 4128
    mx, _ = make(B, cuda, rng, M, K, fmt)
    mw, _ = make(B, cuda, rng, N, K, fmt, K ** -0.5)
    o = torch.randn((M, 8, 64), device=cuda).to(torch.bfloat16)
    A, _ = make(B, cuda, rng, 2 * 128, 256, fmt, 0.06)
    Bm, _ = make(B, cuda, rng, 300, 256, fmt, 0.06)
    g = torch.tensor([6.0 / 2688], device=cuda) if fmt == "nvfp4" else None
    first = lambda m: B.csa_fp4_quantize(B.csa_fp4_dequantize(mx, dtype=torch.float32)[:m], fmt=fmt, tensor_scale=mx.tensor_scale)  # noqa: E731
    try:
        B.csa_set_batch_invariant(True)
        whole = B.csa_fp4_linear(first(M), mw, out_dtype=torch.float32)
        proj = B.csa_grouped_out_proj_fp4(o, A, Bm, groups=2, o_scale=g, z_scale=g)
        for m in (1, 33, 100, 130, 700):
            assert torch.equal(B.csa_fp4_linear(first(m), mw, out_dtype=torch.float32), whole[:m]), m
            assert torch.equal(B.csa_grouped_out_proj_fp4(o[:m], A, Bm, groups=2, o_scale=g, z_scale=g), proj[:m]), m
    finally:
        B.csa_set_batch_invariant(False)
    assert B.csa_get_device_error() == 0


def test_first_call_inside_a_capture(cuda):
    """A process whose first call of the products is captured: the replay gives what an eager call does."""
    code = """
import torch
from compressed_sparse_long_02_b200 import binding as B
dev = torch.device("cuda:0")
x, o = torch.randn((40, 512), device=dev), torch.randn((700, 8, 64), device=dev).to(torch.bfloat16)
w = B.csa_fp4_quantize(torch.randn((1024, 512), device=dev))
A, Bm = B.csa_fp4_quantize(torch.randn((512, 256), device=dev)), B.csa_fp4_quantize(torch.randn((1000, 512), device=dev))
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y = B.csa_fp4_linear(B.csa_fp4_quantize(x), w)
    z = B.csa_grouped_out_proj_fp4(o, A, Bm, groups=2)
g.replay()
torch.cuda.synchronize()
assert torch.equal(y, B.csa_fp4_linear(B.csa_fp4_quantize(x), w))
assert torch.equal(z, B.csa_grouped_out_proj_fp4(o, A, Bm, groups=2))
assert B.csa_get_device_error() == 0
print("captured ok")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "captured ok" in r.stdout, r.stdout + r.stderr


def rescaled(m, v, g):
    """The same codes and block scales under the tensor scale g, and the float64 values."""
    g0 = float(m.tensor_scale.item())
    g = np.float32(g)
    return m._replace(tensor_scale=torch.full_like(m.tensor_scale, float(g))), v / g0 * float(g)


def small_sums(B, dev, rng, rows, cols):
    """Random codes under the smallest block scale, 2^-9: products of sums far below 1."""
    codes = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    sb = np.ones((rows, cols // 16), np.uint8)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    m = B.Fp4Matrix("nvfp4", rows, cols, up(R.pack(codes)), up(R.block_scales(sb)), torch.ones(1, device=dev))
    return m, R.decode(codes, sb, "nvfp4", 1.0)


@pytest.mark.parametrize("M,N,K", [(1, 130, 512), (3, 257, 4096), (40, 200, 2080), (300, 1001, 288), (1700, 1301, 288), (2000, 512, 256)])
@pytest.mark.parametrize("gx,gw,small", [(2.0 ** -80, 2.0 ** -75, False), (1e-22, 1e-22, False), (2.0 ** -98, 2.0 ** -40, False),
                                         (2.0 ** -149, 2.0 ** 60, False), (2.0 ** -149, 2.0 ** -149, False),
                                         (2.0 ** 95, 2.0 ** 37, True), (2.0 ** 70, 2.0 ** 60, True), (2.0 ** 127, 2.0 ** 127, True),
                                         (2.0 ** 127, 2.0 ** -149, False)])
def test_product_of_extreme_tensor_scales(B, cuda, M, N, K, gx, gw, small):
    """Tensor scales whose product leaves float32's normal range, or just about: results that float32 can hold
    are right, others are 0 or infinite, and rows of zeros give zeros.  The bound is assert_product's, and half a
    step of the subnormals (of float32, and of the type rounded to)."""
    rng = np.random.default_rng(M + N + K)
    build = (lambda r, std: small_sums(B, cuda, rng, r, K)) if small else (lambda r, std: make(B, cuda, rng, r, K, "nvfp4", std))
    (mx, x), (mw, w) = rescaled(*build(M, 1.0), gx), rescaled(*build(N, K ** -0.5), gw)
    mx.packed[M // 2] = 0
    mw.packed[N // 3] = 0
    x[M // 2], w[N // 3] = 0.0, 0.0
    ref, mag = product(x, w, 1)
    for dtype, sub in ((torch.float32, 2.0 ** -150), (torch.bfloat16, 2.0 ** -134)):
        y = B.csa_fp4_linear(mx, mw, out_dtype=dtype)
        assert B.csa_get_device_error() == 0
        y = y.double().cpu().numpy()
        assert not y[M // 2].any() and not y[:, N // 3].any()
        tol = ((-(-K // 64) + 8) * 2.0 ** -23 + 4 * 2.0 ** -24) * mag + torch.finfo(dtype).eps / 2 * np.abs(ref) + sub + 2.0 ** -150
        over = np.abs(ref) + tol > torch.finfo(dtype).max  # may be infinite
        must = np.abs(ref) - tol > 2.0 ** 128              # has to be
        with np.errstate(invalid="ignore"):
            near = np.abs(y - ref) <= tol
        assert np.where(must, np.isinf(y) & (np.sign(y) == np.sign(ref)), near | (over & np.isinf(y))).all()
        if M > 1 and max(gx, gw) < 2.0 ** 100 and min(gx, gw) > 2.0 ** -100:  # (of one row, it is the one of zeros)
            assert (near & (ref != 0)).any() and y.any()   # there are results to be right about


@pytest.mark.parametrize("T,H,D,G,Rk,d", [(37, 16, 128, 4, 256, 512), (2100, 8, 64, 2, 640, 96)])
def test_projection_between_extreme_scales(B, cuda, T, H, D, G, Rk, d):
    """o and A so small that o_scale times A's scale is no normal float32, z's tensor scale subnormal and Bm's
    large: y is right against the reference's encoding of z, and z against the reference's product."""
    rng = np.random.default_rng(T)
    o = torch.from_numpy((rng.standard_normal((T, H, D)) * 2.0 ** -70).astype(np.float32)).to(cuda).to(torch.bfloat16)
    A, a64 = rescaled(*make(B, cuda, rng, G * Rk, H // G * D, "nvfp4"), 2.0 ** -66)
    Bm, b64 = rescaled(*make(B, cuda, rng, d, G * Rk, "nvfp4"), 2.0 ** 50)
    one = lambda v: torch.tensor([v], dtype=torch.float32, device=cuda)  # noqa: E731
    og = one(2.0 ** -67 / 2688)
    oq = B.csa_fp4_quantize(o.reshape(T, -1), fmt="nvfp4", tensor_scale=og)
    codes, sb = R.encode(o.float().cpu().numpy().reshape(T, -1), "nvfp4", og.item())
    assert np.array_equal(R.unpack(t2np(oq.packed)), codes)
    o64 = R.decode(codes, sb, "nvfp4", og.item())
    z = B.csa_fp4_linear(oq, A, groups=G)
    zref, zmag = product(o64, a64, G)
    K = H // G * D
    tol = ((-(-K // 64) + 8) * 2.0 ** -23 + 4 * 2.0 ** -24) * zmag + 2.0 ** -8 * np.abs(zref) + 2.0 ** -134 + 2.0 ** -150
    zf = z.double().cpu().numpy()
    assert zf.any() and (np.abs(zf - zref) <= tol).all()
    zg = one(float(np.abs(zf).max() / 2688))
    assert 0 < zg.item() < 2.0 ** -126 and og.item() * 2.0 ** -66 < 2.0 ** -126
    y = B.csa_grouped_out_proj_fp4(o, A, Bm, groups=G, o_scale=og, z_scale=zg)
    codes, sb = R.encode(z.float().cpu().numpy(), "nvfp4", zg.item())
    ref, mag = product(R.decode(codes, sb, "nvfp4", zg.item()), b64, 1)
    assert np.abs(ref).max() > 2.0 ** -110
    assert_product(y, ref, mag, G * Rk, torch.bfloat16, "projection")
    assert B.csa_get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tensors_of_zeros(B, cuda, dtype):
    """A tensor of zeros under the tensor scale that its largest value gives, 0: bytes, values and products of
    zeros; a tensor scale of 0 makes zeros of any values."""
    for rows, cols in ((1, 32), (300, 1056)):
        x = torch.zeros((rows, cols), dtype=dtype, device=cuda)
        x[rows // 2] = -0.0
        g = (x.abs().amax() / 2688).float().reshape(1)
        m = B.csa_fp4_quantize(x, fmt="nvfp4", tensor_scale=g)
        assert g.item() == 0 and not m.packed.any() and not m.scales.any()
        assert not B.csa_fp4_dequantize(m, dtype=torch.float32).any()
        x = torch.randn((rows, cols), device=cuda).to(dtype)
        x[0, :3] = torch.tensor([float("nan"), float("inf"), -float("inf")])
        m0 = B.csa_fp4_quantize(x, fmt="nvfp4", tensor_scale=g)
        assert not m0.packed.any() and not B.csa_fp4_dequantize(m0, dtype=torch.float32).any()
        rng = np.random.default_rng(cols)
        w, _ = make(B, cuda, rng, 2000, cols, "nvfp4")  # lone tiles or pairs by the rows
        big, _ = make(B, cuda, rng, 2100, cols, "nvfp4")
        for out in (torch.float32, torch.bfloat16):
            for a, b in ((m, w), (m0, w), (big, m), (big, m0), (m, m0)):
                assert not B.csa_fp4_linear(a, b, out_dtype=out).any()


@pytest.mark.parametrize("T,H,D,G,Rk,d", [(1, 16, 128, 4, 256, 512), (37, 16, 128, 4, 256, 512), (2100, 8, 64, 2, 640, 96)])
def test_projection_of_zeros(B, cuda, T, H, D, G, Rk, d):
    """o of zeros under o_scale 0, and an intermediate of zeros under z_scale 0, give zeros."""
    rng = np.random.default_rng(T)
    A, _ = make(B, cuda, rng, G * Rk, H // G * D, "nvfp4")
    Bm, _ = make(B, cuda, rng, d, G * Rk, "nvfp4")
    zero, one = torch.zeros(1, device=cuda), torch.full((1,), 6.0 / 2688, device=cuda)
    o = torch.zeros((T, H, D), dtype=torch.bfloat16, device=cuda)
    for og, zg in ((zero, zero), (zero, one), (one, zero), (one, one)):
        y = B.csa_grouped_out_proj_fp4(o, A, Bm, groups=G, o_scale=og, z_scale=zg)
        assert not y.any(), (og.item(), zg.item())
    o = torch.randn((T, H, D), device=cuda).to(torch.bfloat16)
    assert not B.csa_grouped_out_proj_fp4(o, A, Bm, groups=G, o_scale=one, z_scale=zero).any()
    assert not B.csa_grouped_out_proj_fp4(o, A, Bm, groups=G, o_scale=zero, z_scale=one).any()
    assert B.csa_get_device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_calls_allocate_nothing(B, cuda, fmt):
    """With out, workspace and the library's first calls behind them, the calls take no device memory, torch's
    or their own."""
    rng = np.random.default_rng(12)
    A, _ = make(B, cuda, rng, 512, 256, fmt)
    Bm, _ = make(B, cuda, rng, 1000, 512, fmt)
    g = torch.tensor([6.0 / 2688], device=cuda) if fmt == "nvfp4" else None
    sets = []
    for T in (1, 40, 2000):
        o = torch.randn((T, 8, 64), device=cuda).to(torch.bfloat16)
        q = B.csa_fp4_quantize(o.reshape(T, 512), fmt=fmt, tensor_scale=g)
        ws = torch.empty(B.csa_grouped_out_proj_fp4_workspace(fmt, T, 8, 64, 2, 256), dtype=torch.uint8, device=cuda)
        new = lambda c, d=torch.bfloat16: torch.empty((T, c), dtype=d, device=cuda)  # noqa: E731,B023
        sets.append((o, q, ws, new(512), new(512), new(512, torch.float32), new(1000)))

    def run():
        for o, q, ws, v, z, zf, y in sets:
            B.csa_fp4_quantize(o.reshape(o.shape[0], 512), fmt=fmt, tensor_scale=g, out=q)
            B.csa_fp4_dequantize(q, out=v)
            B.csa_fp4_linear(q, A, groups=2, out=z)
            B.csa_fp4_linear(q, A, groups=2, out=zf)
            B.csa_grouped_out_proj_fp4(o, A, Bm, groups=2, o_scale=g, z_scale=g, out=y, workspace=ws)
        torch.cuda.synchronize()

    run()
    free, held = torch.cuda.mem_get_info(cuda)[0], torch.cuda.memory_stats(cuda)["allocation.all.allocated"]
    for _ in range(5):
        run()
    assert torch.cuda.memory_stats(cuda)["allocation.all.allocated"] == held
    assert torch.cuda.mem_get_info(cuda)[0] == free
