"""Microscaled 4-bit matrices without a GPU: the C calls refuse bad arguments before any device
work, the binding refuses what does not fit together, the sizes follow the layout, and the
tests' reference agrees with the oracle's MXFP4 encoder."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from tests import fp4_reference as R

INVALID, ALIGNMENT, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4
MX, NV, F32, BF16 = 0, 1, 0, 1


@pytest.fixture(scope="module")
def B():
    from compressed_sparse_long_02_b200 import build as bld
    bld.build()
    from compressed_sparse_long_02_b200 import binding
    binding.lib()
    return binding


def mat(B, packed=16, scales=16, g=None):
    return ctypes.byref(B._Fp4Mat(packed, scales, g))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_scale_bytes(B, fmt):
    for rows, cols in [(1, 32), (128, 128), (129, 160), (1000, 4128)]:
        nb = cols // R.BLOCK[fmt]
        assert B.csa_fp4_scale_bytes(fmt, rows, cols) == -(-rows // 128) * -(-nb // 4) * 512
        assert B.csa_fp4_scale_bytes(fmt, rows, cols) == R.block_scales(np.zeros((rows, nb), np.uint8)).size
    assert B.csa_fp4_scale_bytes(fmt, 0, 32) == 0
    L = B.lib()
    assert L.csa_fp4_scale_bytes(2, 4, 32) == 0 and L.csa_fp4_scale_bytes(MX, -1, 32) == 0
    # 128 x 2^24 rows of 2^10 columns: past 32 bits
    assert B.csa_fp4_scale_bytes("mxfp4", 1 << 31, 1024) == (1 << 24) * 8 * 512


def test_quantize_and_dequantize_refusals(B):
    L, P = B.lib(), ctypes.c_void_p

    def q(fmt=MX, x=P(16), dt=BF16, rows=4, cols=64, ld=64, out=None):
        return L.csa_fp4_quantize(fmt, x, dt, rows, cols, ld, mat(B) if out is None else out, None)

    def d(fmt=MX, m=None, rows=4, cols=64, dt=BF16, y=P(16), ld=64):
        return L.csa_fp4_dequantize(fmt, mat(B) if m is None else m, rows, cols, dt, y, ld, None)

    for f in (q, d):
        assert f(fmt=2) == INVALID and f(rows=-1) == INVALID and f(cols=0) == INVALID and f(cols=48) == INVALID
        assert f(ld=32) == INVALID and f(dt=2) == INVALID
        assert f(ld=68) == ALIGNMENT and f(ld=66, dt=F32) == ALIGNMENT
        assert f(rows=0) == 0 and f(cols=(1 << 30) + 32, ld=1 << 31) == UNSUPPORTED
    assert q(x=None) == INVALID and q(x=P(24)) == ALIGNMENT and d(y=None) == INVALID and d(y=P(24)) == ALIGNMENT
    for kw in ("out", "m"):
        f = q if kw == "out" else d
        assert f(**{kw: mat(B, packed=None)}) == INVALID and f(**{kw: mat(B, scales=None)}) == INVALID
        assert f(**{kw: mat(B, packed=24)}) == ALIGNMENT and f(**{kw: mat(B, scales=24)}) == ALIGNMENT
        assert f(**{kw: mat(B, g=16)}) == INVALID                 # MXFP4 has no tensor scale
        assert f(fmt=NV) == INVALID                               # NVFP4 needs one
        assert f(fmt=NV, **{kw: mat(B, g=18)}) == ALIGNMENT
    assert L.csa_fp4_quantize(MX, P(16), BF16, 4, 64, 64, None, None) == INVALID
    assert L.csa_fp4_pack_scales(MX, None, 4, 64, P(16), None) == INVALID
    assert L.csa_fp4_pack_scales(MX, P(3), 4, 64, P(17), None) == ALIGNMENT
    assert L.csa_fp4_pack_scales(MX, P(3), 4, 40, P(16), None) == INVALID
    assert L.csa_fp4_pack_scales(MX, None, 0, 64, None, None) == 0
    assert L.csa_fp4_pack_scales(MX, P(3), 4, (1 << 30) + 32, P(16), None) == UNSUPPORTED
    assert L.csa_fp4_scale_bytes(MX, 4, (1 << 30) + 32) == 0


def test_linear_refusals(B):
    L, P = B.lib(), ctypes.c_void_p

    def f(fmt=MX, M=4, N=256, K=256, G=1, x=None, w=None, dt=BF16, y=P(16), ldy=None):
        return L.csa_fp4_linear(fmt, M, N, K, G, x or mat(B), w or mat(B), dt, y, G * N if ldy is None else ldy, None)

    assert f(fmt=-1) == INVALID and f(M=-1) == INVALID and f(N=0) == INVALID and f(K=0) == INVALID and f(G=0) == INVALID
    assert f(dt=7) == INVALID and f(ldy=255) == INVALID and f(G=2, ldy=500) == INVALID
    assert f(K=48) == UNSUPPORTED
    assert f(G=2, K=160) == UNSUPPORTED and f(G=2, N=200) == UNSUPPORTED
    assert f(G=1 << 20, K=1 << 12) == UNSUPPORTED and f(G=1 << 20, N=1 << 12, K=128) == UNSUPPORTED
    assert f(M=0, y=None) == 0
    assert f(y=None) == INVALID and f(y=P(20)) == ALIGNMENT
    assert f(x=mat(B, packed=None)) == INVALID and f(w=mat(B, scales=None)) == INVALID
    assert f(x=mat(B, packed=24)) == ALIGNMENT and f(w=mat(B, scales=20)) == ALIGNMENT
    assert f(w=mat(B, g=16)) == INVALID and f(fmt=NV, x=mat(B, g=16)) == INVALID


def test_projection_refusals(B):
    L, P = B.lib(), ctypes.c_void_p

    def f(fmt=MX, T=4, H=16, D=128, G=4, R_=256, d=512, o=P(16), os_=None, A=None, zs=None, Bm=None, y=P(16), ws=P(16), n=1 << 40):
        return L.csa_grouped_out_proj_fp4(fmt, T, H, D, G, R_, d, o, os_, A or mat(B), zs, Bm or mat(B), y, ws, n, None)

    assert f(fmt=3) == INVALID and f(T=-1) == INVALID and f(G=3) == INVALID and f(d=0) == INVALID and f(R_=0) == INVALID
    assert f(H=4, D=96) == UNSUPPORTED and f(R_=192) == UNSUPPORTED
    assert f(T=0, o=None, y=None, ws=None) == 0
    assert f(o=None) == INVALID and f(y=None) == INVALID and f(ws=None) == INVALID
    assert f(o=P(24)) == ALIGNMENT and f(y=P(24)) == ALIGNMENT and f(ws=P(24)) == ALIGNMENT
    assert f(os_=P(16)) == INVALID and f(zs=P(16)) == INVALID
    assert f(fmt=NV, A=mat(B, g=16), Bm=mat(B, g=16)) == INVALID
    assert f(fmt=NV, A=mat(B, g=16), Bm=mat(B, g=16), os_=P(16)) == INVALID
    need = L.csa_grouped_out_proj_fp4_workspace(MX, 4, 16, 128, 4, 256)
    assert need > 0 and f(n=need - 1) == WORKSPACE
    assert L.csa_grouped_out_proj_fp4_workspace(MX, 4, 16, 128, 0, 256) == 0
    assert L.csa_grouped_out_proj_fp4_workspace(2, 4, 16, 128, 4, 256) == 0


def test_binding_refuses_what_does_not_fit(B):
    """Shapes, types and formats that do not belong together, before any pointer is passed on."""
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    m = B.Fp4Matrix("mxfp4", 4, 64, u8(4, 32), u8(512))
    with pytest.raises(ValueError):
        B.csa_fp4_quantize(torch.zeros((4, 64)), fmt="fp4")
    with pytest.raises(TypeError):
        B.csa_fp4_quantize(torch.zeros((4, 64), dtype=torch.float16))
    for x in (torch.zeros((4, 48)), torch.zeros((4, 128))[:, ::2], torch.zeros((4, 64, 2))[:, :, 0], torch.zeros((4, 0))):
        with pytest.raises(ValueError):
            B.csa_fp4_quantize(x)
    with pytest.raises(ValueError):  # a CPU tensor
        B.csa_fp4_quantize(torch.zeros((4, 64)))
    with pytest.raises(ValueError):  # out of another shape
        B.csa_fp4_quantize(torch.zeros((5, 64)), out=m)
    with pytest.raises(ValueError):
        B.csa_fp4_pack_scales(u8(4, 3), 64)
    with pytest.raises(TypeError):
        B.csa_fp4_pack_scales(torch.zeros((4, 2)), 64)
    nv = m._replace(fmt="nvfp4")
    for x, w, kw in ((m, nv, {}), (m, m._replace(cols=32), {}), (m, m, {"groups": 3}), (m, m, {"groups": 0}),
                     (m, m, {"out": torch.zeros((4, 5), dtype=torch.bfloat16)})):
        with pytest.raises(ValueError):
            B.csa_fp4_linear(x, w, **kw)
    with pytest.raises(TypeError):
        B.csa_fp4_linear(m, m, out_dtype=torch.float16)
    o = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    for kw in ({"groups": 3}, {"groups": 0}, {"groups": 2}):
        with pytest.raises(ValueError):
            B.csa_grouped_out_proj_fp4(o, m, m, **kw)
    with pytest.raises(TypeError):
        B.csa_grouped_out_proj_fp4(o.float(), m, m, groups=2)


def test_rows_of_a_view(B):
    z = torch.zeros((4, 6, 64))
    assert B._rows_2d(z, "x") == (24, 64, 64)
    assert B._rows_2d(z[:, ::2], "x") == (12, 64, 128)
    assert B._rows_2d(z[1, 1:3, 8:40], "x") == (2, 32, 64)
    assert B._rows_2d(z[:, 3, :32], "x") == (4, 32, 384)
    assert B._rows_2d(z[0, 0], "x") == (1, 64, 64)
    for bad in (z[:, 1:3], z[:, :, ::2], z[::2, :5]):
        with pytest.raises(ValueError):
            B._rows_2d(bad, "x")


def test_reference_encoder_agrees_with_the_oracle():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((33, 96)) * 2.0 ** rng.integers(-20, 20, (33, 1))).astype(np.float32)
    codes, sb = R.encode(x, "mxfp4")
    p, s = oracle.mxfp4_quantize(x)
    assert np.array_equal(R.pack(codes), p) and np.array_equal(sb, s)
    assert np.array_equal(R.unpack(p), codes)
    # decoding: the stored value is the nearest of the grid, within half a step of 6 / 4 amax
    v = R.decode(codes, sb, "mxfp4")
    assert (np.abs(v - x) <= np.repeat(2.0 ** (sb.astype(float) - 127), 32, 1)).all()


def test_reference_nvfp4_error_bound():
    """Half a step of the code (at most 1 in units of T) plus what a saturated or rounded scale loses."""
    rng = np.random.default_rng(4)
    x = rng.standard_normal((16, 64)).astype(np.float32)
    g = np.float32(np.abs(x).max() / 2688)
    codes, sb = R.encode(x, "nvfp4", g)
    v = R.decode(codes, sb, "nvfp4", g)
    T = np.repeat(R.E4M3[sb] * float(g), 16, 1)
    # the scale rounds down by at most 2^-4, so the largest code clips at most 6 (1 + 2^-4) - 6 = 0.375 T
    assert (np.abs(v - x) <= T * (1.0 + 1e-6)).all()


def test_refuses_more_rows_than_it_counts(B):
    L, P, BIG = B.lib(), ctypes.c_void_p, (1 << 30) + 1
    m = mat(B)
    assert L.csa_fp4_linear(MX, BIG, 256, 256, 1, m, m, BF16, P(16), 256, None) == UNSUPPORTED
    assert L.csa_grouped_out_proj_fp4_workspace(MX, BIG, 4, 128, 2, 128) == 0
    assert L.csa_grouped_out_proj_fp4(MX, BIG, 4, 128, 2, 128, 64, P(16), None, m, None, m, P(16), P(16), 1 << 62,
                                      None) == UNSUPPORTED
    rows = (1 << 40) + 1
    assert L.csa_fp4_scale_bytes(MX, rows, 64) == 0
    assert L.csa_fp4_quantize(MX, P(16), BF16, rows, 64, 64, m, None) == UNSUPPORTED
    assert L.csa_fp4_dequantize(MX, m, rows, 64, BF16, P(16), 64, None) == UNSUPPORTED
    assert L.csa_fp4_pack_scales(MX, P(16), rows, 64, P(16), None) == UNSUPPORTED


def test_rows_of_an_expanded_view_are_refused(B):
    """A stride of 0 in any dimension longer than 1 (inside, between, outside), or rows that overlap, names
    fewer rows than it counts: refused, since a call would read or write past the storage."""
    base = torch.zeros((4, 64))
    for t in (base[:, None].expand(4, 3, 64),                         # the inner row dimension
              torch.zeros((2, 1, 64)).expand(2, 3, 64),
              torch.zeros((2, 1, 4, 64)).expand(2, 5, 4, 64),         # between
              torch.zeros((1, 4, 64)).expand(3, 4, 64),               # the outer one
              torch.zeros((1, 1, 64)).expand(3, 4, 64),               # all of them
              torch.zeros((1, 64)).expand(5, 64), torch.zeros(64).expand(5, 64),
              torch.zeros(64).as_strided((2, 3, 16), (0, 16, 1)),
              torch.zeros(256).as_strided((5, 64), (32, 1))):         # rows half on one another
        with pytest.raises(ValueError):
            B._rows_2d(t, "x")
    # dimensions of one element may have any stride
    assert B._rows_2d(base.as_strided((1, 4, 64), (0, 64, 1)), "x") == (4, 64, 64)
    assert B._rows_2d(base.as_strided((4, 1, 64), (64, 0, 1)), "x") == (4, 64, 64)
    assert B._rows_2d(base[:1].as_strided((1, 1, 64), (0, 0, 1)), "x") == (1, 64, 64)


@pytest.mark.parametrize("seed", range(4))
def test_rows_of_any_view_stay_in_its_storage(B, seed):
    """Whatever view is taken as evenly spaced rows, the rows so described are the view's, in order."""
    rng = np.random.default_rng(seed)
    taken = 0
    for _ in range(400):
        nd = int(rng.integers(1, 5))
        shape = [int(v) for v in rng.integers(1, 4, nd - 1)] + [8]
        stride = [int(v) for v in rng.choice([0, 4, 8, 16, 24, 32, 48, 64, 96, 144], nd - 1)] + [1]
        size = 1 + sum((n - 1) * s for n, s in zip(shape, stride))
        base = torch.arange(size)
        t = base.as_strided(shape, stride)
        try:
            rows, cols, ld = B._rows_2d(t, "x")
        except ValueError:
            continue
        taken += 1
        assert rows * cols == t.numel() and (rows - 1) * ld + cols <= size
        assert torch.equal(base.as_strided((rows, cols), (ld, 1)), t.reshape(rows, cols))
    assert taken > 40


def test_give_up_refusals(B):
    L, P, I = B.lib(), ctypes.c_void_p, ctypes.c_int
    f = L.csa_selftest_fp4_give_up
    f.argtypes = [I, I, I, I, I, I, I, ctypes.POINTER(B._Fp4Mat), ctypes.POINTER(B._Fp4Mat), I, P, ctypes.c_int64, P]
    for barrier, ranks in ((0, 1), (8, 1), (1, 0), (1, 256), (-1, 1)):
        assert f(barrier, ranks, MX, 4, 256, 256, 1, mat(B), mat(B), BF16, P(16), 256, None) == INVALID
    assert f(1, 1, MX, 4, 256, 256, 1, mat(B), mat(B), F32, P(16), 256, None) == UNSUPPORTED
    assert f(1, 1, NV, 4, 256, 256, 1, mat(B, g=16), mat(B, g=16), BF16, P(16), 256, None) == UNSUPPORTED
    assert f(1, 1, MX, 4, 256, 48, 1, mat(B), mat(B), BF16, P(16), 256, None) == UNSUPPORTED
    assert f(1, 1, MX, 0, 256, 256, 1, mat(B), mat(B), BF16, None, 256, None) == 0
