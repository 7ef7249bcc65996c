"""The FP4 product when a wait runs out, without a fault.

``csa_selftest_fp4_give_up`` runs a product one of whose barriers waits for an arrival that never
comes.  Every role must leave within its limit, the copies under way must land before the shared
memory is given back, the host reads the timeout, and the next product, on the same SMs, is right.
Lone CTAs, clusters that split K and pairs of CTAs; the barrier starved in every CTA or in one.
"""
import ctypes
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

LOADED, FREE, SF_LOADED, SF_READY, DONE, ACC_FREE, RECEIVED = range(1, 8)
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def B(cuda):
    from compressed_sparse_long_02_b200 import binding
    L = binding.lib()
    I, P, MAT = ctypes.c_int, ctypes.c_void_p, ctypes.POINTER(binding._Fp4Mat)
    L.csa_selftest_fp4_give_up.argtypes = [I, I, I, I, I, I, I, MAT, MAT, I, P, ctypes.c_int64, P]
    L.csa_selftest_fp4_give_up.restype = I
    return binding


def check(B, dev, fmt, M, N, K, dtype, barrier, ranks):
    g = torch.full((1,), 6.0 / 2688, device=dev) if fmt == "nvfp4" else None
    x = B.csa_fp4_quantize(torch.randn((M, K), device=dev), fmt=fmt, tensor_scale=g)
    w = B.csa_fp4_quantize(torch.randn((N, K), device=dev), fmt=fmt, tensor_scale=g)
    want = B.csa_fp4_linear(x, w, out_dtype=dtype)
    assert B.csa_get_device_error() == 0
    y = torch.zeros_like(want)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    st = B.lib().csa_selftest_fp4_give_up(barrier, ranks, B._FP4_FMT[fmt], M, N, K, 1, ctypes.byref(B._fp4_mat(x, "x", dev)),
                                          ctypes.byref(B._fp4_mat(w, "w", dev)), B._dt(y), y.data_ptr(), N, B._stream(y))
    again = B.csa_fp4_linear(x, w, out_dtype=dtype)  # queued behind it
    torch.cuda.synchronize()
    took = time.perf_counter() - t0
    assert st == 0 and B.csa_get_device_error() == B.DEVERR_TIMEOUT  # read and cleared
    assert took < 1.5, f"{took:.2f} s: more than a limit for the roles, one for the copies and one for the other CTA"
    assert torch.equal(again, want)
    assert torch.equal(B.csa_fp4_linear(x, w, out_dtype=dtype), want) and B.csa_get_device_error() == 0


@pytest.mark.parametrize("barrier", [LOADED, FREE, SF_LOADED, SF_READY, DONE])
def test_lone_ctas_give_up(B, cuda, barrier):
    try:
        B.csa_set_batch_invariant(True)  # K in one piece
        check(B, cuda, "mxfp4", 1, 512, 8192, BF16, barrier, 1)
    finally:
        B.csa_set_batch_invariant(False)


@pytest.mark.parametrize("M,N,K", [(40000, 128, 64)])
def test_lone_ctas_give_up_between_tiles(B, cuda, M, N, K):
    check(B, cuda, "nvfp4", M, N, K, F32, ACC_FREE, 1)


@pytest.mark.parametrize("ranks", [1, 2, 255])
@pytest.mark.parametrize("barrier", [LOADED, FREE, SF_LOADED, SF_READY, DONE, RECEIVED])
def test_clusters_that_split_k_give_up(B, cuda, barrier, ranks):
    check(B, cuda, "nvfp4", 20, 512, 32768, F32, barrier, ranks)


@pytest.mark.parametrize("fmt,dtype", [("mxfp4", BF16), ("nvfp4", F32)])
@pytest.mark.parametrize("barrier,ranks", [(LOADED, 3), (FREE, 3), (FREE, 1), (FREE, 2), (SF_LOADED, 3), (SF_LOADED, 1),
                                           (SF_LOADED, 2), (SF_READY, 3), (DONE, 3), (DONE, 1), (DONE, 2)])
def test_pairs_give_up(B, cuda, fmt, dtype, barrier, ranks):
    """FREE in one CTA only: the other goes on to load up to a ring of slabs that the leader has not announced,
    or the leader announces slabs that the other never loads."""
    check(B, cuda, fmt, 600, 4096, 8192, dtype, barrier, ranks)


@pytest.mark.parametrize("fmt,dtype", [("mxfp4", BF16), ("nvfp4", F32)])
def test_pairs_give_up_between_tiles(B, cuda, fmt, dtype):
    check(B, cuda, fmt, 2048, 4096, 4096, dtype, ACC_FREE, 3)
