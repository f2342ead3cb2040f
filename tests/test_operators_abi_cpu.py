"""Host-side checks of the 8-bit and orthogonalisation entry points that need
no GPU: bad arguments are rejected before a device is touched, empty problems
are no-ops."""
import ctypes
import os
import subprocess

import pytest
import torch

import tiled_matrix_multiplication_output_gb300 as tg
from tiled_matrix_multiplication_output_gb300 import build as tgbuild

INV, UNS = tg.binding.ERR_INVALID_VALUE, tg.binding.ERR_UNSUPPORTED
BIG = tg.binding.MAX_DIM
P = 256  # a dummy aligned address; never dereferenced on these paths


@pytest.fixture(scope="module", autouse=True)
def lib():
    if tgbuild.nvcc_path() is None:
        pytest.skip("nvcc not available")
    tgbuild.build()
    return tg.load_library()


def _quantize(X=P, ldx=128, rows=4, cols=128, dt=tg.BF16, f8=tg.E4M3, block=0, Q=P, ldq=128, S=P,
              lds=4):
    return tg.gemm_fp8_quantize(X, ldx, rows, cols, dt, f8, block, Q, ldq, S, lds)


def test_quantize_rejects_bad_arguments():
    for bad in (dict(X=None), dict(Q=None), dict(S=None), dict(rows=-1), dict(cols=-1),
                dict(rows=BIG + 1), dict(ldx=127), dict(ldq=112), dict(lds=3), dict(dt=3),
                dict(f8=2), dict(block=3), dict(block=-1)):
        assert _quantize(**bad) == INV, bad
    assert _quantize(Q=P + 8) == UNS
    assert _quantize(ldq=136) == UNS
    assert _quantize(block=1, lds=127) == INV       # a scale for each column
    assert _quantize(block=2, lds=0) == INV
    assert _quantize(rows=0, X=None, Q=None, S=None) == 0
    assert _quantize(cols=0, X=None, Q=None, S=None, ldx=0) == 0
    pair = tg.gemm_fp8_quantize_pair
    assert pair(P, 128, 4, 128, tg.F32, 0, P, 128, P, 4, P, 128, P, 127) == INV
    assert pair(P, 128, 4, 128, tg.F32, 0, P, 128, P, 3, P, 128, P, 128) == INV
    assert pair(P, 128, 4, 128, tg.F32, 0, P, 128, P, 4, P + 1, 128, P, 128) == UNS
    assert pair(None, 128, 0, 128, tg.F32, 0, None, 0, None, 0, None, 0, None, 0) == 0


def _matrix(data=P, ld=128, type=0, block=0, scale=P, scale_ld=8, op=0):
    return tg.Fp8Matrix(data, ld, type, block, scale, scale_ld, op)


def _product(A=None, B=None, C=P, ldc=8, M=8, N=8, K=128, out=tg.F32):
    return tg.gemm_fp8(A or _matrix(), B or _matrix(op=1), C, ldc, M, N, K, 1.0, 0.0, out)


def test_product_rejects_bad_arguments():
    for bad in (dict(C=None), dict(ldc=7), dict(M=-1), dict(N=-1), dict(K=-1), dict(M=BIG + 1),
                dict(K=BIG + 1), dict(out=3)):
        assert _product(**bad) == INV, bad
    for bad in (dict(data=None), dict(scale=None), dict(ld=112), dict(type=2), dict(block=3),
                dict(scale_ld=7), dict(op=2)):
        assert _product(A=_matrix(**bad)) == INV, bad
        assert _product(B=_matrix(**{"op": 1, **bad})) == INV, bad
    assert tg.gemm_fp8(None, _matrix(), P, 8, 8, 8, 128, 1.0, 0.0, tg.F32) == INV
    for bad in (dict(data=P + 8), dict(ld=136), dict(block=1, scale_ld=128)):  # the last: across K
        assert _product(A=_matrix(**bad)) == UNS, bad
    assert _product(M=0, C=None) == 0
    assert _product(N=0, C=None, ldc=0) == 0


def test_orthogonalisation_rejects_bad_arguments():
    abc = (ctypes.c_float * 6)(3.0, -3.0, 1.0, 3.0, -3.0, 1.0)
    size = tg.gemm_newton_schulz_workspace_size
    assert size(1, 32, 48) > 0 and size(2, 32, 48) > size(1, 32, 48)
    assert size(0, 32, 48) == size(1, 0, 48) == size(1, 32, -1) == size(65536, 1, 1) == 0

    def call(G=P, ldg=48, sg=1536, O=P, ldo=48, so=1536, batch=2, rows=32, cols=48, dt=tg.F32,
             out=tg.F32, steps=2, coef=abc, eps=1e-7, ws=P, nbytes=1 << 30):
        return tg.gemm_newton_schulz(G, ldg, sg, O, ldo, so, batch, rows, cols, dt, out, steps,
                                     coef, eps, ws, nbytes)

    for bad in (dict(G=None), dict(O=None), dict(ldg=47), dict(ldo=47), dict(sg=1535),
                dict(so=1535), dict(batch=-1), dict(batch=65536), dict(rows=-1), dict(cols=BIG + 1),
                dict(dt=7), dict(out=-1), dict(steps=0), dict(steps=33), dict(coef=None),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(ws=None),
                dict(ws=P + 16), dict(nbytes=size(2, 32, 48) - 1)):
        assert call(**bad) == INV, bad
    bad = (ctypes.c_float * 6)(3.0, -3.0, 1.0, 3.0, float("nan"), 1.0)
    assert call(coef=bad) == INV
    for empty in (dict(batch=0), dict(rows=0), dict(cols=0)):
        assert call(**empty, G=None, O=None, ws=None) == 0


def test_cpu_tensors_are_rejected():
    x = torch.zeros(4, 4)
    for call in (lambda: tg.quantize_fp8(x), lambda: tg.quantize_fp8_pair(x),
                 lambda: tg.newton_schulz(x), lambda: tg.matmul_fp8(x, x, x, x)):
        with pytest.raises(ValueError):
            call()


def test_bench_floor_of_an_operator():
    import bench
    peaks = {"hbm_gbs": 6800.0, "bf16_tflops": 1876.6}
    work = {"bytes": 6.8e9, "flops": 1.8766e12}
    assert bench.operator_floor_us("quant", work, peaks) == pytest.approx(1000.0)
    assert bench.operator_floor_us("orth", work, peaks) == pytest.approx(1000.0)
    assert bench.operator_floor_us("orth", {"bytes": 1, "flops": 1.8766e12}, peaks) == pytest.approx(1000.0)
    assert bench.operator_floor_us("product", {"bytes": 1, "flops": 1.8766e12}, peaks) == pytest.approx(500.0)


def test_orthogonalisation_rejects_batches_that_overlap():
    """Strides up to the ends of 64 bits, too."""
    abc = (ctypes.c_float * 3)(3.0, -3.0, 1.0)
    big = 2 ** 63 - 1

    def call(ldg=48, sg=1536, ldo=48, so=1536, batch=3, rows=32, cols=48):
        return tg.gemm_newton_schulz(P, ldg, sg, P, ldo, so, batch, rows, cols, tg.F32, tg.F32, 1,
                                     abc, 1e-7, P, 1 << 30)

    for bad in (dict(so=0), dict(so=1535), dict(so=-1), dict(so=-big), dict(sg=1535), dict(sg=-1536),
                dict(ldo=143, so=48), dict(ldg=143, sg=48), dict(ldo=big, so=47),
                dict(ldo=big // 8, so=big // 2), dict(ldg=big // 8, sg=big // 2)):
        assert call(**bad) == INV, bad


def test_a_failed_occupancy_query_is_no_launch_error(tmp_path):
    """ns_resident.cu linked against a stand-in for the CUDA runtime."""
    here = os.path.dirname(os.path.abspath(__file__))
    exe = str(tmp_path / "fake_occupancy")
    cmd = [tgbuild.nvcc_path(), *tgbuild.ARCH, *tgbuild.NVCC_FLAGS, "-O1", "-Xptxas", "-O0", "-cudart", "none",
           "-o", exe, os.path.join(here, "c", "fake_occupancy.cpp"),
           os.path.join(tgbuild.CSRC, "ns_resident.cu")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout
