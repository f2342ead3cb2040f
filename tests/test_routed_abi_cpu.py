"""Host-side checks of the grouped products and the adapters that need no GPU:
bad arguments are rejected before a device is touched, empty problems are
no-ops."""
import pytest
import torch

import tiled_matrix_multiplication_output_gb300 as tg
from tiled_matrix_multiplication_output_gb300 import build as tgbuild

INV, UNS = tg.binding.ERR_INVALID_VALUE, tg.binding.ERR_UNSUPPORTED
BIG = tg.binding.MAX_DIM
P = 4096  # a dummy aligned address; never dereferenced on these paths


@pytest.fixture(scope="module", autouse=True)
def lib():
    if tgbuild.nvcc_path() is None:
        pytest.skip("nvcc not available")
    tgbuild.build()
    return tg.load_library()


def _grouped(X=P, ldx=64, W=P, ldw=64, stride=64 * 32, op=1, off=P, Y=P, ldy=32, rows=10, groups=3,
             N=32, K=64, dt=tg.BF16, out=tg.F32, ws=None, nbytes=0):
    return tg.gemm_grouped(X, ldx, W, ldw, stride, op, off, Y, ldy, rows, groups, N, K, 1.0, 0.0, 0,
                           dt, out, ws, nbytes)


def test_grouped_rejects_bad_arguments():
    for bad in (dict(X=None), dict(W=None), dict(off=None), dict(Y=None), dict(ldx=63), dict(ldw=63),
                dict(op=0, ldw=31), dict(op=2), dict(op=-1), dict(ldy=31), dict(stride=-1),
                dict(rows=-1), dict(rows=BIG + 1), dict(groups=-1), dict(N=-1), dict(K=-1),
                dict(N=BIG + 1), dict(K=BIG + 1), dict(dt=3), dict(out=3)):
        assert _grouped(**bad) == INV, bad
    assert _grouped(groups=1025) == UNS
    size = tg.gemm_grouped_workspace_size
    assert size(P, 64, P, 64, 64 * 32, 10, 3, 32, 64, 1, tg.BF16) == 0
    assert size(P, 65, P, 65, 65 * 32, 10, 3, 32, 64, 1, tg.F32) == 0
    assert size(P + 2, 64, P, 64, 64 * 32, 10, 3, 32, 64, 1, tg.BF16) >= 10 * 64 * 2
    need = size(P, 64, P, 65, 65 * 32, 10, 3, 32, 64, 1, tg.BF16)
    assert need >= 3 * 64 * 32 * 2  # copies to aligned rows
    for bad in (dict(ws=None, nbytes=need), dict(ws=P + 16, nbytes=need), dict(ws=P, nbytes=need - 1)):
        assert _grouped(ldw=65, stride=65 * 32, **bad) == INV, bad
    assert _grouped(rows=0, X=None, Y=None, off=None) == 0
    assert _grouped(N=0, W=None, Y=None, ldy=0) == 0


def _wgrad(D=P, ldd=32, X=P, ldx=64, off=P, C=P, ldc=64, stride=64 * 32, rows=10, groups=3, N=32,
           K=64, dt=tg.BF16, out=tg.F32):
    return tg.gemm_grouped_wgrad(D, ldd, X, ldx, off, C, ldc, stride, rows, groups, N, K, 1.0, 0.0,
                                 dt, out)


def test_wgrad_rejects_bad_arguments():
    for bad in (dict(D=None), dict(X=None), dict(off=None), dict(C=None), dict(ldd=31), dict(ldx=63),
                dict(ldc=63), dict(stride=64 * 32 - 1), dict(stride=-1), dict(rows=-1),
                dict(rows=BIG + 1), dict(groups=-1), dict(N=-1), dict(K=BIG + 1), dict(dt=-1),
                dict(out=9)):
        assert _wgrad(**bad) == INV, bad
    assert _wgrad(ldc=2 ** 62, stride=2 ** 62) == INV  # rows of one result reach into the next
    assert _wgrad(groups=1025) == UNS
    assert tg.gemm_grouped_wgrad_workspace_size(P, 32, P, 64, 10, 32, 64, tg.F16) == 0
    assert tg.gemm_grouped_wgrad_workspace_size(P, 33, P, 64, 10, 32, 64, tg.F16) >= 10 * 32 * 2
    assert _wgrad(ldd=33) == INV  # no workspace for the copy
    assert _wgrad(groups=0, off=None, C=None) == 0
    assert _wgrad(N=0, C=None) == _wgrad(K=0, C=None, ldc=0) == 0


def _adapters(A=P, lda=64, sa=64 * 8, B=P, ldb=8, sb=32 * 8, scale=None, G=3, r=8):
    return tg.LoraAdapters(A, lda, sa, B, ldb, sb, scale, G, r)


def _lora(X=P, ldx=64, W=P, ldw=64, lora=None, of=P, Y=P, ldy=32, rows=10, N=32, K=64, dt=tg.BF16,
          out=tg.F32, ws=P, nbytes=1 << 30):
    return tg.gemm_lora(X, ldx, W, ldw, lora or _adapters(), of, Y, ldy, rows, N, K, dt, out, ws,
                        nbytes)


def test_lora_rejects_bad_arguments():
    def size(rows, r=40, G=3, dt=tg.BF16, ldx=64):
        return tg.gemm_lora_workspace_size(P, ldx, P, 64, _adapters(G=G, r=r), rows, 32, 64, dt, tg.F32)

    assert 0 < size(10) < size(1000) < size(1000, r=200)
    assert size(10, ldx=67) >= size(10) + 10 * 64 * 2  # room for a copy
    assert size(-1) == size(10, r=257) == size(10, G=-1) == size(10, dt=5) == 0
    need = size(10)
    for bad in (dict(X=None), dict(W=None), dict(Y=None), dict(of=None), dict(ldx=63), dict(ldw=63),
                dict(ldy=31), dict(rows=-1), dict(N=BIG + 1), dict(K=-1), dict(dt=3), dict(out=-1),
                dict(ws=None), dict(ws=P + 16), dict(nbytes=need - 1)):
        assert _lora(lora=_adapters(r=40, ldb=40, sb=32 * 40), **bad) == INV, bad
    for bad in (dict(A=None), dict(B=None), dict(lda=63), dict(ldb=7), dict(sa=-1), dict(sb=-1),
                dict(G=-1), dict(G=65536), dict(r=-1)):
        assert _lora(lora=_adapters(**bad)) == INV, bad
    assert _lora(lora=_adapters(r=257, ldb=300)) == UNS
    assert _lora(rows=0, X=None, Y=None, of=None, ws=None) == 0
    assert _lora(N=0, W=None, Y=None, ws=None) == 0


def _backward(D=P, ldd=32, X=P, ldx=64, W=P, ldw=64, lora=None, of=P, DX=P, lddx=64, DA=P, ldda=64,
              sda=64 * 8, DB=P, lddb=8, sdb=32 * 8, rows=10, N=32, K=64, dt=tg.BF16, out=tg.F32,
              grad=tg.F32, ws=P, nbytes=1 << 30):
    return tg.gemm_lora_backward(D, ldd, X, ldx, W, ldw, lora or _adapters(), of, DX, lddx, DA, ldda,
                                 sda, DB, lddb, sdb, rows, N, K, dt, out, grad, ws, nbytes)


def test_lora_backward_rejects_bad_arguments():
    need = tg.gemm_lora_backward_workspace_size(P, 32, P, 64, P, 64, _adapters(), 10, 32, 64, tg.BF16,
                                                tg.F32, tg.F32)
    for bad in (dict(D=None), dict(X=None), dict(W=None), dict(of=None), dict(ldd=31), dict(ldx=63),
                dict(ldw=63), dict(lddx=63), dict(ldda=63), dict(sda=64 * 8 - 1), dict(lddb=7),
                dict(sdb=32 * 8 - 1), dict(rows=-1), dict(grad=3), dict(out=3), dict(dt=3),
                dict(ws=None), dict(ws=P + 128), dict(nbytes=need - 1)):
        assert _backward(**bad) == INV, bad
    assert _backward(lora=_adapters(r=257, ldb=300)) == UNS
    assert _backward(DX=None, DA=None, DB=None, X=None, W=None, ws=None) == 0


def test_cpu_tensors_are_rejected():
    x, w, o = torch.zeros(4, 4), torch.zeros(2, 4, 4), torch.zeros(3, dtype=torch.int32)
    of = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: tg.matmul_grouped(x, w, o), lambda: tg.matmul_grouped_wgrad(x, x, o),
                 lambda: tg.matmul_lora(x, x, w, w, of),
                 lambda: tg.matmul_lora_backward(x, x, x, w, w, of)):
        with pytest.raises(ValueError):
            call()


def test_bench_floor_of_the_routed_operators():
    import bench
    peaks = {"hbm_gbs": 6800.0, "bf16_tflops": 1876.6}
    for op in ("grouped", "wgrad", "lora", "lora_backward"):
        assert bench.operator_floor_us(op, {"bytes": 6.8e9, "flops": 1.0}, peaks) == pytest.approx(1000.0)
        assert bench.operator_floor_us(op, {"bytes": 1, "flops": 1.8766e12}, peaks) == pytest.approx(1000.0)


def test_row_stacks_and_vectors_are_checked_before_the_library():
    """The binding's own checks, on tensors that say they are on a device."""
    from tiled_matrix_multiplication_output_gb300 import binding

    class T:
        def __init__(self, shape, stride, dtype=torch.bfloat16, device=0, contiguous=True):
            self.shape, self._s, self.dtype, self._d, self._c = shape, stride, dtype, device, contiguous

        def stride(self):
            return self._s

        def get_device(self):
            return self._d

        def is_contiguous(self):
            return self._c

        def data_ptr(self):
            return 64

    bf16, i32 = torch.bfloat16, torch.int32
    assert binding._rows_of(T((4, 8), (10, 1)), "x", bf16, 0) == (4, 8, 10)
    assert binding._rows_of(T((1, 9), (3, 1)), "x", bf16, 0) == (1, 9, 16)
    assert binding._rows_of(T((4, 1), (5, 7)), "x", None, 0) == (4, 1, 5)
    for bad in (T((4, 8), (7, 1)), T((4, 8), (16, 2)), T((4, 8, 2), (16, 2, 1)), T((4, 8), (8, 1), device=1)):
        with pytest.raises(ValueError):
            binding._rows_of(bad, "x", bf16, 0)
    with pytest.raises(TypeError):
        binding._rows_of(T((4, 8), (8, 1)), "x", torch.float16, 0)
    assert binding._stack_of(T((3, 4, 8), (32, 8, 1)), "w", bf16, 0) == (3, 4, 8, 8, 32)
    assert binding._stack_of(T((3, 4, 8), (0, 8, 1)), "w", bf16, 0) == (3, 4, 8, 8, 0)
    assert binding._stack_of(T((1, 4, 8), (7, 8, 1)), "w", bf16, 0) == (1, 4, 8, 8, 32)
    for bad in (T((3, 4, 8), (32, 8, 2)), T((3, 4, 8), (32, 7, 1)), T((4, 8), (8, 1)),
                T((3, 4, 8), (32, 8, 1), device=-1)):
        with pytest.raises(ValueError):
            binding._stack_of(bad, "w", bf16, 0)
    assert binding._vector_of(T((5,), (1,), i32), "o", 5, i32, 0) == 64
    for bad in (T((4,), (1,), i32), T((5,), (2,), i32, contiguous=False), T((5, 1), (1, 1), i32),
                T((5,), (1,), i32, device=2)):
        with pytest.raises(ValueError):
            binding._vector_of(bad, "o", 5, i32, 0)
    with pytest.raises(TypeError):
        binding._vector_of(T((5,), (1,), torch.int64), "o", 5, i32, 0)


def test_interleaved_results_that_overlap_are_rejected():
    """Results may be interleaved row by row (the pitch holds a row of each); rows that
    reach into the next are not accepted."""
    for stride, ldc in ((7, 24), (8, 23), (9, 25), (31, 8), (0, 24), (-8, 24), (2 ** 62, 2 ** 62)):
        assert _wgrad(stride=stride, ldc=ldc, N=4, K=8, ldx=8) == INV, (stride, ldc)
