"""Block-scaled 8-bit products, further forms: the block shapes of square
operands, and every form of the kernel for few output tiles."""
import pytest
import torch

import tiled_matrix_multiplication_output_gb300 as tg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    tg.load_library(build_if_missing=True)
    tg.gemm_debug_config(0, -1)


def _status():
    assert tg.gemm_device_status(torch.cuda.current_stream().cuda_stream) == tg.binding.OK


# ------------------------------------------------- block shapes of square operands

@pytest.mark.parametrize("n", [2, 128, 200, 512])
def test_vectors_across_the_contraction_of_a_square_matrix_are_refused(n):
    x = torch.randn(n, n, device="cuda")
    (rq, rs), (cq, cs) = tg.quantize_fp8_pair(x)
    assert rs.shape == cs.shape
    w, ws = tg.quantize_fp8(torch.randn(n, n, device="cuda"), block="tile")
    for call in (lambda: tg.matmul_fp8(rq, rs, w, ws, op_a="t"),
                 lambda: tg.matmul_fp8(cq, cs, w, ws),
                 lambda: tg.matmul_fp8(w, ws, rq, rs, op_b="n"),
                 lambda: tg.matmul_fp8(w, ws, cq, cs),
                 lambda: tg.matmul_fp8(cq, cs.clone(), w, ws, block_a="col"),
                 lambda: tg.matmul_fp8(w, ws, rq, rs.clone(), op_b="n", block_b="row")):
        with pytest.raises(ValueError):
            call()
    # along the contraction all of them are taken, and so are scales that say nothing
    q1, s1 = tg.quantize_fp8(x)
    want = tg.matmul_fp8(rq, rs, w, ws)
    assert torch.equal(tg.matmul_fp8(q1, s1, w, ws), want)
    assert torch.equal(tg.matmul_fp8(rq, rs.clone(), w, ws), want)
    assert torch.equal(tg.matmul_fp8(rq, cs.copy_(rs), w, ws, block_a="row"), want)
    tg.matmul_fp8(w, ws, rq, rs)
    tg.matmul_fp8(rq, rs, w, ws, op_b="n")
    with pytest.raises(ValueError):
        tg.matmul_fp8(rq, rs, w, ws, block_a="diagonal")
    _status()


def test_block_shapes_of_one_element_and_of_rows_are_one():
    one = torch.full((1, 1), 3.0, device="cuda")
    for block in ("row", "col", "tile"):
        q, s = tg.quantize_fp8(one, block=block)
        for op in ("n", "t"):
            C = tg.matmul_fp8(q, s, q, s, op_a=op, op_b=op)
            assert abs(float(C) - 9.0) <= 2 * 9.0 * 2.0 ** -4
    row = torch.ones(1, 100, device="cuda")
    q, s = tg.quantize_fp8(row, block="tile")      # one block: the scales are a row form's
    assert abs(float(tg.matmul_fp8(q, s, q, s)) - 100.0) <= 2 * 100.0 * 2.0 ** -4
    _status()


# ------------------------------------------------------- waits that run out

@pytest.mark.parametrize("M,N,K", [
    (8, 512, 4096), (40, 512, 2048), (24, 384, 1024),     # C's columns along the tile's rows
    (512, 8, 4096), (512, 60, 2048), (384, 24, 1024),     # C's rows along them
    (120, 1000, 384), (2048, 2048, 1024)])                # one block a tile; CTA pairs
def test_nothing_is_stored_after_a_wait_that_runs_out(M, N, K):
    """One K step's copies are left out.  Where K is divided over a cluster, only
    the block that holds the step gives up: the others' sums are whole, but none of
    them makes a result."""
    x, w = torch.randn(M, K, device="cuda"), torch.randn(N, K, device="cuda")
    a, b = tg.quantize_fp8(x), tg.quantize_fp8(w, block="tile")
    C = torch.full((M, N), 5.0, device="cuda")
    tg.gemm_debug_config(20_000_000, 2)
    try:
        tg.matmul_fp8(*a, *b, out=C)
        sh = torch.cuda.current_stream().cuda_stream
        assert tg.gemm_device_status(sh) == tg.binding.ERR_TIMEOUT
    finally:
        tg.gemm_debug_config(0, -1)
    assert torch.all(C == 5.0)
    tg.matmul_fp8(*a, *b, out=C)
    _status()
    want = x.double() @ w.double().t()
    # both operands are rounded to four bits: half an ulp is 2^-4 of an element at worst
    assert ((C.double() - want).abs() <= 2 * 2.0 ** -4 * 1.1 * (x.abs().double() @ w.abs().double().t())).all()
