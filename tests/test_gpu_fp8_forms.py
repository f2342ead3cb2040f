"""Block-scaled 8-bit products, further forms: the block shapes of square
operands, and every form of the kernel for few output tiles."""
import numpy as np
import pytest
import torch

import tiled_matrix_multiplication_output_gb300 as tg
from tests.test_gpu_fp8 import DT, _expect, _product, _reference

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


# ------------------------------------------- every form of the few-tiles kernel

# (columns of a tile, blocks a tile's K is divided over, whether C's rows lie
# along the tile's columns): the shorter side gives the columns, K the blocks
FEW = [(1, 1024, 4096),      # 16, 8, no
       (1, 4096, 4096),      # 16, 4, no
       (16, 9000, 1000),     # 16, 2, no
       (13, 18000, 600),     # 16, 1, no
       (24, 512, 4096),      # 32, 8, no
       (32, 1000, 1200),     # 32, 4, no
       (20, 300, 600),       # 32, 2, no
       (64, 512, 4096),      # 64, 8, no
       (64, 2500, 2500),     # 64, 4, no
       (50, 700, 1000),      # 64, 4, no
       (60, 9001, 1000),     # 64, 2, no
       (200, 257, 1100)]     # 64, 4, no; several columns of tiles


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("op_a,op_b,block_b", [("n", "t", "tile"), ("n", "n", "tile"), ("t", "n", "vector"),
                                               ("t", "t", "vector")])
@pytest.mark.parametrize("M,N,K", FEW + [(n, m, k) for m, n, k in FEW])
def test_few_tiles_in_every_form(M, N, K, op_a, op_b, block_b, out):
    """Integers (exact in FP32), then values of any size, with alpha alone and with beta."""
    a, b = _product(M, N, K, op_a, op_b, "vector", block_b, integers=True, seed=M + K)
    C = tg.matmul_fp8(*a[:2], *b[:2], op_a=op_a, op_b=op_b)
    again = tg.matmul_fp8(*a[:2], *b[:2], op_a=op_a, op_b=op_b)
    cref, _ = _reference(*a, op_a, *b, op_b)
    np.testing.assert_array_equal(C.double().cpu().numpy(), cref)
    assert torch.equal(C, again)
    a, b = _product(M, N, K, op_a, op_b, "vector", block_b, "e5m2", seed=M + K + 1)
    D = tg.matmul_fp8(*a[:2], *b[:2], op_a=op_a, op_b=op_b, out_dtype=out, alpha=0.5)
    _expect(D, a, op_a, b, op_b, K, 0.5)
    E = D.clone()
    tg.matmul_fp8(*a[:2], *b[:2], op_a=op_a, op_b=op_b, out=E, alpha=-2.0, beta=0.25)
    _status()
    _expect(E, a, op_a, b, op_b, K, -2.0, 0.25, D.double().cpu().numpy())


# ------------------------------------------------------------- alpha without beta

@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(40, 512, 2000),        # few tiles
                                   (300, 520, 640),        # 128 x 128 tiles
                                   (2048, 4096, 512),      # CTA pairs
                                   (2300, 2296, 640)])     # a last wave in parts
@pytest.mark.parametrize("op_a,op_b,block_b", [("n", "t", "tile"), ("t", "n", "vector")])
def test_alpha_into_aligned_outputs(M, N, K, op_a, op_b, block_b, out):
    """Stored by TMA (but for few tiles), where alpha is the only factor."""
    a, b = _product(M, N, K, op_a, op_b, "vector", block_b, seed=M)
    if out == "f16":  # keep the results in its range
        a = (a[0], a[1] * 2.0 ** -24, a[2])
    C = torch.full((M, N), float("nan"), device="cuda", dtype=DT[out])
    tg.matmul_fp8(*a[:2], *b[:2], op_a=op_a, op_b=op_b, out=C, alpha=0.375)
    _status()
    _expect(C, a, op_a, b, op_b, K, 0.375)


# ------------------------------------------------------------------ in a graph

def test_few_tiles_inside_a_cuda_graph():
    """K of more than six blocks: the cluster kernel."""
    def draws(seed):
        g = torch.Generator().manual_seed(seed)
        return torch.randn(48, 1500, generator=g).to(torch.bfloat16).cuda()

    x, w = draws(1), torch.randn(264, 1500, device="cuda")
    wq, ws = tg.quantize_fp8(w, block="tile")
    tg.matmul_fp8(*tg.quantize_fp8(x), wq, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        xq, xs = tg.quantize_fp8(x)
        C = tg.matmul_fp8(xq, xs, wq, ws)
    x.copy_(draws(2))
    g.replay()
    torch.cuda.synchronize()
    _expect(C, (xq, xs, "row"), "n", (wq, ws, "tile"), "t", 1500)
