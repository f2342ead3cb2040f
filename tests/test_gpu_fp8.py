"""The block-scaled 8-bit operators against their definitions in 64 bits:
quantisation bit for bit, products within the bound of FP32 accumulation (and
bit for bit on integers), over every operand layout, block shape and type,
ragged sizes, strides, and values that are not finite."""
import numpy as np
import pytest
import torch

import tiled_matrix_multiplication_output_gb300 as tg
from tests import fp8_reference as ref
from tests.helpers import HALF_ULP

pytestmark = pytest.mark.gpu

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    tg.load_library(build_if_missing=True)
    tg.gemm_debug_config(0, -1)


def _status():
    assert tg.gemm_device_status(torch.cuda.current_stream().cuda_stream) == tg.binding.OK


def _draw(rows, cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))
    x = x * torch.exp(torch.randn(1, cols, generator=g))
    return x.to(DT[dtype])


def _check_codes(q, s, x, block, f8):
    want_q, want_s = ref.quantize(x.float().cpu().numpy(), block, f8)
    np.testing.assert_array_equal(s.cpu().numpy(), want_s)
    np.testing.assert_array_equal(q.float().cpu().numpy().astype(np.float64), want_q)


# ------------------------------------------------------------ quantisation

@pytest.mark.parametrize("block", ["row", "col", "tile"])
@pytest.mark.parametrize("dtype,f8", [("bf16", "e4m3"), ("f16", "e5m2"), ("f32", "e4m3")])
@pytest.mark.parametrize("rows,cols", [(1, 128), (1, 1), (16, 4096), (129, 127), (300, 1000),
                                       (127, 8), (257, 391)])
def test_quantize_is_the_definition(rows, cols, dtype, f8, block):
    x = _draw(rows, cols, dtype, seed=rows + cols).cuda()
    q, s = tg.quantize_fp8(x, block=block, dtype=f8)
    assert q.dtype == F8[f8] and tuple(q.shape) == (rows, cols)
    _check_codes(q, s, x, block, f8)


@pytest.mark.parametrize("dtype,f8", [("bf16", "e4m3"), ("f32", "e5m2")])
@pytest.mark.parametrize("rows,cols", [(1, 1), (200, 333), (128, 256)])
def test_quantize_pair_is_both_vector_forms(rows, cols, dtype, f8):
    x = _draw(rows, cols, dtype, seed=5).cuda()
    (qr, sr), (qc, sc) = tg.quantize_fp8_pair(x, dtype=f8)
    _check_codes(qr, sr, x, "row", f8)
    _check_codes(qc, sc, x, "col", f8)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quantize_strided_and_unaligned_rows(dtype):
    base = _draw(70, 600, dtype, seed=6).cuda()
    for x in (base[:, 8:300], base[3:40, 1:258], base[::2, :129]):
        for block in ("row", "col", "tile"):
            q, s = tg.quantize_fp8(x, block=block)
            _check_codes(q, s, x, block, "e4m3")


@pytest.mark.parametrize("block", ["row", "col", "tile"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quantize_zeros_nonfinite_and_extremes(dtype, block):
    x = _draw(140, 260, dtype, seed=7)
    big = torch.finfo(DT[dtype]).max
    tiny = torch.finfo(DT[dtype]).smallest_normal
    x[0:3] = 0.0                              # a row block of zeros
    x[:, 5] = 0.0                             # a column block of zeros
    x[9, 40], x[10, 41], x[11, 42] = float("nan"), float("inf"), float("-inf")
    x[20, 130] = big                          # the largest value is its block's scale
    x[21] = tiny * 0.5                        # subnormal rows
    x[22, :] = float("inf")                   # a row with nothing finite
    q, s = tg.quantize_fp8(x.cuda(), block=block)
    _check_codes(q, s, x, block, "e4m3")
    assert torch.isfinite(s).all()
    assert torch.isnan(q[9, 40].float()) and torch.isnan(q[10, 41].float())


def test_quantize_empty_and_refusals():
    q, s = tg.quantize_fp8(torch.empty(0, 5, device="cuda"))
    assert q.shape == (0, 5)
    x = torch.randn(8, 256, device="cuda")
    with pytest.raises(ValueError):
        tg.quantize_fp8(x.cpu())
    with pytest.raises(ValueError):
        tg.quantize_fp8(x.t())
    with pytest.raises(ValueError):
        tg.quantize_fp8(x, block="diagonal")
    with pytest.raises(TypeError):
        tg.quantize_fp8(x.double())
    q = torch.empty(8, 256, dtype=torch.uint8, device="cuda")
    s = torch.empty(2, 8, device="cuda")
    args = (x.data_ptr(), 256, 8, 256, tg.F32, tg.E4M3, 0)
    INV, UNS = tg.binding.ERR_INVALID_VALUE, tg.binding.ERR_UNSUPPORTED
    assert tg.gemm_fp8_quantize(*args, q.data_ptr() + 8, 256, s.data_ptr(), 8) == UNS
    assert tg.gemm_fp8_quantize(*args, q.data_ptr(), 260, s.data_ptr(), 8) == UNS
    assert tg.gemm_fp8_quantize(*args, q.data_ptr(), 240, s.data_ptr(), 8) == INV
    assert tg.gemm_fp8_quantize(*args, q.data_ptr(), 256, s.data_ptr(), 7) == INV
    assert tg.gemm_fp8_quantize(*args, None, 256, s.data_ptr(), 8) == INV


# ---------------------------------------------------------------- products

def _codes(values, f8):
    """Codes with 16-byte row pitch of exactly representable values."""
    rows, cols = values.shape
    buf = torch.zeros(rows, (cols + 15) // 16 * 16, device="cuda").to(F8[f8])
    buf[:, :cols] = torch.as_tensor(values, dtype=torch.float32).cuda().to(F8[f8])
    return buf[:, :cols]


def _operand(outer, K, k_rows, block, f8, seed, integers=False):
    """(codes, scales, block name) of an operand stored outer x K (k_rows) or K x outer."""
    rows, cols = (outer, K) if k_rows else (K, outer)
    name = "tile" if block == "tile" else ("row" if k_rows else "col")
    rng = np.random.default_rng(seed)
    br, bc = ref.BLOCK[name]
    sshape = (-(-rows // br), -(-cols // bc))
    if integers:
        v = rng.integers(-3, 4, (rows, cols)).astype(np.float64)
        s = 2.0 ** rng.integers(-1, 2, sshape)
    else:
        v = ref.round8(rng.standard_normal((rows, cols)) * 60, f8)
        s = np.exp(rng.standard_normal(sshape) * 2)
    s = s.astype(np.float32)
    s = np.ascontiguousarray(s.T if name == "row" else s)
    return _codes(v, f8), torch.from_numpy(s).cuda(), name


def _reference(a, sa, ba, op_a, b, sb, bb, op_b):
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    return ref.product(f(a), f(sa), ba, op_a, f(b), f(sb), bb, op_b)


def _product(M, N, K, op_a, op_b, block_a, block_b, f8_a="e4m3", f8_b="e4m3", integers=False,
             seed=0):
    a = _operand(M, K, op_a == "n", block_a, f8_a, seed, integers)
    b = _operand(N, K, op_b == "t", block_b, f8_b, seed + 1, integers)
    return a, b


def _expect(C, a, op_a, b, op_b, K, alpha=1.0, beta=0.0, C0=None):
    cref, cabs = _reference(*a, op_a, *b, op_b)
    cref, cabs = alpha * cref, abs(alpha) * cabs
    if beta != 0.0:
        cref = cref + beta * C0
        cabs = cabs + abs(beta) * np.abs(C0)
    bound = ref.product_bound(cabs, cref, K, HALF_ULP[C.dtype])
    got = C.double().cpu().numpy()
    assert np.isfinite(got).all()
    err = np.abs(got - cref)
    assert (err <= bound).all(), f"{(err > bound).sum()} out of bound, worst {np.max(err / bound)}"


SHAPES = [(1, 64, 128), (1, 1, 1), (7, 33, 100), (64, 136, 512), (96, 200, 1000), (129, 257, 385),
          (300, 520, 640)]


@pytest.mark.parametrize("op_a", ["n", "t"])
@pytest.mark.parametrize("op_b", ["n", "t"])
@pytest.mark.parametrize("block_a,block_b", [("vector", "tile"), ("vector", "vector"),
                                             ("tile", "vector"), ("tile", "tile")])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_integer_products_are_exact(M, N, K, block_a, block_b, op_a, op_b):
    a, b = _product(M, N, K, op_a, op_b, block_a, block_b, integers=True, seed=M + N)
    C = tg.matmul_fp8(*a[:2], *b[:2], op_a=op_a, op_b=op_b)
    _status()
    cref, _ = _reference(*a, op_a, *b, op_b)
    np.testing.assert_array_equal(C.double().cpu().numpy(), cref)


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("f8_a,f8_b", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2")])
@pytest.mark.parametrize("op_a,op_b,block_b", [("n", "t", "tile"), ("n", "n", "tile"),
                                               ("t", "n", "vector")])
@pytest.mark.parametrize("M,N,K", [(5, 200, 1000), (257, 384, 520)])
def test_random_products_within_the_bound(M, N, K, op_a, op_b, block_b, f8_a, f8_b, out):
    a, b = _product(M, N, K, op_a, op_b, "vector", block_b, f8_a, f8_b, seed=3)
    if out == "f16":  # keep the results in its range
        a = (a[0], a[1] * 2.0 ** -18, a[2])
    if f8_a != f8_b and out == "f16":
        a = (a[0], a[1] * 2.0 ** -6, a[2])
    C = tg.matmul_fp8(*a[:2], *b[:2], op_a=op_a, op_b=op_b, out_dtype=out)
    _status()
    _expect(C, a, op_a, b, op_b, K)


@pytest.mark.parametrize("M,N,K", [(2048, 2048, 1152), (1536, 2309, 700), (4000, 1290, 130)])
@pytest.mark.parametrize("op_a,op_b,block_b", [("n", "t", "tile"), ("t", "n", "vector")])
def test_many_tiles(M, N, K, op_a, op_b, block_b):
    """Several tiles per CTA or CTA pair, ragged in every dimension."""
    a, b = _product(M, N, K, op_a, op_b, "vector", block_b, seed=11)
    C = tg.matmul_fp8(*a[:2], *b[:2], op_a=op_a, op_b=op_b, out_dtype="bf16")
    C2 = tg.matmul_fp8(*a[:2], *b[:2], op_a=op_a, op_b=op_b, out_dtype="bf16")
    _status()
    assert torch.equal(C.view(torch.int16), C2.view(torch.int16))
    _expect(C, a, op_a, b, op_b, K)


@pytest.mark.parametrize("M,N,K", [(500, 4850, 300), (2300, 2290, 1160), (2500, 2100, 64)])
@pytest.mark.parametrize("op_a,op_b,block_b", [("n", "t", "tile"), ("n", "n", "vector"),
                                               ("t", "t", "vector"), ("t", "n", "tile")])
def test_last_tiles_shared_by_two_pairs(M, N, K, op_a, op_b, block_b):
    """A last wave of at most half as many tiles as there are CTA pairs (5 and
    14 beyond a whole one): their columns are split.  The first shape is one
    full wave of the smaller tiles."""
    a, b = _product(M, N, K, op_a, op_b, "vector", block_b, seed=13)
    kw = dict(op_a=op_a, op_b=op_b)
    C = tg.matmul_fp8(*a[:2], *b[:2], out_dtype="bf16", **kw)
    wide = torch.empty(M, N + 5, device="cuda")[:, :N].copy_(C)  # rows not on 16-byte boundaries
    C0 = wide.double().cpu().numpy()
    tg.matmul_fp8(*a[:2], *b[:2], out=wide, alpha=0.5, beta=-0.75, **kw)
    F = tg.matmul_fp8(*a[:2], *b[:2], **kw)
    F2 = tg.matmul_fp8(*a[:2], *b[:2], **kw)
    _status()
    assert torch.equal(F, F2)
    _expect(C, a, op_a, b, op_b, K)
    _expect(F, a, op_a, b, op_b, K)
    _expect(wide, a, op_a, b, op_b, K, 0.5, -0.75, C0)


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(3, 77, 300), (520, 512, 256), (520, 511, 256)])
def test_alpha_beta_into_a_strided_output(M, N, K, out):
    a, b = _product(M, N, K, "n", "t", "vector", "tile", integers=True, seed=21)
    store = torch.randint(-8, 8, (M, N + 5), device="cuda").to(DT[out])
    before = store.clone()
    C = store[:, 3:3 + N]
    C0 = C.double().cpu().numpy()
    got = tg.matmul_fp8(*a[:2], *b[:2], alpha=0.25, beta=-2.0, out=C)
    _status()
    assert got is C
    _expect(C, a, "n", b, "t", K, 0.25, -2.0, C0)
    assert torch.equal(store[:, :3], before[:, :3]) and torch.equal(store[:, 3 + N:], before[:, 3 + N:])


def test_beta_zero_ignores_what_the_output_held():
    a, b = _product(40, 130, 260, "n", "t", "vector", "tile", integers=True, seed=22)
    C = torch.full((40, 130), float("nan"), device="cuda")
    tg.matmul_fp8(*a[:2], *b[:2], out=C)
    _expect(C, a, "n", b, "t", 260)


def test_empty_contraction_and_empty_outputs():
    a = torch.empty(5, 0, device="cuda").to(F8["e4m3"])
    b = torch.empty(9, 0, device="cuda").to(F8["e4m3"])
    sa, sb = torch.empty(0, 5, device="cuda"), torch.empty(1, 0, device="cuda")
    C = torch.full((5, 9), 3.0, device="cuda")
    tg.matmul_fp8(a, sa, b, sb, out=C, beta=2.0)
    assert torch.all(C == 6.0)
    tg.matmul_fp8(a, sa, b, sb, out=C)
    assert torch.all(C == 0.0)
    z = tg.matmul_fp8(*_operand(130, 64, True, "tile", "e4m3", 1)[:2],
                      torch.empty(0, 64, device="cuda").to(F8["e4m3"]), torch.empty(0, 1, device="cuda"))
    assert z.shape == (130, 0)


def test_nan_stays_in_its_row_and_column():
    x = _draw(200, 384, "bf16", seed=30).cuda()
    w = _draw(136, 384, "bf16", seed=31).cuda()
    x[17, 200] = float("inf")
    w[50, 3] = float("nan")
    xq, xs = tg.quantize_fp8(x)
    wq, ws = tg.quantize_fp8(w, block="tile")
    C = tg.matmul_fp8(xq, xs, wq, ws)
    bad = torch.zeros(200, 136, dtype=torch.bool, device="cuda")
    bad[17] = True
    bad[:, 50] = True
    assert torch.equal(torch.isnan(C), bad)


def test_operands_inside_larger_matrices():
    """Row pitches above the row: neighbours are neither read nor written."""
    a, sa, na = _operand(100, 512, True, "vector", "e4m3", 40, True)
    wide = torch.full((100, 1024), 448.0, device="cuda").to(F8["e4m3"])
    wide[:, 256:768] = a
    part = wide[:, 256:700]                       # K = 444, ends inside a block
    b, sb, nb = _operand(72, 444, True, "tile", "e4m3", 41, True)
    C = tg.matmul_fp8(part, sa, b, sb)
    cref, _ = _reference(part, sa, na, "n", b, sb, nb, "t")
    np.testing.assert_array_equal(C.double().cpu().numpy(), cref)


def test_another_stream():
    x = _draw(333, 1000, "bf16", seed=50).cuda()
    w = _draw(200, 1000, "bf16", seed=51).cuda()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    xq, xs = tg.quantize_fp8(x, stream=s)
    wq, ws = tg.quantize_fp8(w, block="tile", stream=s)
    C = tg.matmul_fp8(xq, xs, wq, ws, stream=s)
    s.synchronize()
    _expect(C, (xq, xs, "row"), "n", (wq, ws, "tile"), "t", 1000)


def test_inside_a_cuda_graph():
    x = _draw(48, 640, "bf16", seed=52).cuda()
    w = _draw(264, 640, "bf16", seed=53).cuda()
    wq, ws = tg.quantize_fp8(w, block="tile")
    tg.matmul_fp8(*tg.quantize_fp8(x), wq, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        xq, xs = tg.quantize_fp8(x)
        C = tg.matmul_fp8(xq, xs, wq, ws)
    x.copy_(_draw(48, 640, "bf16", seed=54))
    g.replay()
    torch.cuda.synchronize()
    _check_codes(xq, xs, x, "row", "e4m3")
    _expect(C, (xq, xs, "row"), "n", (wq, ws, "tile"), "t", 640)


def test_product_refusals():
    a, sa, _ = _operand(32, 256, True, "vector", "e4m3", 60)
    b, sb, _ = _operand(64, 256, True, "tile", "e4m3", 61)
    with pytest.raises(ValueError):
        tg.matmul_fp8(a, sa, b[:, :128], sb[:, :1])                # inner sizes differ
    with pytest.raises(ValueError):
        tg.matmul_fp8(a, sa.t().contiguous(), b, sb)               # scales of another shape
    with pytest.raises(ValueError):
        tg.matmul_fp8(a, sa, b, sb, beta=1.0)                      # beta without out
    with pytest.raises(TypeError):
        tg.matmul_fp8(a.float(), sa, b, sb)
    with pytest.raises(ValueError):
        tg.matmul_fp8(a.cpu(), sa, b, sb)
    with pytest.raises(ValueError):
        tg.matmul_fp8(a, sa, b, sb, out=torch.empty(32, 65, device="cuda"))
    M = tg.Fp8Matrix
    C = torch.full((32, 64), 5.0, device="cuda")

    def call(am, bm, ldc=64):
        return tg.gemm_fp8(am, bm, C.data_ptr(), ldc, 32, 64, 256, 1.0, 0.0, tg.F32, None)

    A = M(a.data_ptr(), 256, 0, 0, sa.data_ptr(), 32, 0)
    B = M(b.data_ptr(), 256, 0, 2, sb.data_ptr(), 2, 1)
    INV, UNS = tg.binding.ERR_INVALID_VALUE, tg.binding.ERR_UNSUPPORTED
    assert call(M(a.data_ptr() + 1, 256, 0, 0, sa.data_ptr(), 32, 0), B) == UNS
    assert call(M(a.data_ptr(), 264, 0, 0, sa.data_ptr(), 32, 0), B) == UNS
    assert call(M(a.data_ptr(), 256, 0, 1, sa.data_ptr(), 256, 0), B) == UNS   # vectors across K
    assert call(M(a.data_ptr(), 240, 0, 0, sa.data_ptr(), 32, 0), B) == INV
    assert call(M(a.data_ptr(), 256, 2, 0, sa.data_ptr(), 32, 0), B) == INV
    assert call(M(a.data_ptr(), 256, 0, 0, sa.data_ptr(), 31, 0), B) == INV
    assert call(M(a.data_ptr(), 256, 0, 0, None, 32, 0), B) == INV
    assert call(M(None, 256, 0, 0, sa.data_ptr(), 32, 0), B) == INV
    assert call(M(a.data_ptr(), 256, 0, 0, sa.data_ptr(), 32, 5), B) == INV
    assert call(A, B, 63) == INV
    torch.cuda.synchronize()
    assert torch.all(C == 5.0)
    assert call(A, B) == 0


@pytest.mark.parametrize("M,N,K", [(8, 512, 1024), (200, 512, 1024), (2048, 2048, 1024)])
def test_a_wait_that_runs_out_is_reported(M, N, K):
    """The copies of one K step are left out, so a wait on them ends by its
    budget: the status says so, and the next product is right."""
    a, b = _product(M, N, K, "n", "t", "vector", "tile", integers=True, seed=70)
    tg.gemm_debug_config(20_000_000, 2)
    try:
        tg.matmul_fp8(*a[:2], *b[:2])
        sh = torch.cuda.current_stream().cuda_stream
        assert tg.gemm_device_status(sh) == tg.binding.ERR_TIMEOUT
    finally:
        tg.gemm_debug_config(0, -1)
    C = tg.matmul_fp8(*a[:2], *b[:2])
    _status()
    _expect(C, a, "n", b, "t", K)


def test_offsets_beyond_32_bits():
    """Inputs, codes and outputs of more than 2^31 elements: the last rows
    are as exact as the first."""
    rows, cols = 36000, 60000
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    some = [0, 17, rows // 2, rows - 1]
    x[some] = _draw(4, cols, "bf16", seed=80).cuda()
    q, s = tg.quantize_fp8(x)
    want_q, want_s = ref.quantize(x[some].float().cpu().numpy(), "row", "e4m3")
    np.testing.assert_array_equal(s[:, some].cpu().numpy(), want_s)
    np.testing.assert_array_equal(q[some].float().cpu().numpy(), want_q)
    del x
    # the contraction over the rows of the first: 36000 x 60000, as a K x M operand
    w, ws, _ = _operand(24, rows, True, "vector", "e4m3", 81, True)
    sc = torch.ones(-(-rows // 128), cols, device="cuda")
    C = tg.matmul_fp8(w, ws, q, sc, op_a="n", op_b="n")
    _status()
    b = q[some].double().cpu().numpy()
    a = w[:, some].double().cpu().numpy() * ws.t()[:, [r // 128 for r in some]].double().cpu().numpy()
    np.testing.assert_allclose(C.double().cpu().numpy(), a @ b, rtol=1e-6, atol=1e-6 * np.abs(a @ b).max())
    del C, q, sc
    # an output beyond 2^31 elements
    a, sa, na = _operand(rows, 64, True, "vector", "e4m3", 82, True)
    b, sb, nb = _operand(cols, 64, True, "tile", "e4m3", 83, True)
    C = tg.matmul_fp8(a, sa, b, sb, out_dtype="bf16")
    _status()
    pick = a[some], sa[:, some].contiguous()
    cref, _ = _reference(*pick, na, "n", b, sb, nb, "t")
    np.testing.assert_array_equal(C[some].double().cpu().numpy(),
                                  torch.from_numpy(cref).to(torch.bfloat16).double().numpy())
