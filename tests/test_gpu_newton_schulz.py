"""Newton-Schulz orthogonalisation against its definition in 64 bits."""
import ctypes

import numpy as np
import pytest
import torch

import tiled_matrix_multiplication_output_gb300 as tg

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ABC = tg.NEWTON_SCHULZ_COEFFICIENTS

# The result is stated to be within 2e-3 of exact arithmetic (relative, 2-norm
# of all elements) before it is rounded to the output type; FP16 storage of
# A and B alone moves it by about 1e-3.  4e-3 leaves a factor of two.  The
# output's rounding, half an ulp (2^-8 of an element for BF16) at worst and
# evenly spread, adds less than half of that over all elements.
STATED = 4e-3
ROUNDING = {"f32": 0.0, "f16": 2.0 ** -12, "bf16": 2.0 ** -9}


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    tg.load_library(build_if_missing=True)
    tg.gemm_debug_config(0, -1)


def _status():
    assert tg.gemm_device_status(torch.cuda.current_stream().cuda_stream) == tg.binding.OK


def reference(g, steps=5, abc=ABC, eps=1e-7):
    """The definition in 64 bits, one matrix."""
    x = np.asarray(g, np.float64)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    x = x / (np.sqrt((x * x).sum()) + eps)
    abc = [abc] * steps if not hasattr(abc[0], "__len__") else abc
    for a, b, c in abc:
        m = x @ x.T
        x = a * x + (b * m + c * (m @ m)) @ x
    return x.T if tall else x


def draw(rows, cols, dtype, kind, seed):
    rng = np.random.default_rng(seed)
    m = min(rows, cols)
    if kind == "flat":
        g = rng.standard_normal((rows, cols))
    elif kind == "low rank":
        r = max(1, m // 16)
        g = rng.standard_normal((rows, r)) @ rng.standard_normal((r, cols)) / np.sqrt(r) \
            + 0.05 * rng.standard_normal((rows, cols))
    else:  # decaying: singular values 1 / k
        u = np.linalg.qr(rng.standard_normal((rows, m)))[0]
        v = np.linalg.qr(rng.standard_normal((cols, m)))[0]
        g = (u / np.arange(1, m + 1)) @ v.T
    return torch.from_numpy(1e-2 * g).to(DT[dtype])


def expect(got, g, out, **kw):
    want = reference(g.double().cpu().numpy(), **kw)
    d = got.double().cpu().numpy() - want
    rel = np.linalg.norm(d) / np.linalg.norm(want)
    assert rel <= STATED + ROUNDING[out], f"{rel:.2e}"


SHAPES = [(1, 1), (1, 300), (300, 1), (8, 8), (16, 129), (100, 100), (128, 128), (129, 257),
          (200, 1000), (1000, 200), (333, 334), (640, 512)]


@pytest.mark.parametrize("kind", ["flat", "low rank", "decaying"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_matches_the_definition(rows, cols, kind):
    g = draw(rows, cols, "f32", kind, seed=rows * 7 + cols).cuda()
    got = tg.newton_schulz(g)
    _status()
    assert got.dtype == torch.float32 and got.shape == g.shape
    expect(got, g, "f32")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(96, 200), (515, 130)])
def test_types(rows, cols, dtype, out):
    g = draw(rows, cols, dtype, "low rank", seed=3).cuda()
    got = tg.newton_schulz(g, out_dtype=out)
    _status()
    assert got.dtype == DT[out]
    expect(got, g, out)


@pytest.mark.parametrize("rows,cols", [(2048, 2048), (1100, 3001), (4096, 1000)])
def test_many_tiles(rows, cols):
    """Several tiles per CTA pair in every product; the first twice the same."""
    g = draw(rows, cols, "bf16", "flat", seed=4).cuda()
    got = tg.newton_schulz(g)
    again = tg.newton_schulz(g)
    _status()
    assert torch.equal(got.view(torch.int16), again.view(torch.int16))
    expect(got, g, "bf16")


@pytest.mark.parametrize("rows,cols", [(96, 72), (64, 300), (513, 130)])
def test_batches_are_independent_matrices(rows, cols):
    g = torch.stack([draw(rows, cols, "f32", k, seed=i) * 10.0 ** (3 * i) for i, k in
                     enumerate(["flat", "low rank", "decaying", "flat", "flat"])]).cuda()
    got = tg.newton_schulz(g)
    _status()
    for i in range(g.shape[0]):
        expect(got[i], g[i], "f32")
    other = g.clone()
    other[1] = float("nan")
    alone = tg.newton_schulz(other)
    _status()
    assert torch.isnan(alone[1]).all()
    keep = [0, 2, 3, 4]
    assert torch.equal(alone[keep], got[keep])


def test_result_is_nearly_orthogonal():
    g = draw(256, 600, "f32", "low rank", seed=8).cuda()
    s = torch.linalg.svdvals(tg.newton_schulz(g, steps=8).double())
    assert s.min() > 0.6 and s.max() < 1.3


@pytest.mark.parametrize("steps", [1, 2, 7])
def test_steps_and_coefficients(steps):
    g = draw(150, 270, "f32", "decaying", seed=9).cuda()
    one = (2.0, -1.5, 0.5)
    expect(tg.newton_schulz(g, steps=steps, coefficients=one), g, "f32", steps=steps, abc=one)
    many = [(3.0 - 0.2 * i, -3.0 + 0.3 * i, 1.0 - 0.1 * i) for i in range(steps)]
    expect(tg.newton_schulz(g, steps=steps, coefficients=many), g, "f32", steps=steps, abc=many)
    _status()


def test_strides_offsets_and_in_place():
    big = draw(300, 500, "f32", "flat", seed=10).cuda()
    for g in (big[3:120, 1:258], big[::2, 7:40], big[:257, 4:204]):
        got = tg.newton_schulz(g)
        expect(got, g, "f32")
        store = torch.full((g.shape[0], g.shape[1] + 9), 7.0, device="cuda", dtype=torch.bfloat16)
        out = store[:, 5:5 + g.shape[1]]
        assert tg.newton_schulz(g, out=out) is out
        expect(out, g, "bf16")
        assert torch.all(store[:, :5] == 7.0) and torch.all(store[:, 5 + g.shape[1]:] == 7.0)
    batch = torch.stack([big, 2 * big])[:, 10:90, :100]
    want = tg.newton_schulz(batch.contiguous())
    assert torch.equal(tg.newton_schulz(batch), want)
    x = batch.contiguous()
    assert torch.equal(tg.newton_schulz(x, out=x), want)
    _status()


def test_workspace_and_stream():
    g = draw(130, 270, "bf16", "flat", seed=11).cuda()
    want = tg.newton_schulz(g)
    ws = torch.full((tg.gemm_newton_schulz_workspace_size(1, 130, 270),), 255, dtype=torch.uint8,
                    device="cuda")           # holds NaN wherever it is read before it is written
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = tg.newton_schulz(g, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_inside_a_cuda_graph():
    g = draw(96, 160, "f32", "flat", seed=12).cuda()
    ws = torch.empty(tg.gemm_newton_schulz_workspace_size(1, 96, 160), dtype=torch.uint8, device="cuda")
    tg.newton_schulz(g, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tg.newton_schulz(g, workspace=ws)
    g.copy_(draw(96, 160, "f32", "low rank", seed=13))
    graph.replay()
    torch.cuda.synchronize()
    expect(out, g, "f32")


def test_zero_tiny_huge_and_nonfinite():
    z = torch.zeros(40, 70, device="cuda")
    assert torch.all(tg.newton_schulz(z) == 0)
    assert torch.isnan(tg.newton_schulz(z, eps=0.0)).all()
    g = draw(40, 70, "f32", "flat", seed=14).cuda()
    for scale in (1e-12, 1e12):
        expect(tg.newton_schulz(g * scale, eps=0.0), g * scale, "f32", eps=0.0)
    for bad in (float("nan"), float("inf"), -float("inf")):
        h = g.clone()
        h[39, 69] = bad
        assert torch.isnan(tg.newton_schulz(h)).all()
    _status()


def test_empty_and_refusals():
    assert tg.newton_schulz(torch.empty(0, 5, device="cuda")).shape == (0, 5)
    assert tg.newton_schulz(torch.empty(0, 3, 5, device="cuda")).shape == (0, 3, 5)
    assert tg.newton_schulz(torch.empty(2, 3, 0, device="cuda")).shape == (2, 3, 0)
    g = torch.randn(32, 48, device="cuda")
    for bad in (g.cpu(), g.t(), g[0]):
        with pytest.raises(ValueError):
            tg.newton_schulz(bad)
    with pytest.raises(TypeError):
        tg.newton_schulz(g.double())
    with pytest.raises(ValueError):
        tg.newton_schulz(g, steps=0)
    with pytest.raises(ValueError):
        tg.newton_schulz(g, coefficients=[(1.0, 2.0)] * 5)
    with pytest.raises(ValueError):
        tg.newton_schulz(g, out=torch.empty(32, 47, device="cuda"))
    with pytest.raises(tg.GemmError):
        tg.newton_schulz(g, coefficients=(float("inf"), 0.0, 0.0))
    with pytest.raises(tg.GemmError):
        tg.newton_schulz(g, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(tg.GemmError):
        tg.newton_schulz(g, eps=-1.0)
    INV = tg.binding.ERR_INVALID_VALUE
    need = tg.gemm_newton_schulz_workspace_size(1, 32, 48)
    assert need > 0 and tg.gemm_newton_schulz_workspace_size(1, 0, 48) == 0
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    o = torch.full((32, 48), 5.0, device="cuda")
    abc = (ctypes.c_float * 3)(*ABC)

    def call(G=g.data_ptr(), ldg=48, O=o.data_ptr(), ldo=48, batch=1, steps=1, coef=abc,
             work=ws.data_ptr(), nbytes=need, dt=tg.F32):
        return tg.gemm_newton_schulz(G, ldg, 0, O, ldo, 0, batch, 32, 48, dt, tg.F32, steps, coef,
                                     1e-7, work, nbytes)

    assert call(G=None) == INV and call(O=None) == INV and call(coef=None) == INV
    assert call(ldg=47) == INV and call(ldo=47) == INV and call(steps=33) == INV
    assert call(work=None) == INV and call(work=ws.data_ptr() + 16) == INV
    assert call(nbytes=need - 1) == INV and call(dt=9) == INV and call(batch=-1) == INV
    assert call(batch=2) == INV                  # matrices would overlap
    torch.cuda.synchronize()
    assert torch.all(o == 5.0)
    assert call() == 0


@pytest.mark.parametrize("rows,cols", [(256, 256), (2048, 2048)])
def test_a_wait_that_runs_out_is_reported(rows, cols):
    g = draw(rows, cols, "f32", "flat", seed=15).cuda()
    tg.gemm_debug_config(20_000_000, 2)
    try:
        tg.newton_schulz(g, steps=1)
        sh = torch.cuda.current_stream().cuda_stream
        assert tg.gemm_device_status(sh) == tg.binding.ERR_TIMEOUT
    finally:
        tg.gemm_debug_config(0, -1)
    expect(tg.newton_schulz(g), g, "f32")
    _status()
