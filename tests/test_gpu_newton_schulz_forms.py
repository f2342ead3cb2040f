"""Newton-Schulz orthogonalisation, further forms: batches that are not
stacked, every size of the one-launch form, extreme norms, precision by the
result's type, and waits that run out."""
import numpy as np
import pytest
import torch

import tiled_matrix_multiplication_output_gb300 as tg
from tests.test_gpu_newton_schulz import DT, draw, expect, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    tg.load_library(build_if_missing=True)
    tg.gemm_debug_config(0, -1)


def _status():
    assert tg.gemm_device_status(torch.cuda.current_stream().cuda_stream) == tg.binding.OK


# ------------------------------------------------------------------ batches

@pytest.mark.parametrize("rows,cols", [(40, 96), (1, 17), (150, 137), (300, 130)])
def test_interleaved_and_expanded_batches(rows, cols):
    g = draw(rows, 5 * cols, "f32", "flat", seed=31).cuda().view(rows, 5, cols)
    before = g.clone()
    inter = g.transpose(0, 1)                  # matrix i in the columns from i * cols on
    want = tg.newton_schulz(inter.contiguous())
    assert torch.equal(tg.newton_schulz(inter), want)
    out = torch.full((rows, 5, cols), 7.0, device="cuda")
    tg.newton_schulz(inter.contiguous(), out=out.transpose(0, 1))
    assert torch.equal(out.transpose(0, 1), want)
    tg.newton_schulz(inter, out=inter)         # in place
    assert torch.equal(inter, want)
    one = draw(rows, cols, "bf16", "low rank", seed=32).cuda()
    many = tg.newton_schulz(one.expand(4, rows, cols))
    again = tg.newton_schulz(one.expand(4, rows, cols).contiguous())
    _status()
    assert torch.equal(many, again)
    for i in range(5):
        expect(want[i], before[:, i], "f32")


def test_results_that_share_elements_are_refused():
    g = torch.randn(3, 16, 24, device="cuda")
    with pytest.raises(tg.GemmError):
        tg.newton_schulz(g, out=torch.empty(16, 24, device="cuda").expand(3, 16, 24))
    wide = torch.empty(17, 3 * 24 - 1, device="cuda")
    for store, stride in ((wide, 23), (wide, 25), (torch.empty(46, 24, device="cuda"), 15 * 24)):
        with pytest.raises(tg.GemmError):
            tg.newton_schulz(g, out=store.as_strided((3, 16, 24), (stride, store.shape[1], 1)))
    _status()


# ------------------------------------------------------- waits that run out

@pytest.mark.parametrize("product", [0, 1, 2, 4])
@pytest.mark.parametrize("batch,rows,cols", [(1, 128, 128), (1, 64, 400), (3, 64, 1000), (1, 1000, 64),
                                             (1, 100, 2500)])
def test_nothing_is_stored_after_a_wait_that_runs_out(batch, rows, cols, product):
    """One-launch form: the completion of one product (of six) is not signalled in
    the first block of each cluster.  The other blocks' columns would be made of
    that block's unfinished sums: nobody stores.  The next call is right."""
    g = torch.stack([draw(rows, cols, "f32", "flat", seed=41 + i) for i in range(batch)]).cuda()
    out = torch.full_like(g, 5.0)
    tg.gemm_debug_config(20_000_000, product)
    try:
        tg.newton_schulz(g, steps=2, out=out)
        sh = torch.cuda.current_stream().cuda_stream
        assert tg.gemm_device_status(sh) == tg.binding.ERR_TIMEOUT
    finally:
        tg.gemm_debug_config(0, -1)
    if product == 4:       # the last step's B: only the columns of the first blocks come of it
        tg.newton_schulz(g, steps=2, out=(want := torch.empty_like(g)))
        assert ((out == 5.0) | (out == want)).all() and (out == 5.0).any()
    else:
        assert torch.all(out == 5.0)
    tg.newton_schulz(g, steps=2, out=out)
    _status()
    for i in range(batch):
        expect(out[i], g[i], "f32", steps=2)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("batch,rows,cols", [(1, 200, 1000), (2, 700, 150), (1, 1900, 2300), (1, 256, 256)])
def test_nothing_is_stored_after_a_product_that_did_not_finish(batch, rows, cols, out):
    """Separate launches: the copies of one K step are left out, one that only the
    products over the longer side have (the last: every product)."""
    g = torch.stack([draw(rows, cols, "f32", "flat", seed=45 + i) for i in range(batch)]).cuda()
    res = torch.full_like(g, 5.0, dtype=DT[out])
    tg.gemm_debug_config(20_000_000, (max(rows, cols) - 1) // 64)
    try:
        tg.newton_schulz(g, steps=2, out=res)
        sh = torch.cuda.current_stream().cuda_stream
        assert tg.gemm_device_status(sh) == tg.binding.ERR_TIMEOUT
    finally:
        tg.gemm_debug_config(0, -1)
    assert torch.all(res == 5.0)
    tg.newton_schulz(g, steps=2, out=res)
    _status()
    for i in range(batch):
        expect_stated(res[i], g[i], out, steps=2)


# ------------------------------------------------------------ extreme norms

# one-launch form on one block and on clusters, separate launches
@pytest.mark.parametrize("rows,cols", [(40, 70), (100, 900), (150, 270), (700, 520)])
@pytest.mark.parametrize("dtype,scale", [("f32", 1e21), ("f32", 1e39), ("bf16", 3e38), ("f32", 1e-21),
                                         ("f32", 1e-24), ("bf16", 1e-32), ("f32", 1e-35), ("f32", 1e-38)])
def test_norms_whose_squares_leave_fp32(rows, cols, dtype, scale):
    """Entries of about 1e-2 times the scale: up to a norm near the end of FP32,
    down to values with a few bits left (the definition is of the values given)."""
    g = draw(rows, cols, "f32", "low rank", seed=rows).double()
    norm = float(g.norm())
    g = (g * min(scale, 3.0e38 / norm)).to(torch.float32 if dtype == "f32" else torch.bfloat16).cuda()
    assert torch.isfinite(g).all() and (g != 0).any()
    got = tg.newton_schulz(g, eps=0.0, out_dtype="f32")
    _status()
    expect(got, g, "f32", eps=0.0)
    if scale > 1:                        # eps does not matter, nor do zeros
        g[: rows // 2] = 0
        g[rows // 2 + 1 :] *= 2.0 ** -90
        expect(tg.newton_schulz(g, out_dtype="f32"), g, "f32")
    else:                                # a result that eps makes small
        tiny = tg.newton_schulz(g, eps=1e-7, out_dtype="f32")
        assert torch.isfinite(tiny).all() and float(tiny.abs().max()) < 1e-10


@pytest.mark.parametrize("rows,cols", [(40, 70), (100, 900), (150, 270)])
def test_norms_beyond_fp32_and_one_large_value(rows, cols):
    g = torch.full((2, rows, cols), 3.3e38, device="cuda")
    g[1] = 1e-3
    g[1, rows - 1, cols - 1] = 3.3e38    # the norm is this value
    got = tg.newton_schulz(g)
    _status()
    assert torch.isnan(got[0]).all()     # the norm is infinite in FP32
    expect(got[1], g[1], "f32")


# -------------------------------------------------- precision by the result's type

KINDS = ["flat", "low rank", "decaying"]


def bound(rows, cols, out):
    """What the header states, before the result's own rounding."""
    if out == "bf16" and min(rows, cols) > 128:
        return 2e-3
    return 1e-5 + max(rows, cols) * 2.0 ** -25


def expect_stated(got, g, out, **kw):
    """Within the stated error, and the rounding of the exact result to the type
    (independent of it, so that the two add as squares)."""
    want = reference(g.double().cpu().numpy(), **kw)
    size = np.linalg.norm(want)
    rounding = np.linalg.norm(torch.from_numpy(want).to(DT[out]).double().numpy() - want) / size
    off = np.linalg.norm(got.double().cpu().numpy() - want) / size
    assert off <= np.hypot(bound(*g.shape, out), rounding), f"{off:.2e}, rounding {rounding:.2e}"


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 300), (32, 33), (63, 64), (64, 64), (100, 100), (128, 128),
                                       (129, 129), (200, 1000), (1000, 200), (333, 334), (640, 512)])
def test_results_are_as_exact_as_stated(rows, cols, out, kind):
    g = draw(rows, cols, "f32", kind, seed=rows + 3 * cols).cuda()
    got = tg.newton_schulz(g, out_dtype=out)
    _status()
    expect_stated(got, g, out)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(2048, 700), (1500, 1500), (300, 3001)])
def test_large_results_are_as_exact_as_stated(rows, cols, out):
    """CTA pairs, with one and with two halves an operand."""
    g = draw(rows, cols, "bf16", "flat", seed=51).cuda()
    got = tg.newton_schulz(g, out_dtype=out)
    again = tg.newton_schulz(g, out_dtype=out)
    _status()
    assert torch.equal(got, again)
    expect_stated(got, g, out)


def test_more_steps_and_other_coefficients_in_fp32():
    g = draw(150, 270, "f32", "decaying", seed=52).cuda()
    expect_stated(tg.newton_schulz(g, steps=12, coefficients=(2.0, -1.5, 0.5)), g, "f32", steps=12,
                  abc=(2.0, -1.5, 0.5))
    expect_stated(tg.newton_schulz(g, steps=1), g, "f32", steps=1)
    g = draw(90, 700, "f32", "low rank", seed=53).cuda()
    expect_stated(tg.newton_schulz(g, steps=2), g, "f32", steps=2)
    _status()


# --------------------------------------------- every size of the one-launch form

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [
    (100, 256), (100, 257), (384, 65), (128, 500), (100, 1000), (1000, 100), (128, 2048), (2049, 65),
    (37, 4096),           # 1, 2, 2, 4, 8, 8, 16, 16 and 16 blocks, the last in halves
    (128, 3000), (3500, 128), (4096, 128),
    (90, 1537), (1, 4000),    # 16 blocks of 112 columns, 2 of them without any; a single row
    (4097, 128), (60, 5000)])  # no cluster holds these: separate launches
def test_every_cluster_size(rows, cols, kind):
    g = draw(rows, cols, "f32", kind, seed=rows + cols).cuda()
    got = tg.newton_schulz(g)
    again = tg.newton_schulz(g)
    _status()
    assert torch.equal(got, again)
    expect_stated(got, g, "f32")


@pytest.mark.parametrize("batch,rows,cols", [(9, 64, 2500), (40, 1000, 50), (300, 90, 70), (16, 128, 1024),
                                             (64, 400, 16), (24, 16, 2000), (3, 128, 3900)])
def test_batches_of_clusters(batch, rows, cols):
    """More clusters than fit at a time, some with 256 columns a block, which alone
    they would not have, and the same result wherever in the batch a matrix is."""
    g = torch.stack([draw(rows, cols, "f32", KINDS[i % 3], seed=i) for i in range(batch)]).cuda()
    got = tg.newton_schulz(g, out_dtype="bf16")
    _status()
    assert torch.equal(tg.newton_schulz(g.roll(1, 0), out_dtype="bf16").roll(-1, 0), got)
    for i in sorted({0, 1, batch // 2, batch - 1}):
        expect_stated(got[i], g[i], "bf16")
    x = g.clone()
    assert torch.equal(tg.newton_schulz(x, out=x), tg.newton_schulz(g))     # in place
    _status()


@pytest.mark.parametrize("rows,cols", [(64, 1000), (2049, 65), (128, 3900)])
def test_clusters_with_unaligned_rows(rows, cols):
    store = draw(rows + 2, cols + 5, "bf16", "flat", seed=61).cuda()
    g = store[1:-1, 3:3 + cols]
    out = torch.full((rows, cols + 3), 7.0, device="cuda")
    tg.newton_schulz(g, out=out[:, 1:1 + cols])
    _status()
    expect_stated(out[:, 1:1 + cols], g, "f32")
    assert torch.all(out[:, 0] == 7.0) and torch.all(out[:, 1 + cols:] == 7.0)
