"""Newton-Schulz orthogonalisation, further forms: batches that are not
stacked, every size of the one-launch form, extreme norms, precision by the
result's type, and waits that run out."""
import pytest
import torch

import tiled_matrix_multiplication_output_gb300 as tg
from tests.test_gpu_newton_schulz import draw, expect

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
