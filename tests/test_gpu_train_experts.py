"""The grouped products and the adapters together, as examples/train_experts.py
uses them: a routed layer's and an adapted layer's gradients against those of
64-bit arithmetic on the same operands, and the program's run."""
import importlib.util
import os

import pytest
import torch

import tiled_matrix_multiplication_output_gb300 as tg
from tests.routed_reference import DT

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    tg.load_library(build_if_missing=True)
    tg.gemm_debug_config(0, -1)
    spec = importlib.util.spec_from_file_location(
        "train_experts", os.path.join(ROOT, "examples", "train_experts.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,width,hidden,experts,top", [(70, 64, 136, 5, 2), (1, 40, 24, 3, 3),
                                                             (300, 136, 72, 16, 1)])
def test_experts_gradients(example, tokens, width, hidden, experts, top, dtype):
    """Against autograd in 64 bits through the same routing.  Every step of the layer
    rounds to the type once (five in a row at most, forward and backward), so a
    gradient's error is within ten half steps of the largest magnitudes it is summed
    from; the bound takes the largest gradient's magnitude for those, times
    sqrt of the hidden width that they are spread over."""
    torch.manual_seed(tokens)
    layer = example.ExpertLayer(experts, width, hidden, top, DT[dtype])
    x = torch.randn(tokens, width, device="cuda").to(DT[dtype]).requires_grad_()
    dy = torch.randn(tokens, width, device="cuda").to(DT[dtype])
    layer(x).backward(dy)
    rows, offsets, _ = example.route(x.detach().float() @ layer.router.detach().t(), top)
    ends = offsets.tolist()

    xd = x.detach().double().requires_grad_()
    up, down = (p.detach().double().requires_grad_() for p in (layer.up, layer.down))
    scores = torch.softmax(xd @ layer.router.detach().double().t(), dim=-1)
    out = torch.zeros(tokens, width, dtype=torch.float64, device="cuda")
    for g, (b, e) in enumerate(zip(ends, ends[1:])):
        if e > b:
            mine = rows[b:e]
            y = torch.nn.functional.silu(xd[mine] @ up[g].t()) @ down[g].t()
            out = out.index_add(0, mine, scores[mine, g][:, None] * y)
    out.backward(dy.double())
    half = torch.finfo(DT[dtype]).eps / 2
    for got, want in ((x.grad, xd.grad), (layer.up.grad, up.grad), (layer.down.grad, down.grad)):
        assert got.dtype == DT[dtype]
        limit = 10 * half * want.abs().max() * hidden ** 0.5
        assert ((got.double() - want).abs() <= limit).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_adapted_layer_behind_experts(example, dtype):
    """Both layers in one graph: the adapters' gradients through the experts, against
    the same graph with the adapted layer in 64 bits (its operands and the gradient
    that reaches it are the same, so that only its own sums and roundings differ)."""
    torch.manual_seed(3)
    w = (torch.randn(72, 64, device="cuda") / 8).to(DT[dtype])
    adapted = example.AdapterLayer(w, 4, 8, DT[dtype])
    with torch.no_grad():
        adapted.b.copy_(torch.randn_like(adapted.b))
    moe = example.ExpertLayer(6, 72, 40, 2, DT[dtype])
    x = torch.randn(130, 64, device="cuda").to(DT[dtype]).requires_grad_()
    task = torch.randint(-1, 4, (130,), device="cuda", dtype=torch.int32)
    y = adapted(x, task)
    y.retain_grad()
    moe(y).square().mean().backward()
    xd, a, b = (t.detach().double().requires_grad_() for t in (x, adapted.a, adapted.b))
    yd = xd @ w.double().t()
    for g in range(4):
        rows = torch.nonzero(task == g)[:, 0]
        yd = yd.index_add(0, rows, 2.0 * xd[rows] @ a[g].t() @ b[g].t())
    yd.backward(y.grad.double())
    half = torch.finfo(DT[dtype]).eps / 2
    for got, want in ((x.grad, xd.grad), (adapted.a.grad, a.grad), (adapted.b.grad, b.grad)):
        assert want.abs().max() > 0
        # one rounding, and FP32 sums (and rank values in 24 bits) of up to 130 terms
        limit = half * want.abs() + 2.0 ** -14 * want.abs().max()
        assert ((got.double() - want).abs() <= limit).all()


def test_the_program_runs(example):
    losses = example.train(steps=4, tokens=200, width=64, experts=4, tasks=3, rank=8, log=lambda s: None)
    assert len(losses) == 4 and all(torch.isfinite(torch.tensor(losses)))
