"""The operators together, as examples/train_linear.py uses them: gradients of
a layer against those of its dequantised operands and against differences,
and a short training run."""
import importlib.util
import os

import pytest
import torch

import tiled_matrix_multiplication_output_gb300 as tg
from tests.helpers import HALF_ULP

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    tg.load_library(build_if_missing=True)
    spec = importlib.util.spec_from_file_location(
        "train_linear", os.path.join(ROOT, "examples", "train_linear.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _dequant(q, s, block):
    s = s.t() if block == "row" else s
    s = s if block == "row" else s.repeat_interleave(128, 0)
    s = s if block == "col" else s.repeat_interleave(128, 1)
    return q.double() * s[:q.shape[0], :q.shape[1]].double()


@pytest.mark.parametrize("tokens,width,out", [(96, 200, 136), (300, 257, 129), (1, 64, 40)])
def test_gradients_are_the_formulas(example, tokens, width, out):
    """dx = dy W and dW = dy^T x on the quantised operands.  Tolerances: FP32
    sums of at most 300 terms (2^-14 of the magnitudes leaves a factor of
    ten), and half an ulp of BF16 for y and dx."""
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x = torch.randn(tokens, width, generator=g, device="cuda").bfloat16().requires_grad_()
    w = torch.randn(out, width, generator=g, device="cuda").requires_grad_()
    dy = torch.randn(tokens, out, generator=g, device="cuda").bfloat16()
    y = example.Linear.apply(x, w)
    y.backward(dy)
    (xq, xs), (xtq, xts) = tg.quantize_fp8_pair(x.detach())
    (dq, ds), (dtq, dts) = tg.quantize_fp8_pair(dy)
    wq, ws = tg.quantize_fp8(w.detach(), block="tile")
    W = _dequant(wq, ws, "tile")
    for got, left, right, half in (
            (y, _dequant(xq, xs, "row"), W.t(), HALF_ULP[torch.bfloat16]),
            (x.grad, _dequant(dq, ds, "row"), W, HALF_ULP[torch.bfloat16]),
            (w.grad, _dequant(dtq, dts, "col").t(), _dequant(xtq, xts, "col"), 0.0)):
        want, size = left @ right, left.abs() @ right.abs()
        err = (got.double() - want).abs()
        assert (err <= 2.0 ** -14 * size + half * want.abs()).all()


def test_gradients_agree_with_differences(example):
    """The loss sum(y * c) is linear in x and W, so a difference over any
    distance is exact but for quantisation: each product's operands are
    rounded to 4 significant bits, relative error at most 2^-4, so along a
    direction d the two sides differ by at most 2 * (2^-4 + 2^-4) of the
    terms' magnitudes (both operands, both sides); random signs make it far
    less, and 2^-4 of the magnitudes' 2-norm is asked here."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(128, 256, generator=g, device="cuda").bfloat16().requires_grad_()
    w = torch.randn(192, 256, generator=g, device="cuda").requires_grad_()
    c = torch.randn(128, 192, generator=g, device="cuda").bfloat16()
    example.Linear.apply(x, w).backward(c)

    def loss(xv, wv):
        return (example.Linear.apply(xv, wv).double() * c.double()).sum()

    with torch.no_grad():
        dx = torch.randn(128, 256, generator=g, device="cuda").bfloat16()
        dw = torch.randn(192, 256, generator=g, device="cuda")
        for ana, num, d, other in (
                (x.grad, loss(x + dx, w) - loss(x - dx, w), dx, c.double() @ w.double()),
                (w.grad, loss(x, w + dw) - loss(x, w - dw), dw, c.double().t() @ x.double())):
            want = (ana.double() * d.double()).sum()
            scale = (other.square() * d.double().square()).sum().sqrt()
            assert (num / 2 - want).abs() <= 2.0 ** -4 * 16 * scale


def test_the_layer_learns(example):
    losses = example.train(steps=40, tokens=512, width=256, hidden=256)
    assert all(torch.isfinite(torch.tensor(losses)))
    assert losses[-1] < 0.2 * losses[0]
