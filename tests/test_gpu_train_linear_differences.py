"""Gradients of the example's 8-bit layer against differences, in random
directions and along the gradient itself."""
import pytest
import torch

from tests.test_gpu_train_linear import example  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def bound(want, scale):
    """The loss sum(y * c) is linear in x and in W, so that a difference over any
    distance differs from the gradient only by quantisation.  Rounding to four
    significant bits is off by at most 2^-4 of an element, by 0.036 of it in the
    mean square (evenly spread), at random.  Of the four roundings involved
    (Q(x +- d) or Q(W +- d), the other operand on either side, Q(c)) each moves the
    scalar by at most 0.036 * scale in the mean square, `scale` being the 2-norm
    of the terms that it is the sum of: 0.072 together, 0.25 is 3.5 times that.
    What rounding does on the average (its error is not quite independent of the
    value: 2^-4 squared of it) is proportional to the scalar: 0.01 of it."""
    return 0.25 * scale + 0.01 * want.abs()


@pytest.mark.parametrize("seed", range(6))
def test_gradients_agree_with_differences_in_any_direction(example, seed):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(100 + seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    x = normal(128, 256).bfloat16().requires_grad_()
    w = normal(192, 256).requires_grad_()
    c = normal(128, 192).bfloat16()
    example.Linear.apply(x, w).backward(c)

    def loss(xv, wv):
        return (example.Linear.apply(xv, wv).double() * c.double()).sum()

    with torch.no_grad():
        of_x, of_w = c.double() @ w.double(), c.double().t() @ x.double()
        for aligned in (False, True):
            dx = (of_x / of_x.square().mean().sqrt()).bfloat16() if aligned else normal(128, 256).bfloat16()
            dw = (of_w / of_w.square().mean().sqrt()).float() if aligned else normal(192, 256)
            for grad, num, d, other in ((x.grad, (loss(x + dx, w) - loss(x - dx, w)) / 2, dx, of_x),
                                        (w.grad, (loss(x, w + dw) - loss(x, w - dw)) / 2, dw, of_w)):
                want = (grad.double() * d.double()).sum()
                scale = (other * d.double()).square().sum().sqrt()
                off = (num - want).abs()
                assert off <= bound(want, scale), f"{aligned}: {float(off / scale):.3f} of the scale"
                if aligned:  # a gradient that is half as large, zero or turned round is far outside
                    assert want > 10 * bound(want, scale)
