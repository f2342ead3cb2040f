"""Each expert's gradients by themselves, in the layer of examples/train_experts.py,
against 64-bit arithmetic through the same routing: an expert whose gradients are small
beside another's counts as much."""
import pytest
import torch

import tiled_matrix_multiplication_output_gb300 as tg
from tests.routed_reference import DT, sums_bound
from tests.test_gpu_train_experts import example  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status():
    yield
    assert tg.gemm_device_status(torch.cuda.current_stream().cuda_stream) == tg.binding.OK


def reference(layer, x, dy, top, route):
    """(gradients of x, up, down, and elementwise bounds of what the layer's roundings may
    change in them): every step's error is carried on to the next, in magnitudes."""
    half = torch.finfo(x.dtype).eps / 2 + 2.0 ** -21  # (and FP32's exponentials and scores)
    experts, hidden, width = layer.up.shape
    up, down, router = (p.detach().double() for p in (layer.up, layer.down, layer.router))
    rows, offsets, _ = route(x.float() @ layer.router.detach().t(), top)
    ends = offsets.tolist()
    x, dy = x.double(), dy.double()
    p = torch.softmax(x @ router.t(), dim=-1)
    dx, ex = torch.zeros_like(x), torch.zeros_like(x)
    dp, ep = torch.zeros_like(p), torch.zeros_like(p)
    du, eu, dd, ed = (torch.zeros_like(t) for t in (up, up, down, down))

    def product(a, ea, b):  # of a with an error and an exact b, rounded: (value, error)
        v, mag = a @ b, (a.abs() + ea) @ b.abs()
        return v, ea @ b.abs() + half * (v.abs() + ea @ b.abs()) + sums_bound(a.shape[1]) * mag

    for g, (b, e) in enumerate(zip(ends, ends[1:])):
        if e == b:
            continue
        mine = rows[b:e]
        xg, s = x[mine], p[mine, g][:, None]
        pre, e_pre = product(xg, torch.zeros_like(xg), up[g].t())
        sig = torch.sigmoid(pre)
        a, slope = pre * sig, sig * (1 + pre * (1 - sig))
        e_a = 1.1 * e_pre + half * (a.abs() + 1.1 * e_pre)  # |silu'| < 1.1
        y, e_y = product(a, e_a, down[g].t())
        dg = s * dy[mine]
        e_dg = half * dg.abs()
        da, e_da = product(dg, e_dg, down[g])
        dpre = da * slope
        e_dpre = slope.abs() * e_da + 0.5 * (da.abs() + e_da) * e_pre  # |silu''| <= 0.5
        e_dpre += half * (dpre.abs() + e_dpre)
        dd[g], du[g] = dg.t() @ a, dpre.t() @ xg
        n = sums_bound(e - b)
        ed[g] = (dg.abs() + e_dg).t() @ (e_a + n * a.abs()) + e_dg.t() @ a.abs()
        eu[g] = (e_dpre + n * (dpre.abs() + e_dpre)).t() @ xg.abs()
        ed[g] += half * (dd[g].abs() + ed[g])
        eu[g] += half * (du[g].abs() + eu[g])
        dxg, e_dxg = product(dpre, e_dpre, up[g])
        dx.index_add_(0, mine, dxg)
        # (a token's copies are added in the type: a rounding for each, of all so far)
        ex.index_add_(0, mine, e_dxg + (top + 1) * half * (dxg.abs() + e_dxg))
        dp[mine, g] = (dy[mine] * y).sum(1)
        ep[mine, g] = (dy[mine].abs() * (e_y + sums_bound(width) * y.abs())).sum(1)
    # the scores' way back to x: the softmax's and the router's, in FP32, then one rounding
    mean = (p * dp).sum(1, True)
    ds = p * (dp - mean)
    e_ds = p * (ep + (p * ep).sum(1, True)) + 2.0 ** -18 * p * (dp.abs() + (p * dp.abs()).sum(1, True))
    dxr, e_dxr = ds @ router, e_ds @ router.abs()
    total = dx + dxr
    ex += e_dxr + half * (dxr.abs() + e_dxr)
    ex += half * (total.abs() + ex)
    return (total, ex), (du, eu), (dd, ed)


CASES = [(70, 64, 136, 5, 2), (1, 40, 24, 3, 3), (300, 136, 72, 16, 1)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,width,hidden,experts,top", CASES)
def test_each_experts_gradients(example, tokens, width, hidden, experts, top, dtype):  # noqa: F811
    torch.manual_seed(tokens)
    layer = example.ExpertLayer(experts, width, hidden, top, DT[dtype])
    with torch.no_grad():  # gradients of a hundredth and less beside ordinary ones
        layer.down[0] *= 0.01
        layer.up[-1] *= 0.1
    x = torch.randn(tokens, width, device="cuda").to(DT[dtype]).requires_grad_()
    dy = torch.randn(tokens, width, device="cuda").to(DT[dtype])
    layer(x).backward(dy)
    want = reference(layer, x.detach(), dy, top, example.route)
    for got, (ref, bound) in zip((x.grad, layer.up.grad, layer.down.grad), want):
        assert got.dtype == DT[dtype]
        assert ((got.double() - ref).abs() <= bound + torch.finfo(DT[dtype]).smallest_normal).all()
    # In the norm a gradient's roundings do not add up faster than its terms, as both have any
    # sign: seven in a row, each by its most, and FP32 sums
    limit = 7 * torch.finfo(DT[dtype]).eps / 2 + 2.0 ** -14
    for got, (ref, _) in zip((layer.up.grad, layer.down.grad), want[1:]):
        for g in range(experts):
            assert (got[g].double() - ref[g]).norm() <= limit * ref[g].norm()
    # x's: one more product, its copies' sum and the router's part
    limit = (9 + top) * torch.finfo(DT[dtype]).eps / 2 + 2.0 ** -14
    assert (x.grad.double() - want[0][0]).norm() <= limit * want[0][0].norm()
