"""Low-rank adapters beside a shared projection against their definition in 64
bits: rows of every adapter in any order, every type, ranks, strides, adapters
that are not finite, streams and graphs, and the gradients."""
import pytest
import torch

import tiled_matrix_multiplication_output_gb300 as tg
from tests import routed_reference as ref
from tests.routed_reference import DT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    tg.load_library(build_if_missing=True)
    tg.gemm_debug_config(0, -1)


@pytest.fixture(autouse=True)
def _status():
    yield
    assert tg.gemm_device_status(torch.cuda.current_stream().cuda_stream) == tg.binding.OK


class Case:
    def __init__(self, rows, N, K, G, r, dtype, order="mixed", seed=0, ints=False):
        g = torch.Generator().manual_seed(seed)

        def draw(*shape):
            v = (torch.randint(-2, 3, shape, generator=g).float() if ints
                 else torch.randn(*shape, generator=g))
            return v.to(DT[dtype]).cuda()

        self.x, self.w, self.dy = draw(rows, K), draw(N, K), draw(rows, N)
        self.a, self.b = draw(G, r, K), draw(G, N, r)
        self.scale = (torch.randint(1, 3, (G,), generator=g).float() if ints
                      else torch.rand(G, generator=g) * 2 - 0.5).cuda()
        if order == "mixed":
            of = torch.randint(-1, G, (rows,), generator=g)
        elif order == "runs":
            of = (torch.arange(rows) * (G + 1) // max(rows, 1)) - 1
        elif order == "one":
            of = torch.full((rows,), G - 1)
        else:
            of = torch.full((rows,), -1)
        self.adapter = of.to(torch.int32).cuda()

    def forward(self, **k):
        return tg.matmul_lora(self.x, self.w, self.a, self.b, self.adapter, self.scale, **k)

    def backward(self, **k):
        return tg.matmul_lora_backward(self.dy, self.x, self.w, self.a, self.b, self.adapter,
                                       self.scale, **k)

    def check_forward(self, y):
        ref.check(y, *ref.lora(self.x, self.w, self.a, self.b, self.adapter, self.scale, y.dtype))

    def check_backward(self, got):
        want = ref.lora_backward(self.dy, self.x, self.w, self.a, self.b, self.adapter, self.scale,
                                 got[0].dtype)
        for g, w in zip(got, want):
            ref.check(g, *w)


# rows, N, K, adapters, rank, order of the rows' adapters
SHAPES = [
    (1, 8, 8, 1, 1, "one"), (1, 1000, 2048, 4, 8, "mixed"), (5, 264, 200, 3, 4, "mixed"),
    (64, 256, 512, 64, 16, "mixed"), (33, 77, 99, 2, 5, "mixed"), (130, 384, 72, 7, 64, "mixed"),
    (300, 136, 264, 3, 12, "runs"), (513, 520, 1032, 5, 33, "runs"), (257, 264, 136, 2, 128, "one"),
    (129, 128, 64, 2, 256, "mixed"), (200, 264, 136, 3, 16, "none"), (700, 1000, 40, 40, 8, "runs"),
    (2100, 64, 72, 100, 8, "mixed"), (64, 1000, 328, 30, 24, "mixed"), (1300, 2056, 264, 9, 40, "runs"),
]


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32"), ("bf16", "f32"),
                                       ("f16", "f16")])
@pytest.mark.parametrize("rows,N,K,G,r,order", SHAPES)
def test_lora(rows, N, K, G, r, order, dtype, out):
    c = Case(rows, N, K, G, r, dtype, order)
    y = c.forward(out_dtype=DT[out])
    assert y.dtype == DT[out]
    c.check_forward(y)


@pytest.mark.parametrize("dtype,out,grad", [("bf16", "bf16", "f32"), ("f16", "f32", "f16"), ("f32", "f32", "f32"),
                                            ("bf16", "f32", "bf16")])
@pytest.mark.parametrize("rows,N,K,G,r,order", SHAPES)
def test_lora_backward(rows, N, K, G, r, order, dtype, out, grad):
    c = Case(rows, N, K, G, r, dtype, order)
    got = c.backward(out_dtype=DT[out], grad_dtype=DT[grad])
    assert [t.dtype for t in got] == [DT[out], DT[grad], DT[grad]]
    c.check_backward(got)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,N,K,G,r,order", [(100, 136, 64, 9, 8, "mixed"), (300, 264, 128, 4, 20, "runs")])
def test_lora_is_exact_on_integers(rows, N, K, G, r, order, dtype):
    """Every sum is an integer below 2^24 (and every rank value fits 16 bits)."""
    c = Case(rows, N, K, G, r, dtype, order, ints=True)
    args = (c.x, c.w, c.a, c.b, c.adapter, c.scale)
    assert torch.equal(c.forward().double(), ref.lora(*args, torch.float32)[0])
    for g, w in zip(c.backward(), ref.lora_backward(c.dy, *args, torch.float32)):
        assert torch.equal(g.double(), w[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_row_sees_nothing_of_other_adapters(dtype):
    c = Case(150, 264, 200, 6, 16, dtype)
    y, (dx, da, db) = c.forward(), c.backward()
    c.a[2], c.b[4] = float("nan"), float("inf")
    c.x[7], c.dy[9] = float("inf"), float("nan")
    y2, (dx2, da2, db2) = c.forward(), c.backward()
    of = c.adapter.tolist()
    keep = [i for i in range(150) if of[i] not in (2, 4) and i != 7]
    assert torch.equal(y2[keep], y[keep])
    keep = [i for i in range(150) if of[i] not in (2, 4) and i != 9]
    assert torch.equal(dx2[keep], dx[keep])
    keep = [g for g in range(6) if g not in (2, 4, of[7], of[9])]
    assert keep and torch.equal(da2[keep], da[keep]) and torch.equal(db2[keep], db[keep])
    assert torch.isnan(y2[[i for i in range(150) if of[i] == 2]]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_adapters_out_of_range_are_none(dtype):
    c = Case(200, 136, 72, 4, 8, dtype, "none")
    plain = c.forward()
    c.adapter[:] = torch.tensor([4, 5, -1, -2, 2 ** 31 - 1, -2 ** 31, 1000, 4] * 25, dtype=torch.int32)
    assert torch.equal(c.forward(), plain)
    dx, da, db = c.backward()
    assert (da == 0).all() and (db == 0).all()
    ref.check(dx, *ref.lora_backward(c.dy, c.x, c.w, c.a, c.b, c.adapter, c.scale, torch.float32)[0])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_lora_strides_alignment_and_no_scale(dtype):
    c = Case(150, 264, 400, 5, 24, dtype)
    c.scale = None
    x, w, a, b = c.x, c.w, c.a, c.b
    for k0, r0 in ((0, 0), (8, 8), (3, 1)):
        c.x, c.w, c.a, c.b = x[:, k0:k0 + 304], w[:, k0:k0 + 304], a[:, r0:r0 + 16, k0:k0 + 304], b[:, :, r0:r0 + 16]
        for pitch, c0 in ((264, 0), (272, 8), (267, 1)):
            buf = torch.full((150, pitch + c0), 7.0, device="cuda", dtype=DT[dtype])
            c.check_forward(c.forward(out=buf[:, c0:c0 + 264]))
            assert (buf[:, :c0] == 7).all() and (buf[:, c0 + 264:] == 7).all()
        c.check_backward(c.backward())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lora_empty_sizes(dtype):
    c = Case(0, 24, 16, 2, 4, dtype)
    assert c.forward().shape == (0, 24)
    dx, da, db = c.backward()
    assert dx.shape == (0, 16) and (da == 0).all() and (db == 0).all()
    for G, r in ((0, 4), (2, 0)):
        c = Case(9, 24, 16, G, r, dtype, "none")
        c.adapter[:] = 0
        c.check_forward(c.forward())
        c.check_backward(c.backward())
    c = Case(9, 24, 0, 2, 4, dtype)
    assert (c.forward() == 0).all()
    assert (c.backward()[2] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_against_differences(dtype):
    """The inner product with a direction is the change of <y, dy> along it.  All is
    linear in each operand alone, so that a difference is exact but for roundings."""
    c = Case(90, 136, 72, 3, 8, dtype)
    got = c.backward()

    def loss(x, a, b):
        return (ref.lora(x, c.w, a, b, c.adapter, c.scale, torch.float32)[0] * c.dy.double()).sum()

    for k, name in enumerate(("x", "a", "b")):
        op = {"x": c.x.double(), "a": c.a.double(), "b": c.b.double()}
        step = torch.randn(op[name].shape, generator=torch.Generator().manual_seed(7), dtype=torch.float64).cuda()
        up, down = dict(op), dict(op)
        up[name], down[name] = op[name] + step, op[name] - step
        want = (loss(**up) - loss(**down)) / 2
        bounds = ref.lora_backward(c.dy, c.x, c.w, c.a, c.b, c.adapter, c.scale, torch.float32)[k]
        limit = ((bounds[1] + ref.rounding_bound(bounds[0], torch.float32)) * step.abs()).sum()
        assert abs((got[k].double() * step).sum() - want) <= limit


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lora_repeats_streams_and_graphs(dtype):
    c = Case(300, 264, 256, 6, 16, dtype, "runs")
    adapters = [c.adapter.clone(), c.adapter.flip(0).contiguous(), torch.full_like(c.adapter, -1)]

    def step():
        return c.forward(out_dtype=DT[dtype]), *c.backward()

    first = step()
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.forward(out_dtype=DT[dtype], stream=s), *c.backward(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for of in adapters + adapters[:1]:
        c.adapter.copy_(of)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, step()))
    assert all(torch.equal(a, b) for a, b in zip(first, held))


def test_lora_beyond_32_bit_offsets():
    rows, K = 540_001, 4096
    c = Case(300, 24, K, 3, 8, "bf16", ints=True)
    c.a.clamp_(-1, 1), c.b.clamp_(-1, 1)
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    x[-300:] = c.x
    of = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    of[-300:] = c.adapter
    y = tg.matmul_lora(x, c.w, c.a, c.b, of, c.scale)
    want, bound = ref.lora(c.x, c.w, c.a, c.b, c.adapter, c.scale, torch.float32)
    ref.check(y[-300:], want, bound)
    assert not y[:-300].any()
    dy = torch.zeros(rows, 24, dtype=torch.bfloat16, device="cuda")
    dy[-300:] = c.dy
    dx, da, db = tg.matmul_lora_backward(dy, x, c.w, c.a, c.b, of, c.scale)
    c.check_backward((dx[-300:], da, db))
    assert not dx[:-300].any()


def test_lora_refusals():
    c = Case(6, 24, 16, 2, 4, "bf16")
    args = dict(x=c.x, w=c.w, a=c.a, b=c.b, adapter=c.adapter, scale=c.scale)
    for bad in (dict(x=c.x[:, :8]), dict(a=c.a[0]), dict(b=c.b[:1]), dict(b=c.b[:, :8]),
                dict(adapter=c.adapter[:5]), dict(adapter=c.adapter.cpu()), dict(scale=c.scale[:1]),
                dict(out=c.x), dict(x=c.x.cpu()), dict(a=c.a.transpose(1, 2))):
        with pytest.raises(ValueError):
            tg.matmul_lora(**{**args, **bad})
    for bad in (dict(x=c.x.float()), dict(a=c.a.half()), dict(adapter=c.adapter.long()),
                dict(scale=c.scale.double())):
        with pytest.raises(TypeError):
            tg.matmul_lora(**{**args, **bad})
    with pytest.raises(ValueError):
        tg.matmul_lora_backward(c.dy[:5], **args)
    big = Case(6, 24, 16, 1, 257, "bf16")
    with pytest.raises(tg.GemmError) as e:
        big.forward()
    assert e.value.code == tg.binding.ERR_UNSUPPORTED
