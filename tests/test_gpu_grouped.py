"""Products grouped by rows and their weight gradient against their definitions
in 64 bits: ragged and empty groups, every type and form, strides, values that
are not finite, offsets that make no sense, streams and graphs."""
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


def _randn(seed, dtype, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(DT[dtype]).cuda()


def _ints(seed, dtype, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-3, 4, shape, generator=g).to(DT[dtype]).cuda()


def _offsets(counts, first=0):
    out = [first]
    for n in counts:
        out.append(out[-1] + n)
    return out


def _dev(offsets):
    return torch.tensor(offsets, dtype=torch.int32, device="cuda")


# rows of each group, rows behind the last, N, K
SHAPES = [
    ([1], 0, 8, 8), ([3, 0, 1, 5], 0, 128, 64), ([0, 0, 7], 2, 264, 200), ([130, 31, 0, 257], 5, 256, 72),
    ([32, 64, 96, 128], 0, 384, 128), ([300, 1, 1, 1], 0, 136, 520), ([0, 0], 4, 64, 64),
    ([255, 256, 257], 1, 512, 136), ([5, 6], 0, 1, 1), ([33, 2], 0, 77, 99), ([700], 0, 1000, 24),
]


@pytest.mark.parametrize("op", ["t", "n"])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32"),
                                       ("bf16", "f16"), ("f32", "bf16")])
@pytest.mark.parametrize("counts,rest,N,K", SHAPES)
def test_grouped(counts, rest, N, K, dtype, out, op):
    off = _offsets(counts)
    x = _randn(1, dtype, off[-1] + rest, K)
    w = _randn(2, dtype, len(counts), *((N, K) if op == "t" else (K, N)))
    y = tg.matmul_grouped(x, w, _dev(off), op_b=op, out_dtype=DT[out])
    want, bound, _ = ref.grouped(x, w, off, op == "t")
    assert y.dtype == DT[out]
    ref.check(y, want, bound)  # rows of no group: zeros


@pytest.mark.parametrize("op", ["t", "n"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_grouped_is_exact_on_integers(dtype, op):
    """Every partial sum is an integer below 2^24."""
    for seed, (counts, N, K) in enumerate([([17, 0, 260, 40, 3], 328, 456), ([512, 511], 256, 1000),
                                           ([1] * 40, 128, 2048)]):
        off = _offsets(counts)
        x = _ints(seed, dtype, off[-1], K)
        w = _ints(seed + 9, dtype, len(counts), *((N, K) if op == "t" else (K, N)))
        y = tg.matmul_grouped(x, w, _dev(off), op_b=op)
        assert torch.equal(y.double(), ref.grouped(x, w, off, op == "t")[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_grouped_alpha_beta_and_rows_of_no_group(dtype):
    off = _offsets([40, 0, 90], first=6)
    rows = off[-1] + 11
    x, w = _randn(3, dtype, rows, 128), _randn(4, dtype, 3, 192, 128)
    x[:6] = float("nan")  # rows of no group are not read
    x[off[-1]:] = float("inf")
    for beta in (0.0, 0.5):
        y0 = _randn(5, "f32", rows, 192)
        if beta == 0.0:
            y0[6:off[-1]] = float("nan")  # nor is the output
        y = tg.matmul_grouped(x, w, _dev(off), out=y0.clone(), alpha=-1.5, beta=beta)
        want, bound, mine = ref.grouped(x, w, off, True, -1.5, beta, y0)
        ref.check(y[mine], want[mine], bound[mine])
        assert torch.equal(y[~mine], y0[~mine])
    y = tg.matmul_grouped(x, w, _dev(off))
    assert torch.equal(y[~mine], torch.zeros_like(y[~mine]))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("op", ["t", "n"])
def test_grouped_strides_and_alignment(dtype, op):
    off = _offsets([70, 3, 0, 150])
    big_x = _randn(6, dtype, 260, 700)
    big_w = _randn(7, dtype, 4, 330, 420)
    for x0, k0, n0 in ((0, 0, 0), (8, 16, 24), (1, 3, 5), (0, 1, 0)):
        K, N = 200, 136
        x = big_x[2:225, x0:x0 + K]
        w = (big_w[:, n0:n0 + N, k0:k0 + K] if op == "t" else big_w[:, k0:k0 + K, n0:n0 + N])
        for pitch, c0 in ((N, 0), (N + 8, 8), (N + 3, 1)):
            buf = torch.full((223, pitch + c0), 7.0, device="cuda", dtype=DT[dtype])
            out = buf[:, c0:c0 + N]
            tg.matmul_grouped(x, w, _dev(off), op_b=op, out=out)
            want, bound, _ = ref.grouped(x, w, off, op == "t")
            ref.check(out, want, bound)
            assert (buf[:, :c0] == 7).all() and (buf[:, c0 + N:] == 7).all()
    # one matrix for every group, and interleaved ones
    w = _randn(8, dtype, 136, 200).expand(4, 136, 200)
    w = w if op == "t" else w.transpose(1, 2).contiguous()[:1].expand(4, 200, 136)
    x = big_x[:223, :200]
    want, bound, _ = ref.grouped(x, w, off, op == "t")
    ref.check(tg.matmul_grouped(x, w, _dev(off), op_b=op), want, bound)
    w = _randn(8, dtype, *((136, 4, 200) if op == "t" else (200, 4, 136))).transpose(0, 1)
    want, bound, _ = ref.grouped(x, w, off, op == "t")
    ref.check(tg.matmul_grouped(x, w, _dev(off), op_b=op), want, bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_grouped_values_that_are_not_finite_stay_in_their_rows(dtype):
    off = _offsets([20, 37, 9])
    x, w = _randn(9, dtype, 66, 96), _randn(10, dtype, 3, 160, 96)
    clean = tg.matmul_grouped(x, w, _dev(off))
    x[5, 3], x[40, 0] = float("nan"), float("inf")
    w[2] = float("nan")
    y = tg.matmul_grouped(x, w, _dev(off))
    assert torch.isnan(y[5]).all() and torch.isnan(y[57:]).all()
    assert not torch.isfinite(y[40]).any()
    keep = [i for i in range(57) if i not in (5, 40)]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offsets", [[5, 2, 9, 4], [-7, 3, 3, 1000], [10, 5, 200, 100], [90, 91, 92, 93],
                                     [0, 2 ** 31 - 1, -2 ** 31, 7]])
def test_offsets_that_make_no_sense_stay_in_bounds(dtype, offsets):
    x, w = _ints(11, dtype, 60, 64), _ints(12, dtype, 3, 72, 64)
    buf = torch.full((200, 72), 5.0, device="cuda")
    y = tg.matmul_grouped(x, w, _dev(offsets), out=buf[70:130])
    want, _, mine = ref.grouped(x, w, offsets, True)
    assert torch.equal(y[mine].double(), want[mine]) and (y[~mine] == 5).all()
    assert (buf[:70] == 5).all() and (buf[130:] == 5).all()
    z = tg.matmul_grouped(x, w, _dev(offsets))
    assert torch.equal(z.double(), want)
    dw = tg.matmul_grouped_wgrad(y.to(DT[dtype]), x, _dev(offsets))
    assert torch.equal(dw.double(), ref.wgrad(y.to(DT[dtype]), x, offsets)[0])


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32")])
def test_grouped_empty_sizes(dtype, out):
    off = _dev([0, 2, 5])
    w = _randn(1, dtype, 2, 16, 8)
    assert tg.matmul_grouped(_randn(1, dtype, 0, 8), w, _dev([0, 0, 0])).shape == (0, 16)
    assert tg.matmul_grouped(_randn(1, dtype, 5, 8), w[:, :0], off).shape == (5, 0)
    assert (tg.matmul_grouped(_randn(1, dtype, 5, 0), w[:, :, :0], off, out_dtype=DT[out]) == 0).all()
    y = torch.ones(5, 16, device="cuda")
    tg.matmul_grouped(_randn(1, dtype, 5, 0), w[:, :, :0], off, out=y, beta=2.0)
    assert (y == 2).all()
    assert (tg.matmul_grouped(_randn(1, dtype, 5, 8), w[:0], _dev([0])) == 0).all()
    c = tg.matmul_grouped_wgrad(_randn(1, dtype, 0, 16), _randn(1, dtype, 0, 8), _dev([0, 0, 0]))
    assert c.shape == (2, 16, 8) and (c == 0).all()
    assert tg.matmul_grouped_wgrad(_randn(1, dtype, 4, 16), _randn(1, dtype, 4, 8), _dev([0])).shape == (0, 16, 8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_most_groups(dtype):
    G = 1024
    counts = [(i * 7) % 4 for i in range(G)]
    off = _offsets(counts)
    x, w = _ints(13, dtype, off[-1], 64), _ints(14, dtype, G, 40, 64)
    y = tg.matmul_grouped(x, w, _dev(off))
    assert torch.equal(y.double(), ref.grouped(x, w, off, True)[0])
    c = tg.matmul_grouped_wgrad(y.to(DT[dtype]), x, _dev(off))
    assert torch.equal(c.double(), ref.wgrad(y.to(DT[dtype]), x, off)[0])
    with pytest.raises(tg.GemmError) as e:
        tg.matmul_grouped(x, w[:1].expand(G + 1, 40, 64), torch.zeros(G + 2, dtype=torch.int32, device="cuda"))
    assert e.value.code == tg.binding.ERR_UNSUPPORTED


@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("counts,rest,N,K", SHAPES + [([1000, 17, 63, 64, 65], 9, 264, 264)])
def test_wgrad(counts, rest, N, K, dtype, out):
    off = _offsets(counts)
    dy, x = _randn(15, dtype, off[-1] + rest, N), _randn(16, dtype, off[-1] + rest, K)
    c = tg.matmul_grouped_wgrad(dy, x, _dev(off), out_dtype=DT[out])
    ref.check(c, *ref.wgrad(dy, x, off))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_wgrad_strides_accumulation_and_rest(dtype):
    off = _offsets([70, 0, 3, 129], first=5)
    base = _randn(17, dtype, 230, 900)
    base[:5], base[off[-1]:] = float("nan"), float("inf")  # rows of no group
    for d0, x0 in ((0, 400), (8, 408), (3, 401)):
        dy, x = base[:, d0:d0 + 264], base[:, x0:x0 + 200]
        for out in ("f32", dtype):
            for shape, cut in (((4, 264, 200), slice(0, 200)), ((4, 270, 211), slice(3, 203))):
                c0 = _randn(18, out, *shape)
                c = c0.clone()
                view = c[:, :264, cut]
                tg.matmul_grouped_wgrad(dy, x, _dev(off), out=view, alpha=0.5, beta=1.0)
                ref.check(view, *ref.wgrad(dy, x, off, 0.5, 1.0, c0[:, :264, cut]))
                c[:, :264, cut] = c0[:, :264, cut]
                assert torch.equal(c, c0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_wgrad_values_that_are_not_finite_stay_in_their_group(dtype):
    off = _offsets([20, 37, 9, 70])
    dy, x = _randn(19, dtype, 136, 136), _randn(20, dtype, 136, 264)
    clean = tg.matmul_grouped_wgrad(dy, x, _dev(off))
    dy[21], x[56] = float("inf"), float("nan")
    c = tg.matmul_grouped_wgrad(dy, x, _dev(off))
    for g in (0, 2, 3):
        assert torch.equal(c[g], clean[g])
    assert torch.isnan(c[1]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_grouped_repeats_streams_and_graphs(dtype):
    """The same bits on another stream and from a captured graph whose offsets
    change between replays."""
    off = _offsets([100, 0, 57, 300])
    other = _offsets([0, 457, 0, 0])
    x, w, dy = _randn(21, dtype, 457, 256), _randn(22, dtype, 4, 264, 256), _randn(23, dtype, 457, 264)
    o = _dev(off)

    def step():
        return tg.matmul_grouped(x, w, o, out_dtype=DT[dtype]), tg.matmul_grouped_wgrad(dy, x, o)

    first = [t.clone() for t in step()]
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = (tg.matmul_grouped(x, w, o, out_dtype=DT[dtype], stream=s),
           tg.matmul_grouped_wgrad(dy, x, o, stream=s))
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for offsets in (off, other, off):
        o.copy_(_dev(offsets))
        graph.replay()
        torch.cuda.synchronize()
        eager = step()
        assert all(torch.equal(a, b) for a, b in zip(held, eager))
    assert all(torch.equal(a, b) for a, b in zip(first, held))


def test_grouped_beyond_32_bit_offsets():
    rows, K = 540_001, 4096  # 2.2e9 elements
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    x[-300:] = _ints(24, "bf16", 300, K)
    w = _ints(25, "bf16", 3, 24, K)
    off = [0, rows - 300, rows - 100, rows]
    y = tg.matmul_grouped(x, w, _dev(off))
    want = ref.grouped(x[-300:], w[1:], [0, 200, 300], True)[0]
    assert torch.equal(y[-300:].double(), want) and not y[:-300].any()
    dy = y[-300:].clamp(-8, 8).to(torch.bfloat16)
    full = torch.zeros(rows, 24, dtype=torch.bfloat16, device="cuda")
    full[-300:] = dy
    c = tg.matmul_grouped_wgrad(full, x, _dev(off))
    assert torch.equal(c[1:].double(), ref.wgrad(dy, x[-300:], [0, 200, 300])[0])
    assert not c[0].any()


def test_grouped_refusals():
    x, w, o = _randn(1, "bf16", 6, 16), _randn(2, "bf16", 2, 24, 16), _dev([0, 3, 6])
    for bad in (dict(x=x[:, :8]), dict(w=w[0]), dict(offsets=o[:2]), dict(op_b="x"),
                dict(beta=1.0), dict(out=x), dict(offsets=o.cpu()), dict(x=x.cpu()),
                dict(x=x.t()[:16, :].contiguous().t()), dict(offsets=_dev([0, 0, 3, 3, 6, 6])[::2])):
        with pytest.raises(ValueError):
            tg.matmul_grouped(**{"x": x, "w": w, "offsets": o, **bad})
    for bad in (dict(x=x.float()), dict(offsets=o.long()), dict(x=x.double(), w=w.double())):
        with pytest.raises(TypeError):
            tg.matmul_grouped(**{"x": x, "w": w, "offsets": o, **bad})
    dy = _randn(3, "bf16", 6, 24)
    for bad in (dict(dy=dy[:5]), dict(offsets=o[:0]), dict(beta=1.0), dict(out=w[:1])):
        with pytest.raises(ValueError):
            tg.matmul_grouped_wgrad(**{"x": x, "dy": dy, "offsets": o, **bad})
    with pytest.raises(TypeError):
        tg.matmul_grouped_wgrad(dy.half(), x, o)
    with pytest.raises(tg.GemmError):  # overlapping results
        tg.matmul_grouped_wgrad(dy, x, o, out=torch.zeros(1, 24, 16, device="cuda").expand(2, 24, 16))
