"""The grouped products and the adapters at the limits of their sizes, waits and
ranges: groups of nearly 2^31 rows, waits behind long sums, sums of one sign, FP16
values far from one."""
import pytest
import torch

import tiled_matrix_multiplication_output_gb300 as tg
from tests import routed_reference as ref
from tests.test_gpu_grouped import _dev, _ints, _offsets
from tests.test_gpu_lora import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    tg.load_library(build_if_missing=True)


@pytest.fixture(autouse=True)
def _restore():
    tg.gemm_debug_config(0, -1)
    yield
    tg.gemm_debug_config(0, -1)
    assert tg.gemm_device_status(torch.cuda.current_stream().cuda_stream) == tg.binding.OK


@pytest.mark.parametrize("op", ["t", "n"])
def test_a_group_of_the_most_rows(op):
    """One group of GEMM_MAX_DIM rows: the rows and the tiles that they give do not fit
    32 bits together."""
    rows = tg.binding.MAX_DIM
    blocks = rows // 256
    x = torch.empty(rows, 8, dtype=torch.bfloat16, device="cuda")
    x.view(blocks, 256, 8).copy_(_ints(1, "bf16", 256, 8))
    x.view(blocks, 256, 8)[:, :, 0] = (torch.arange(blocks, device="cuda") % 61 - 30)[:, None]
    w = _ints(2, "bf16", 1, 8, 8)
    y = tg.matmul_grouped(x, w, _dev([0, rows]), op_b=op, out_dtype=torch.bfloat16)
    m = (w[0].t() if op == "t" else w[0]).float()
    for r in range(0, rows, 1 << 25):
        assert torch.equal(y[r:r + (1 << 25)].float(), (x[r:r + (1 << 25)].float() @ m).bfloat16().float())


@pytest.mark.parametrize("counts", [[64 * 40_000 + 5], [64 * 10_000] * 76 + [5, 3]])
def test_wgrad_waits_behind_long_sums(counts):
    """The warp that zeroes the rows behind a ragged end waits for it through all K steps
    before, of its tile and of the even ones that its pair had before: ten times as long
    as a wait may be (0.5 and 1 ms here) while nothing moves."""
    rows = sum(counts)
    dy, x = (torch.ones(rows, 8, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    off = _dev([0] + torch.tensor(counts).cumsum(0).tolist())
    tg.gemm_debug_config(1_000_000 if len(counts) == 1 else 2_000_000, -1)
    c = tg.matmul_grouped_wgrad(dy, x, off)
    assert tg.gemm_device_status(torch.cuda.current_stream().cuda_stream) == tg.binding.OK
    assert torch.equal(c, torch.tensor(counts, dtype=torch.float32, device="cuda")[:, None, None].expand_as(c))


def test_adapter_gradients_wait_behind_long_sums():
    """The warps that zero other adapters' rows in the last row tile, and the epilogue, wait
    for it through ten thousand whole ones (0.5 ms a wait here)."""
    rows = 128 * 10_000 + 5
    dy, x = (torch.ones(rows, 8, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w, a, b = (torch.ones(s, dtype=torch.bfloat16, device="cuda") for s in ((8, 8), (1, 8, 8), (1, 8, 8)))
    adapter = torch.zeros(rows, dtype=torch.int32, device="cuda")
    tg.gemm_debug_config(1_000_000, -1)
    _, da, db = tg.matmul_lora_backward(dy, x, w, a, b, adapter)
    assert tg.gemm_device_status(torch.cuda.current_stream().cuda_stream) == tg.binding.OK
    assert (da == 8 * rows).all() and (db == 8 * rows).all()


@pytest.mark.parametrize("rank", [8, 24])
def test_bf16_gradients_do_not_depend_on_the_other_results_types(rank):
    """BF16 gradients have the same bits beside a BF16 dx as beside an FP32 one: rank values
    of 16 bits would move about one in 300 of them over its rounding's border."""
    c = Case(12, 1000, 1032, 2, rank, "bf16")
    wide = c.backward(out_dtype=torch.float32, grad_dtype=torch.bfloat16)
    narrow = c.backward(out_dtype=torch.bfloat16, grad_dtype=torch.bfloat16)
    assert torch.equal(wide[0].bfloat16(), narrow[0])
    assert torch.equal(wide[1], narrow[1]) and torch.equal(wide[2], narrow[2])


def _positive(seed, dtype, *shape):
    g = torch.Generator().manual_seed(seed)
    return (0.25 + torch.rand(*shape, generator=g)).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rank", [16, 32, 48, 64, 72, 128, 256])
def test_adapter_gradients_of_long_sums_keep_fp32(rank, dtype):
    """Sums over 8000 rows of one sign, for every number of accumulators.  A matrix
    instruction drops less than a unit in the last place (2^-23), and an accumulator takes 48
    of them: 96 half units (2^-24) at most; eleven segments of three parts are added
    with a rounding each: 33; a rank value is four instructions, a rounding for the scale
    and one for the parts: 10.  One accumulator for all rows would drop up to 1000."""
    x, dy = _positive(1, dtype, 8000, 64), _positive(2, dtype, 8000, 64)
    a, b = _positive(3, dtype, 2, rank, 64), _positive(4, dtype, 2, 64, rank)
    adapter = torch.zeros(8000, dtype=torch.int32, device="cuda")
    _, da, db = tg.matmul_lora_backward(dy, x, x[:64], a, b, adapter)
    u, t = dy.double() @ b[0].double(), x.double() @ a[0].double().t()
    for got, want in ((da, u.t() @ x.double()), (db, dy.double().t() @ t)):
        assert ((got[0].double() - want).abs() <= 140 * 2.0 ** -24 * want).all()
        assert not got[1].any()


@pytest.mark.parametrize("rows,N,K,G,order", [(20, 136, 264, 3, "mixed"), (100, 264, 520, 90, "mixed"),
                                              (300, 1000, 264, 3, "runs"), (1300, 2056, 264, 9, "mixed"),
                                              (130, 40008, 72, 2, "mixed")])
@pytest.mark.parametrize("rank", [4, 16, 40, 128])
@pytest.mark.parametrize("size", [1e-4, 1e-2, 1.0, 300.0, 20000.0])
def test_fp16_products_with_rank_values_of_any_size(rows, N, K, G, order, rank, size):
    """Rank values from 1e-8 to 1e9, far below FP16's least step and above its largest
    value, in every form of the product and its input's gradient: rank values keep 24 bits
    (the bound is that of BF16 operands, with no absolute term)."""
    c = Case(rows, N, K, G, rank, "f16", order, seed=rank)
    small = min(size, 1.0)
    for t, by in ((c.x, size), (c.dy, size), (c.w, small), (c.a, min(size, 300.0)), (c.b, min(size, 300.0))):
        t.copy_((t.float() * by).clamp(-60000, 60000))
    y, dx = c.forward(), c.backward()[0]
    x, dy, w, a, b = (t.double() for t in (c.x, c.dy, c.w, c.a, c.b))
    full = (torch.bfloat16, torch.float32)
    ref.check(y, *ref._beside(x, w.t(), a, b.transpose(1, 2), c.adapter, c.scale, *full))
    ref.check(dx, *ref._beside(dy, w, b.transpose(1, 2), a, c.adapter, c.scale, *full))
    if size == 1.0:
        half = c.forward(out_dtype=torch.float16)
        ref.check(half, *ref._beside(x, w.t(), a, b.transpose(1, 2), c.adapter, c.scale, *full))


@pytest.mark.parametrize("rank", [4, 16, 40, 128])
@pytest.mark.parametrize("order", ["mixed", "runs"])
@pytest.mark.parametrize("size", [1.0, 30.0, 300.0, 2000.0])
def test_fp16_gradients_with_rank_values_above_fp16(size, order, rank):
    """Rank values from 10 to 3e8, most of them above 65504 at the larger sizes, beside
    others that are not: sums of the same relative precision."""
    c = Case(700, 136, 264, 3, rank, "f16", order, seed=rank)
    for t in (c.x, c.dy, c.a, c.b):
        t.copy_((t.float() * size).clamp(-60000, 60000))
    c.scale.copy_(torch.tensor([1.0, 0.01, -0.5]))
    _, da, db = c.backward()
    want = ref.lora_backward(c.dy, c.x, c.w, c.a, c.b, c.adapter, c.scale, torch.float32)
    assert torch.isfinite(da).all() and torch.isfinite(db).all()
    ref.check(da, *want[1])
    ref.check(db, *want[2])


# rows, K, the skipped step: of the rank values' 16 K steps (three row tiles); of the
# gradients' 12 row tiles (two K steps), a whole one and the ragged one
@pytest.mark.parametrize("rows,K,skip", [(300, 1024, 8), (1500, 128, 5), (1500, 128, 11)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_waits_of_rank_values_and_gradients_that_run_out_are_reported(rows, K, skip, dtype):
    """The kernels' copies leave out a step (10 ms a wait): the status says so, the context
    stays usable, and the next call is right.  Only B's gradient is asked for, so that no
    product has a step of that number."""
    c = Case(rows, 136, K, 1, 8, dtype, "one", ints=True)
    code = tg.BF16 if dtype == "bf16" else tg.F16
    lora = tg.LoraAdapters(c.a.data_ptr(), K, 8 * K, c.b.data_ptr(), 8, 136 * 8, c.scale.data_ptr(), 1, 8)
    db = torch.empty(136, 8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream

    def call():
        args = (c.dy.data_ptr(), 136, c.x.data_ptr(), K, c.w.data_ptr(), K, lora)
        size = tg.gemm_lora_backward_workspace_size(*args, rows, 136, K, code, tg.F32, tg.F32)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        assert tg.gemm_lora_backward(*args, c.adapter.data_ptr(), None, K, None, K, 8 * K, db.data_ptr(), 8,
                                     136 * 8, rows, 136, K, code, tg.F32, tg.F32, ws.data_ptr(), size,
                                     stream) == tg.binding.OK
        return tg.gemm_device_status(stream)

    assert call() == tg.binding.OK
    want = db.clone()
    tg.gemm_debug_config(20_000_000, skip)
    assert call() == tg.binding.ERR_TIMEOUT
    tg.gemm_debug_config(0, -1)
    assert call() == tg.binding.OK
    t = c.scale[0].double() * (c.x.double() @ c.a[0].double().T)
    assert torch.equal(db, want) and torch.equal(db.double(), c.dy.double().T @ t)


# What sums of one sign over K values may lose where an accumulator takes 64 matrix
# instructions, each of which drops less than a unit (two half units, 2^-24) of what it
# adds up to, and K / 1024 accumulators are added with a rounding each; two more roundings
def _segments(K):
    return (128 + K / 1024 + 2) * 2.0 ** -24


@pytest.mark.parametrize("op", ["t", "n"])
@pytest.mark.parametrize("K", [1024, 1032, 8192, 20_000])
def test_grouped_products_of_long_sums_keep_fp32(K, op):
    """One accumulator for all of K dropped 3e-5 of 8192 values of one sign."""
    off = [0, 300, 300, 333, 360]
    x = _positive(1, torch.bfloat16, 360, K)
    w = _positive(2, torch.bfloat16, 4, *((264, K) if op == "t" else (K, 264)))
    y = tg.matmul_grouped(x, w, _dev(off), op_b=op)
    want = ref.grouped(x, w, off, op == "t")[0]
    assert ((y.double() - want).abs() <= _segments(K) * want).all()
    y0 = torch.rand(360, 264, device="cuda")
    added = tg.matmul_grouped(x, w, _dev(off), op_b=op, out=y0.clone(), alpha=0.5, beta=2.0)
    want = 0.5 * want + 2.0 * y0.double()
    assert ((added.double() - want).abs() <= _segments(K) * want).all()
    # results of 16 bits, through either store: the rounding of the same sums
    for pitch in (264, 265):
        for dtype in (torch.bfloat16, torch.float16):
            out = torch.empty(360, pitch, dtype=dtype, device="cuda")[:, :264]
            tg.matmul_grouped(x, w, _dev(off), op_b=op, out=out, alpha=0.5)
            assert torch.equal(out, (0.5 * y).to(dtype))


@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("name", ["forward", "backward"])
def test_fp16_waits_that_run_out_are_reported(name, few):
    """As BF16's, with the warp that splits factors behind the copies."""
    for c in ([Case(60, 264, 320, 5, 16, "f16", ints=True), Case(60, 264, 320, 60, 40, "f16", ints=True)] if few else
              [Case(2100, 2056, 320, 5, 16, "f16", ints=True)]):
        call = (lambda: (c.forward(),)) if name == "forward" else c.backward
        want = call()
        stream = torch.cuda.current_stream().cuda_stream
        assert tg.gemm_device_status(stream) == tg.binding.OK
        tg.gemm_debug_config(20_000_000, 1)
        call()
        assert tg.gemm_device_status(stream) == tg.binding.ERR_TIMEOUT
        tg.gemm_debug_config(0, -1)
        assert all(torch.equal(a, b) for a, b in zip(call(), want))


# the product on CTA pairs; few tiles, in clusters of one CTA and of several; the kernel that
# makes the rank values too
LONG_SUMS = [(2100, 2056, 8192, 3), (2100, 2056, 1088, 3), (1300, 1300, 8192, 3), (300, 1000, 8192, 3),
             (300, 1000, 8200, 90), (1300, 1300, 2048, 1)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,N,K,G", LONG_SUMS)
def test_adapted_products_of_long_sums_keep_fp32(rows, N, K, G, dtype):
    """The product and its input's gradient, FP32 results of values of one sign.  Rank values
    are summed as the shared product is, with up to eight accumulators (8 more roundings),
    a scale and parts (2), and enter the last accumulator by six instructions (12)."""
    x, w = _positive(1, dtype, rows, K), _positive(2, dtype, N, K)
    a, b = _positive(3, dtype, G, 16, K), _positive(4, dtype, G, N, 16)
    adapter = (torch.arange(rows) * 7 % (G + 1) - 1).to(torch.int32).cuda()
    limit = _segments(K) + 22 * 2.0 ** -24

    def want(x, w, f, e):
        y = x.double() @ w.double()
        for g in range(G):
            mine = adapter == g
            y[mine] += (x[mine].double() @ f[g].double()) @ e[g].double()
        return y

    y = tg.matmul_lora(x, w, a, b, adapter)
    ref_y = want(x, w.t(), a.transpose(1, 2), b.transpose(1, 2))
    assert ((y.double() - ref_y).abs() <= limit * ref_y).all()
    half = tg.matmul_lora(x, w, a, b, adapter, out_dtype=dtype)
    if dtype == torch.float16:
        assert torch.equal(half, y.half())
    # the same product as an input's gradient: from w, and a and b exchanged, turned
    none = torch.zeros(rows, N, dtype=dtype, device="cuda")
    dx = tg.matmul_lora_backward(x, none, w.t().contiguous(), b.transpose(1, 2).contiguous(),
                                 a.transpose(1, 2).contiguous(), adapter)[0]
    assert ((dx.double() - ref_y).abs() <= limit * ref_y).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,G,rank", [(10_000, 1, 256), (10_000, 3, 128), (10_000, 2, 200), (300, 3, 256),
                                         (10_000, 40, 32), (1000, 100, 48), (10_000, 130, 16)])
def test_rank_values_of_long_sums_keep_fp32(rows, G, rank, dtype):
    """Of every number of accumulators and of rounds over a tile's adapters: 32768 values of
    one sign.  Rank values add up as _segments() has it, with eight accumulators' roundings, a
    scale and parts (10); in the product up to six instructions for 16 of them, in one
    accumulator, each dropping two half units at most."""
    K = 32_768
    x = _positive(1, dtype, rows, K)
    a, b = _positive(2, dtype, G, rank, K), _positive(3, dtype, G, 24, rank)
    w = torch.zeros(24, K, dtype=dtype, device="cuda")
    adapter = (torch.arange(rows) * 7 % G).to(torch.int32).cuda()
    y = tg.matmul_lora(x, w, a, b, adapter)
    limit = _segments(K) + (10 + 2 * 6 * ((rank + 15) // 16)) * 2.0 ** -24
    for g in range(G):
        mine = adapter == g
        want = (x[mine].double() @ a[g].double().t()) @ b[g].double().t()
        assert ((y[mine].double() - want).abs() <= limit * want).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("K,pad", [(200, 0), (200, 8), (77, 3)])
def test_wgrad_results_interleaved_row_by_row(K, pad, dtype, out):
    """As matmul_grouped takes its weights: (out, groups, in) in memory."""
    off = _offsets([70, 0, 33, 200])
    dy, x = _ints(1, dtype, off[-1], 136), _ints(2, dtype, off[-1], K)
    want = ref.wgrad(dy, x, off)[0]
    buf = torch.full((136, 4, K + pad), 7.0, dtype=ref.DT[out], device="cuda")
    c = buf[:, :, :K].transpose(0, 1)
    tg.matmul_grouped_wgrad(dy, x, _dev(off), out=c)
    assert torch.equal(c.double(), want.to(ref.DT[out]).double()) and (buf[:, :, K:] == 7).all()
    tg.matmul_grouped_wgrad(dy, x, _dev(off), out=c, alpha=0.0, beta=1.0)
    assert torch.equal(c.double(), want.to(ref.DT[out]).double()) and (buf[:, :, K:] == 7).all()
    with pytest.raises(tg.GemmError):  # each row begins within the one before
        tg.matmul_grouped_wgrad(dy, x, _dev(off), out=torch.zeros(9999999, dtype=ref.DT[out], device="cuda")
                                .as_strided((4, 136, K), (K - 1, 4 * K, 1)))


@pytest.mark.parametrize("rows,N,K,G,rank", [(20, 136, 264, 3, 12), (150, 264, 200, 6, 16), (150, 264, 200, 6, 40),
                                             (1300, 2056, 264, 6, 24)])
def test_fp16_rows_see_nothing_of_other_adapters(rows, N, K, G, rank):
    """Factors, rows and gradients that are not finite stay with their adapters and rows,
    though factors are split in two and rank values go in parts."""
    c = Case(rows, N, K, G, rank, "f16", seed=5)
    y, (dx, da, db) = c.forward(), c.backward()
    c.a[1], c.b[2] = float("nan"), float("inf")
    c.x[7], c.dy[9] = float("inf"), float("nan")
    y2, (dx2, da2, db2) = c.forward(), c.backward()
    of = c.adapter
    clean = (of != 1) & (of != 2)
    keep = clean.clone()
    keep[7] = False
    assert torch.equal(y2[keep], y[keep]) and not torch.isfinite(y2[of == 1]).any()
    keep = clean.clone()
    keep[9] = False
    assert torch.equal(dx2[keep], dx[keep])
    ok = [g for g in range(G) if g not in (1, 2, int(of[7]), int(of[9]))]
    assert torch.equal(da2[ok], da[ok]) and torch.equal(db2[ok], db[ok])
    assert ok or G == 3


@pytest.mark.parametrize("dtype,rows,N,K,G,rank", [("f16", 60, 264, 320, 5, 16), ("f16", 60, 264, 320, 60, 40),
                                                   ("f16", 2100, 2056, 320, 5, 24), ("bf16", 2100, 2056, 2600, 5, 136),
                                                   ("bf16", 1300, 1300, 4200, 3, 200)])
def test_split_factors_and_segments_repeat(dtype, rows, N, K, G, rank):
    """The same bits call by call, on another stream beside the first, and from a graph whose
    adapters change between replays."""
    c = Case(rows, N, K, G, rank, dtype, "runs")
    first = c.forward(), *c.backward()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, (c.forward(), *c.backward())))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    here, there = [], []
    for _ in range(3):
        there.append((c.forward(stream=s), *c.backward(stream=s)))
        here.append((c.forward(), *c.backward()))
    torch.cuda.synchronize()
    for got in here + there:
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = c.forward(), *c.backward()
    adapters = c.adapter.clone()
    for of in (adapters.flip(0), torch.full_like(adapters, -1), adapters):
        c.adapter.copy_(of)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, (c.forward(), *c.backward())))
    assert all(torch.equal(a, b) for a, b in zip(first, held))


@pytest.mark.parametrize("rows,N,K", [(200, 136, 264), (2100, 2056, 264)])
@pytest.mark.parametrize("rank", [16, 40])
def test_fp16_parts_of_the_gradients_alone(rows, N, K, rank):
    """From C, any of the three results may be left out, and with it one of the two sets of
    rank values towards the input."""
    c = Case(rows, N, K, 3, rank, "f16", "mixed")
    want = c.backward()
    lora = tg.LoraAdapters(c.a.data_ptr(), K, rank * K, c.b.data_ptr(), rank, N * rank, c.scale.data_ptr(), 3, rank)
    args = (c.dy.data_ptr(), N, c.x.data_ptr(), K, c.w.data_ptr(), K, lora)
    size = tg.gemm_lora_backward_workspace_size(*args, rows, N, K, tg.F16, tg.F32, tg.F32)
    for keep in ([0], [1], [2], [1, 2], [0, 2], [0, 1]):
        got = [torch.full_like(t, 9.0) for t in want]
        p = [t.data_ptr() if i in keep else None for i, t in enumerate(got)]
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        rc = tg.gemm_lora_backward(*args, c.adapter.data_ptr(), p[0], K, p[1], K, rank * K, p[2], rank, N * rank, rows,
                                   N, K, tg.F16, tg.F32, tg.F32, ws.data_ptr(), size,
                                   torch.cuda.current_stream().cuda_stream)
        assert rc == tg.binding.OK
        for i, t in enumerate(got):
            assert torch.equal(t, want[i]) if i in keep else (t == 9.0).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [20, 200, 1400])
def test_one_pair_of_factors_for_every_adapter(dtype, rows):
    """Expanded factors (no stride from one adapter to the next), with scales of their own."""
    N, K = 1304, 264
    c = Case(rows, N, K, 5, 24, dtype, "mixed")
    c.a, c.b = c.a[:1].expand(5, 24, K), c.b[:1].expand(5, N, 24)
    c.check_forward(c.forward())
    c.check_backward(c.backward())
