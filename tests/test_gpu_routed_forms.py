"""The grouped products and the adapters where their kernels change form or come
to a limit: tiles of every size, waves of tiles, sums beyond a segment, ranks in
several chunks, sizes beyond 32-bit offsets, waits that run out, two calls at
once, and an eager autograd graph beside a captured one."""
import threading

import pytest
import torch

import tiled_matrix_multiplication_output_gb300 as tg
from tests import routed_reference as ref
from tests.routed_reference import DT
from tests.test_gpu_grouped import _dev, _ints, _offsets, _randn
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
@pytest.mark.parametrize("rows", [1, 15, 16, 17, 31, 33, 63, 65, 97, 127, 129, 160, 193, 224, 225, 255, 257,
                                  289, 511, 513, 1000])
def test_every_tile_extent(rows, op):
    """One group of any number of rows: halves of tiles are boxes of 128, 64, 32, 16."""
    off = _offsets([2, rows, 0, 3])
    x = _ints(rows, "bf16", off[-1], 128)
    w = _ints(rows + 1, "bf16", 4, *((264, 128) if op == "t" else (128, 264)))
    for out in (torch.float32, torch.bfloat16):
        y = tg.matmul_grouped(x, w, _dev(off), op_b=op, out_dtype=out)
        assert torch.equal(y, ref.grouped(x, w, off, op == "t")[0].to(out))


@pytest.mark.parametrize("counts", [[700] * 24, [4100, 30, 2500, 1, 900], [130] * 60])
def test_many_waves_of_tiles(counts):
    """More tiles than pairs of CTAs: raster bands, tiles of fewer rows, both accumulators."""
    off = _offsets(counts)
    x, w = _ints(1, "f16", off[-1], 192), _ints(2, "f16", len(counts), 1288, 192)
    y = tg.matmul_grouped(x, w, _dev(off), out_dtype=torch.float16)
    want = ref.grouped(x, w, off, True)[0]
    assert torch.equal(y.double(), want)
    dx = tg.matmul_grouped(y.clamp(-8, 8), w, _dev(off), op_b="n")
    assert torch.equal(dx.double(), ref.grouped(y.clamp(-8, 8), w, off, False)[0])


@pytest.mark.parametrize("rows", [767, 768, 769, 1536, 1537, 5000])
def test_wgrad_sums_of_several_segments(rows):
    off = _offsets([rows, 5, 0, rows // 3])
    dy, x = _ints(3, "bf16", off[-1], 520), _ints(4, "bf16", off[-1], 392)
    c = tg.matmul_grouped_wgrad(dy, x, _dev(off))
    assert torch.equal(c.double(), ref.wgrad(dy, x, off)[0])
    c0 = c.clone()
    tg.matmul_grouped_wgrad(dy, x, _dev(off), out=c, alpha=-1.0, beta=1.0)
    assert not c.any() and c0.any()


def test_wgrad_of_long_sums_keeps_fp32():
    """A sum over 8000 rows of one sign: what the tensor core drops when it adds would
    be 500 instructions' half units, 3e-5; segments of 48 instructions keep it below
    48 * 2^-24 and the segments' own sums below 11 more."""
    g = torch.Generator().manual_seed(5)
    dy, x = (torch.rand(8000, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    c = tg.matmul_grouped_wgrad(dy, x, _dev([0, 8000]))
    want = dy.double().t() @ x.double()
    assert ((c[0].double() - want).abs() <= 60 * 2.0 ** -24 * want).all()


@pytest.mark.parametrize("rows,N,K,G,r", [(3000, 2056, 136, 3, 16), (2600, 136, 2056, 40, 8), (1290, 1288, 264, 2, 96),
                                          (520, 4104, 72, 5, 256), (140, 72, 4104, 140, 16), (1, 4104, 4104, 1, 64)])
@pytest.mark.parametrize("order", ["mixed", "runs", "one"])
def test_lora_forms(rows, N, K, G, r, order):
    """Few and many output tiles, thin last waves, one to sixteen chunks of rank values,
    more adapters than a tile's rows, single rows."""
    c = Case(rows, N, K, G, r, "bf16", order)
    c.check_forward(c.forward(out_dtype=torch.bfloat16))
    c.check_forward(c.forward())
    c.check_backward(c.backward())
    c.check_backward(c.backward(out_dtype=torch.bfloat16, grad_dtype=torch.bfloat16))


def test_lora_parts_of_the_gradients_alone():
    """From C, any of the three results may be left out."""
    c = Case(200, 136, 264, 3, 16, "bf16", "mixed")
    want = c.backward()
    lora = tg.LoraAdapters(c.a.data_ptr(), 264, 16 * 264, c.b.data_ptr(), 16, 136 * 16, c.scale.data_ptr(), 3, 16)
    for keep in ([0], [1], [2], [1, 2], [0, 2]):
        got = [torch.full_like(t, 9.0) for t in want]
        p = [t.data_ptr() if i in keep else None for i, t in enumerate(got)]
        size = tg.gemm_lora_backward_workspace_size(c.dy.data_ptr(), 136, c.x.data_ptr(), 264, c.w.data_ptr(), 264,
                                                    lora, 200, 136, 264, tg.BF16, tg.F32, tg.F32)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        rc = tg.gemm_lora_backward(c.dy.data_ptr(), 136, c.x.data_ptr(), 264, c.w.data_ptr(), 264, lora,
                                   c.adapter.data_ptr(), p[0], 264, p[1], 264, 16 * 264, p[2], 16, 136 * 16, 200,
                                   136, 264, tg.BF16, tg.F32, tg.F32, ws.data_ptr(), size,
                                   torch.cuda.current_stream().cuda_stream)
        assert rc == tg.binding.OK
        for i, t in enumerate(got):
            assert torch.equal(t, want[i]) if i in keep else (t == 9.0).all()


def test_weights_beyond_32_bit_offsets():
    G, N, K = 3, 30_000, 32_768  # 2.9e9 elements
    w = torch.zeros(G, N, K, dtype=torch.bfloat16, device="cuda")
    w[2, -40:] = _ints(6, "bf16", 40, K)
    x = _ints(7, "bf16", 9, K)
    y = tg.matmul_grouped(x, w, _dev([0, 2, 2, 9]))
    assert torch.equal(y[2:, -40:].double(), x[2:].double() @ w[2, -40:].double().t())
    assert not y[:2].any() and not y[:, :-40].any()
    del w
    c = torch.full((G, N, K), 5.0, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros(9, N, dtype=torch.bfloat16, device="cuda")
    dy[2:, -40:] = _ints(8, "bf16", 7, 40)
    tg.matmul_grouped_wgrad(dy, x, _dev([0, 2, 2, 9]), out=c)
    assert torch.equal(c[2, -40:].double(), dy[2:, -40:].double().t() @ x[2:].double())
    assert not c[:2].any() and not c[2, :-40].any()


def _grouped_calls():
    off = _dev(_offsets([300, 0, 40, 700]))
    x, dy = _ints(9, "bf16", 1040, 320), _ints(10, "bf16", 1040, 264)
    w = _ints(11, "bf16", 4, 264, 320)
    few, many = Case(60, 264, 320, 5, 16, "bf16", ints=True), Case(2100, 2056, 320, 5, 16, "bf16", ints=True)
    each = Case(60, 264, 320, 60, 16, "bf16", ints=True)
    return {
        "t": lambda: (tg.matmul_grouped(x, w, off),),
        "n": lambda: (tg.matmul_grouped(dy, w, off, op_b="n"),),
        "wgrad": lambda: (tg.matmul_grouped_wgrad(dy, x, off),),
        "lora few tiles": lambda: (few.forward(),),
        "lora many adapters": lambda: (each.forward(),),
        "lora many tiles": lambda: (many.forward(),),
        "lora backward": lambda: many.backward(),
    }


@pytest.mark.parametrize("name", ["t", "n", "wgrad", "lora few tiles", "lora many adapters", "lora many tiles",
                                  "lora backward"])
def test_a_wait_that_runs_out_is_reported(name):
    """The producer skips one K step (10 ms a wait): the status says so, the context stays
    usable, and the next call is right."""
    call = _grouped_calls()[name]
    want = call()
    stream = torch.cuda.current_stream().cuda_stream
    assert tg.gemm_device_status(stream) == tg.binding.OK
    tg.gemm_debug_config(20_000_000, 1)
    call()
    assert tg.gemm_device_status(stream) == tg.binding.ERR_TIMEOUT
    tg.gemm_debug_config(0, -1)
    assert tg.gemm_device_status(stream) == tg.binding.OK
    assert all(torch.equal(a, b) for a, b in zip(call(), want))


def test_two_calls_at_once():
    """From two host threads on two streams, with workspaces of their own."""
    calls = _grouped_calls()
    want = {k: f() for k, f in calls.items()}
    torch.cuda.synchronize()
    wrong = []

    def work(names):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                for k in names:
                    got = calls[k]()
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[k])):
                        wrong.append(k)

    threads = [threading.Thread(target=work, args=(n,)) for n in (list(calls), list(calls)[::-1])]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_backward_captured_beside_an_eager_graph():
    """The gradients' calls in a captured graph while another autograd graph of the same
    leaves lives; both give what they gave."""
    c = Case(150, 136, 72, 3, 8, "bf16", "mixed")
    a = c.a.clone().requires_grad_()

    class F(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, a):
            ctx.save_for_backward(x, a)
            return tg.matmul_lora(x, c.w, a, c.b, c.adapter, c.scale)

        @staticmethod
        def backward(ctx, dy):
            x, a = ctx.saved_tensors
            dx, da, _ = tg.matmul_lora_backward(dy.to(torch.bfloat16), x, c.w, a, c.b, c.adapter, c.scale,
                                                out_dtype=x.dtype, grad_dtype=a.dtype)
            return dx, da

    eager = F.apply(c.x, a)  # lives throughout
    want = torch.autograd.grad(eager, a, c.dy.float(), retain_graph=True)[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = tg.matmul_lora(c.x, c.w, a.detach(), c.b, c.adapter, c.scale)
        da = tg.matmul_lora_backward(c.dy, c.x, c.w, a.detach(), c.b, c.adapter, c.scale,
                                     out_dtype=torch.bfloat16, grad_dtype=torch.bfloat16)[1]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, eager.detach()) and torch.equal(da, want)
    assert torch.equal(torch.autograd.grad(eager, a, c.dy.float())[0], want)


@pytest.mark.parametrize("dtype", [tg.F32, tg.BF16])
@pytest.mark.parametrize("rows", [3, 300, 5000])
@pytest.mark.parametrize("adapters, rank", [(0, 8), (4, 0), (0, 0)])
def test_no_adapters_reads_no_pointer_of_theirs(dtype, rows, adapters, rank):
    """Small, large and FP32 forms with every adapter pointer null."""
    N, K = 1304, 136
    name = "f32" if dtype == tg.F32 else "bf16"
    x, w, dy = _ints(1, name, rows, K), _ints(2, name, N, K), _ints(3, name, rows, N)
    lora = tg.LoraAdapters(None, 0, 0, None, 0, 0, None, adapters, rank)
    y, dx = torch.empty(rows, N, device="cuda"), torch.empty(rows, K, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    assert tg.gemm_lora_workspace_size(x.data_ptr(), K, w.data_ptr(), K, lora, rows, N, K, dtype,
                                       tg.F32) == 0
    assert tg.gemm_lora(x.data_ptr(), K, w.data_ptr(), K, lora, None, y.data_ptr(), N, rows, N, K,
                        dtype, tg.F32, None, 0, stream) == tg.binding.OK
    assert tg.gemm_lora_backward(dy.data_ptr(), N, None, 0, w.data_ptr(), K, lora, None, dx.data_ptr(),
                                 K, None, 0, 0, None, 0, 0, rows, N, K, dtype, tg.F32, tg.F32, None, 0,
                                 stream) == tg.binding.OK
    assert torch.equal(y.double(), x.double() @ w.double().T)
    assert torch.equal(dx.double(), dy.double() @ w.double())


# rows, N, K, adapters, rank: one kernel makes the rank values (cases with up to 32
# adapters x K steps of a CTA), on clusters of 1, 2, 4 and 8, with the factors of more
# adapters than come beside W, several tiles of rows, K steps that wrap the ring
OWN = [
    (1, 8, 8, 1, 1), (1, 136, 4096, 1, 16), (5, 1000, 2048, 4, 8), (40, 136, 64, 20, 16), (40, 136, 128, 30, 5),
    (90, 264, 130, 10, 32), (128, 2048, 1024, 3, 8), (128, 2432, 520, 2, 17), (130, 4744, 1024, 2, 12),
    (300, 500, 4000, 3, 16), (1000, 1000, 960, 2, 24), (77, 131, 515, 6, 7), (2000, 200, 400, 16, 16),
]


@pytest.mark.parametrize("case", OWN, ids=str)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_rank_values_made_by_the_products_kernel(case, dtype):
    rows, N, K, G, r = case
    for out in (DT[dtype], torch.float32):
        c = Case(rows, N, K, G, r, dtype, seed=rows + r)
        y = c.forward(out_dtype=out)
        c.check_forward(y)
        assert torch.equal(c.forward(out_dtype=out), y)  # identical run to run
        c = Case(rows, N, K, G, r, dtype, ints=True)
        want = c.x.double() @ c.w.double().T
        for g in range(G):
            of = c.adapter == g
            t = c.scale[g].double() * (c.x[of].double() @ c.a[g].double().T)
            want[of] += t @ c.b[g].double().T
        assert torch.equal(c.forward(out_dtype=out).double(), want.to(out).double())


def test_few_adapters_need_one_launch_and_no_workspace():
    c = Case(5, 1000, 2048, 4, 8, "bf16")
    lora = tg.LoraAdapters(c.a.data_ptr(), 2048, 8 * 2048, c.b.data_ptr(), 8, 8000, None, 4, 8)
    assert tg.gemm_lora_workspace_size(c.x.data_ptr(), 2048, c.w.data_ptr(), 2048, lora, 5, 1000, 2048,
                                       tg.BF16, tg.BF16) == 0
    c.forward()
    n = tg.gemm_launch_count()
    c.forward()
    assert tg.gemm_launch_count() == n + 1


@pytest.mark.parametrize("rows", [1, 30, 200])
def test_one_kernel_keeps_infinities_of_other_adapters_away(rows):
    c = Case(rows, 264, 520, 3, 12, "bf16", seed=3)
    c.adapter.copy_(torch.arange(rows) % 4 - 1)
    clean = c.forward()
    c.a[1] = float("inf")
    c.b[2] = float("nan")
    y = c.forward()
    keep = (c.adapter != 1) & (c.adapter != 2)
    assert torch.equal(y[keep], clean[keep]) and not torch.isfinite(y[~keep]).any()
    c.x[0] = float("inf")  # an infinity in a row stays in it
    assert torch.equal(c.forward()[keep][1:], clean[keep][1:])


@pytest.mark.parametrize("rank", [8, 40, 72, 128])
@pytest.mark.parametrize("runs", [(40, 128, 300, 17, 640), (1, 700), (129, 127, 384, 60)])
def test_gradients_where_whole_and_shared_row_tiles_alternate(rank, runs):
    """Row tiles of one adapter beside row tiles of several, in rings of every length."""
    c = Case(5000, 264, 136, 3, rank, "bf16", ints=True)
    of, i = [], 0
    while len(of) < 5000:
        of += [(i * 7 // 3) % 4 - 1] * runs[i % len(runs)]
        i += 1
    c.adapter.copy_(torch.tensor(of[:5000], dtype=torch.int32))
    _, da, db = c.backward(grad_dtype=torch.float32)
    for g in range(3):
        rows = c.adapter == g
        u = c.scale[g].double() * (c.dy[rows].double() @ c.b[g].double())
        t = c.scale[g].double() * (c.x[rows].double() @ c.a[g].double().T)
        for got, want, size in ((da[g], u.T @ c.x[rows].double(), u.abs().T @ c.x[rows].double().abs()),
                                (db[g], c.dy[rows].double().T @ t, c.dy[rows].double().abs().T @ t.abs())):
            # sums of integers: exact while no partial sum needs more than 24 bits
            assert size.max() < 2 ** 24 and torch.equal(got.double(), want)


@pytest.mark.parametrize("rows", [3, 200])
def test_as_many_adapters_as_a_call_takes(rows):
    G, N, K = 65535, 72, 64
    c = Case(rows, N, K, 1, 1, "bf16", ints=True)
    g = torch.Generator().manual_seed(5)
    c.a = torch.randint(-2, 3, (G, 1, K), generator=g).bfloat16().cuda()
    c.b = torch.randint(-2, 3, (G, N, 1), generator=g).bfloat16().cuda()
    c.scale = torch.randint(1, 3, (G,), generator=g).float().cuda()
    c.adapter.copy_(torch.randint(0, G, (rows,), generator=g))
    c.adapter[0], c.adapter[1], c.adapter[2] = G - 1, G, 0
    of = c.adapter.long().clamp(max=G - 1)
    s = c.scale[of].double()[:, None] * (c.adapter < G)[:, None]
    a, b, x, dy, w = c.a[of, 0].double(), c.b[of, :, 0].double(), c.x.double(), c.dy.double(), c.w.double()
    t, u = s * (x * a).sum(1, True), s * (dy * b).sum(1, True)
    assert torch.equal(c.forward().double(), x @ w.T + t * b)
    dx, da, db = c.backward()
    assert torch.equal(dx.double(), dy @ w + u * a)
    want_a, want_b = torch.zeros_like(c.a, dtype=torch.float64), torch.zeros_like(c.b, dtype=torch.float64)
    want_a[:, 0].index_add_(0, of, u * x)
    want_b[:, :, 0].index_add_(0, of, t * dy)
    assert torch.equal(da.double(), want_a) and torch.equal(db.double(), want_b)


@pytest.mark.parametrize("rows", [1, 5, 140])
@pytest.mark.parametrize("rank", [4, 48])
def test_few_rows_of_very_many_outputs(rows, rank):
    """More tiles than the kernel for few of them takes."""
    c = Case(rows, 40008, 72, 2, rank, "bf16", ints=True)
    want = c.x.double() @ c.w.double().T
    for g in range(2):
        of = c.adapter == g
        want[of] += (c.scale[g].double() * (c.x[of].double() @ c.a[g].double().T)) @ c.b[g].double().T
    assert torch.equal(c.forward().double(), want)


@pytest.mark.parametrize("rank", [4, 12, 40, 128])
@pytest.mark.parametrize("size", [1e-2, 1e-3, 1e-4])
def test_fp16_gradients_from_small_values(rank, size):
    """Rank values of 1e-3 down to 1e-7, below what FP16 holds: their gradients keep
    the precision of larger ones."""
    c = Case(300, 136, 264, 3, rank, "f16", seed=rank)
    c.dy.mul_(size)
    c.x.mul_(size)
    c.a.mul_(size)
    c.b.mul_(size)
    want = ref.lora_backward(c.dy, c.x, c.w, c.a, c.b, c.adapter, c.scale, torch.float32)
    _, da, db = c.backward(grad_dtype=torch.float32)
    ref.check(da, *want[1])
    ref.check(db, *want[2])
