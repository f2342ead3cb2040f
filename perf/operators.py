"""Timed cases of the block-scaled 8-bit operators and of the Newton-Schulz
orthogonalisation, with their plain forms.

`run` computes an operator either through the package (`own` true) or as
elementary torch operations in 32 bits; `exact` gives the same outputs from
the definitions in 64 bits.
"""
import math

import torch

own = False

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
F8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
# 1 / F rounded to 32 bits: a scale is the product of this and the block's largest magnitude
F8_INVERSE = {"e4m3": 9586981 * 2.0 ** -32, "e5m2": 9586981 * 2.0 ** -39}
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7


def listed():
    return [
        # the activations of 16 tokens in a decoding step, quantised before a product
        {"name": "quant row 16x4096", "op": "quant", "block": "row", "rows": 16, "cols": 4096,
         "dtype": "bf16", "f8": "e4m3"},
        # a weight matrix after an optimiser's step
        {"name": "quant tile 8192x8192", "op": "quant", "block": "tile", "rows": 8192,
         "cols": 8192, "dtype": "bf16", "f8": "e4m3"},
        # a layer's input in training: blocks along both axes (the forward product and the
        # weight gradient contract over different ones), ragged in both
        {"name": "quant pair 4999x5000", "op": "quant", "block": "pair", "rows": 4999,
         "cols": 5000, "dtype": "bf16", "f8": "e4m3"},
        # one token through a linear layer: the weights are read once
        {"name": "forward 1x4096x4096", "op": "product", "form": "forward", "M": 1, "N": 4096,
         "K": 4096, "out": "bf16"},
        # partial tiles and a partial last block in every dimension
        {"name": "forward 96x200x1000", "op": "product", "form": "forward", "M": 96, "N": 200,
         "K": 1000, "out": "f16"},
        # a decoding batch
        {"name": "forward 64x8192x8192", "op": "product", "form": "forward", "M": 64, "N": 8192,
         "K": 8192, "out": "bf16"},
        # a prompt or a training batch
        {"name": "forward 8192x8192x4096", "op": "product", "form": "forward", "M": 8192,
         "N": 8192, "K": 4096, "out": "bf16"},
        # the gradient of that layer's input: the same weight bytes, contracted over their rows
        {"name": "input grad 4096x4096x8192", "op": "product", "form": "input", "M": 4096,
         "N": 4096, "K": 8192, "out": "bf16"},
        # the gradient of its weight: a contraction over tokens, a scale for each row of both
        {"name": "weight grad 4096x4096x5000", "op": "product", "form": "weight", "M": 4096,
         "N": 4096, "K": 5000, "out": "f32"},
        # the update of a small square weight: latency counts
        {"name": "orthogonalise 128x128", "op": "orth", "batch": 1, "rows": 128, "cols": 128,
         "dtype": "f32", "out": "bf16"},
        # the updates of eight layers' narrow weights together, taller than wide, ragged
        {"name": "orthogonalise 8x1000x200", "op": "orth", "batch": 8, "rows": 1000, "cols": 200,
         "dtype": "bf16", "out": "bf16"},
        # the update of a large square weight
        {"name": "orthogonalise 4096x4096", "op": "orth", "batch": 1, "rows": 4096, "cols": 4096,
         "dtype": "bf16", "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "product", "product", "product", "orth", "orth"])
    if op == "quant":
        return {"op": op, "block": rng.choice(["row", "col", "tile", "pair"]),
                "rows": _log(rng, 1, 8192), "cols": _log(rng, 64, 8192),
                "dtype": rng.choice(["bf16", "f16", "f32"]), "f8": rng.choice(["e4m3", "e5m2"])}
    if op == "product":
        form = rng.choice(["forward", "forward", "input", "weight"])
        M = _log(rng, 1, 8192) if form != "weight" else _log(rng, 64, 4096)
        return {"op": op, "form": form, "M": M, "N": _log(rng, 64, 8192), "K": _log(rng, 64, 4096),
                "out": "f32" if form == "weight" else rng.choice(["bf16", "f16"])}
    rows, cols = _log(rng, 32, 4096), _log(rng, 32, 4096)
    most = max(1, min(8, 4096 * 4096 // (rows * cols)))
    return {"op": op, "batch": rng.randint(1, most), "rows": rows, "cols": cols,
            "dtype": rng.choice(["bf16", "f32"]), "out": "bf16"}


def _blocks(n):
    return (n + 127) // 128


# ------------------------------------------------------------- quantisation
# A block of x has the scale s = amax * (1 / F) (one where the block is all
# zero), and q = rn8(x * (1 / s)), each step rounded to 32 bits.  Blocks are 1 x 128 ("row", scales stored
# [column block][row]), 128 x 1 ("col", [row block][column]) or 128 x 128
# ("tile", [row block][column block]).

def _shape_blocks(x, block):
    """x, padded with zeros to whole blocks, as a view whose last two axes are a block's."""
    R, C = x.shape
    br, bc = {"row": (1, 128), "col": (128, 1), "tile": (128, 128)}[block]
    x = torch.nn.functional.pad(x, (0, -C % bc, 0, -R % br))
    return x.reshape(x.shape[0] // br, br, x.shape[1] // bc, bc).permute(0, 2, 1, 3)


def _plain_quant(x, block, f8):
    """(q as stored, scales as stored) of a 32-bit x."""
    R, C = x.shape
    v = _shape_blocks(x, block)
    amax = v.abs().amax(dim=(2, 3), keepdim=True)
    s = torch.where(amax > 0, (amax * F8_INVERSE[f8]).clamp_min(2.0 ** -126),
                    torch.ones_like(amax))
    q = (v * (1.0 / s)).clamp(-F8_MAX[f8], F8_MAX[f8]).to(F8[f8])
    q = q.permute(0, 2, 1, 3).reshape(v.shape[0] * v.shape[2], -1)[:R, :C]
    s = s[:, :, 0, 0]
    return q, (s.t() if block == "row" else s).contiguous()


def _pitched(q):
    """q with rows that start on 16-byte boundaries, as the quantiser lays them out."""
    R, C = q.shape
    buf = torch.zeros((R, (C + 15) // 16 * 16), dtype=torch.uint8, device=q.device).view(q.dtype)
    view = buf[:, :C]
    view.copy_(q)
    return view


# ------------------------------------------------------------------- inputs

def _activations(rows, cols, gen, dtype):
    """Normal values with a size of their own for each row and a few large columns."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device="cuda"))
    x *= torch.where(torch.rand(1, cols, generator=gen, device="cuda") < 0.01, 10.0, 1.0)
    return x.to(dtype)


def _update(batch, rows, cols, gen, dtype):
    """A gradient's running mean: some strong directions over a noise floor."""
    rank = max(4, min(rows, cols) // 16)
    u = torch.randn(batch, rows, rank, generator=gen, device="cuda")
    v = torch.randn(batch, rank, cols, generator=gen, device="cuda")
    g = 1e-3 * (u @ v / math.sqrt(rank)
                + 0.2 * torch.randn(batch, rows, cols, generator=gen, device="cuda"))
    return (g[0] if batch == 1 else g).to(dtype).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "quant":
        return dict(case, x=_activations(case["rows"], case["cols"], gen, DT[case["dtype"]]))
    if case["op"] == "orth":
        return dict(case, g=_update(case["batch"], case["rows"], case["cols"], gen,
                                    DT[case["dtype"]]))
    M, N, K = case["M"], case["N"], case["K"]
    # what is stored, the form each operand is used in, and its blocks: a scale for
    # each row and 128 of the contraction, or for 128 x 128 of a weight
    if case["form"] == "forward":    # x (tokens x in), W (out x in)
        a, ba = _activations(M, K, gen, torch.float32), "row"
        b, bb = torch.randn(N, K, generator=gen, device="cuda") / math.sqrt(K), "tile"
    elif case["form"] == "input":    # dy (tokens x out), W (out x in)
        a, ba = _activations(M, K, gen, torch.float32), "row"
        b, bb = torch.randn(K, N, generator=gen, device="cuda") / math.sqrt(K), "tile"
    else:                            # dy (tokens x out), x (tokens x in)
        a, ba = _activations(K, M, gen, torch.float32), "col"
        b, bb = _activations(K, N, gen, torch.float32), "col"
    qa, sa = _plain_quant(a, ba, "e4m3")
    qb, sb = _plain_quant(b, bb, "e4m3")
    return dict(case, a=_pitched(qa), sa=sa, b=_pitched(qb), sb=sb)


#: the form of each operand: as stored ("n") or transposed ("t")
FORMS = {"forward": ("n", "t"), "input": ("n", "n"), "weight": ("t", "n")}


# --------------------------------------------------------------- plain forms

def _spread(s, rows, cols, block):
    """A scale for each element of a rows x cols matrix."""
    if block == "row":
        s = s.t()
    if block != "row":
        s = s.repeat_interleave(128, 0)
    if block != "col":
        s = s.repeat_interleave(128, 1)
    return s[:rows, :cols]


def _dequant(q, s, block, dtype):
    return q.to(dtype) * _spread(s.to(dtype), q.shape[0], q.shape[1], block)


def _product(state, dtype):
    weight = state["form"] == "weight"
    a = _dequant(state["a"], state["sa"], "col" if weight else "row", dtype)
    b = _dequant(state["b"], state["sb"], "col" if weight else "tile", dtype)
    op_a, op_b = FORMS[state["form"]]
    return (a.t() if op_a == "t" else a) @ (b.t() if op_b == "t" else b)


def _quantised(q, s):
    return {"codes": q, "scales": s}


def _plain(state):
    if state["op"] == "quant":
        x = state["x"].float()
        if state["block"] == "pair":
            return {b: _quantised(*_plain_quant(x, b, state["f8"])) for b in ("row", "col")}
        return _quantised(*_plain_quant(x, state["block"], state["f8"]))
    if state["op"] == "product":
        return _product(state, torch.float32).to(DT[state["out"]])
    x = state["g"].float()
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    x = x / (x.square().sum(dim=(-2, -1), keepdim=True).sqrt() + EPS)
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        g = x @ x.mT
        x = a * x + (b * g + c * (g @ g)) @ x
    return (x.mT if tall else x).to(DT[state["out"]])


def run(state):
    if not own:
        return _plain(state)
    import tiled_matrix_multiplication_output_gb300 as tg
    if state["op"] == "quant":
        if state["block"] == "pair":
            row, col = tg.quantize_fp8_pair(state["x"], dtype=state["f8"])
            return {"row": _quantised(*row), "col": _quantised(*col)}
        return _quantised(*tg.quantize_fp8(state["x"], block=state["block"], dtype=state["f8"]))
    if state["op"] == "product":
        op_a, op_b = FORMS[state["form"]]
        return tg.matmul_fp8(state["a"], state["sa"], state["b"], state["sb"], op_a=op_a,
                             op_b=op_b, out_dtype=DT[state["out"]])
    return tg.newton_schulz(state["g"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS,
                            out_dtype=DT[state["out"]])


# --------------------------------------------------------------------- work

def work(case):
    if case["op"] == "quant":
        R, C = case["rows"], case["cols"]
        scales = {"row": R * _blocks(C), "col": _blocks(R) * C, "tile": _blocks(R) * _blocks(C)}
        kinds = ("row", "col") if case["block"] == "pair" else (case["block"],)
        return {"bytes": R * C * SIZE[case["dtype"]] + sum(R * C + 4 * scales[k] for k in kinds),
                "flops": 2 * R * C * len(kinds)}
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        other = N if case["form"] == "weight" else _blocks(N)
        return {"bytes": M * K + K * N + 4 * _blocks(K) * (M + other) + M * N * SIZE[case["out"]],
                "flops": 2 * M * N * K}
    m, n = sorted((case["rows"], case["cols"]))
    # x x^T and its square are symmetric: half of each is computed
    return {"bytes": case["batch"] * m * n * (SIZE[case["dtype"]] + SIZE[case["out"]]),
            "flops": case["batch"] * STEPS * (m * m * n + m * m * m + 2 * m * m * n)}


# -------------------------------------------------------------------- exact

def _round8(v, f8):
    """Nearest value (ties to even) of a 64-bit v in the 8-bit type, saturating."""
    bits, low = {"e4m3": (3, -6), "e5m2": (2, -14)}[f8]
    _, e = torch.frexp(v)
    unit = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(low) - bits)
    return (torch.round(v / unit) * unit).clamp(-F8_MAX[f8], F8_MAX[f8])


def _exact_quant(x, block, f8):
    """The definition's own roundings (the scale and its inverse in 32 bits, the quotient in 32
    bits, then 8) applied to values computed in 64 bits."""
    def single(v):
        return v.to(torch.float32).to(torch.float64)

    R, C = x.shape
    v = _shape_blocks(x, block)
    amax = v.abs().amax(dim=(2, 3), keepdim=True)
    s = torch.where(amax > 0, single(amax * F8_INVERSE[f8]).clamp_min(2.0 ** -126), 1.0)
    q = _round8(single(v * single(1.0 / s)), f8)
    q = q.permute(0, 2, 1, 3).reshape(v.shape[0] * v.shape[2], -1)[:R, :C]
    s = s[:, :, 0, 0]
    return _quantised(q, (s.t() if block == "row" else s).contiguous())


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "quant":
        x = state["x"].double()
        if case["block"] == "pair":
            return {b: _exact_quant(x, b, case["f8"]) for b in ("row", "col")}
        return _exact_quant(x, case["block"], case["f8"])
    if case["op"] == "product":
        weight = case["form"] == "weight"
        sums = None
        for k0 in range(0, case["K"], 128):  # block by block of the contraction
            k = slice(k0, min(k0 + 128, case["K"]))
            kb = k0 // 128
            op_a, op_b = FORMS[case["form"]]
            a = (state["a"][k].t() if op_a == "t" else state["a"][:, k]).double()
            b = (state["b"][k] if op_b == "n" else state["b"][:, k].t()).double()
            sa = state["sa"][kb].double()[:, None]
            if weight:
                sb = state["sb"][kb].double()
            else:
                sb = state["sb"][:, kb] if op_b == "t" else state["sb"][kb]
                sb = sb.double().repeat_interleave(128)[:case["N"]]
            part = (a @ b) * sa * sb
            sums = part if sums is None else sums.add_(part)
        return sums
    g = state["g"].double()
    g = g[None] if g.dim() == 2 else g
    a, b, c = COEFFICIENTS
    out = []
    for x in g:
        x = x / (torch.linalg.norm(x) + EPS)
        for _ in range(STEPS):  # from the side that is shorter, without transposing
            if x.shape[0] <= x.shape[1]:
                p = x @ x.t()
                x = a * x + b * (p @ x) + c * (p @ (p @ x))
            else:
                p = x.t() @ x
                x = a * x + b * (x @ p) + c * ((x @ p) @ p)
        out.append(x)
    return out[0] if case["batch"] == 1 else torch.stack(out)
