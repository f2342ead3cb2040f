"""Timed cases of the products grouped by expert and of low-rank adapters beside a
shared projection, forward and backward, with their plain forms.

`run` computes an operator either through the package (`own` true) or as
elementary torch operations in 32 bits; `exact` gives the same outputs from
the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    # N: outputs, K: inputs of a weight (N x K); "tokens" each choose "top" of "experts"
    return [
        # one token of a decoding step through the eight experts chosen for it
        {"name": "grouped decode 8 of 64, 2048x1024", "op": "grouped", "form": "forward",
         "tokens": 1, "top": 8, "experts": 64, "pad": 0, "skew": 0.0, "deal": 1, "N": 2048,
         "K": 1024, "dtype": "bf16", "out": "bf16"},
        # a decoding batch of 64 requests: a few rows for each expert, some experts with none
        {"name": "grouped batch 256 of 64, 4096x2048", "op": "grouped", "form": "forward",
         "tokens": 64, "top": 4, "experts": 64, "pad": 0, "skew": 0.7, "deal": 2, "N": 4096,
         "K": 2048, "dtype": "bf16", "out": "bf16"},
        # prompts or a training batch through sixteen experts
        {"name": "grouped 16384 of 16, 4096x4096", "op": "grouped", "form": "forward",
         "tokens": 8192, "top": 2, "experts": 16, "pad": 0, "skew": 0.5, "deal": 3, "N": 4096,
         "K": 4096, "dtype": "bf16", "out": "bf16"},
        # the gradient of the experts' input, odd sizes, a buffer with room behind the last row
        {"name": "grouped input grad 4998 of 12, 2056x1000", "op": "grouped", "form": "input",
         "tokens": 2499, "top": 2, "experts": 12, "pad": 37, "skew": 1.5, "deal": 4, "N": 2056,
         "K": 1000, "dtype": "f16", "out": "f16"},
        # experts kept in 32 bits, a small batch
        {"name": "grouped fp32 999 of 8, 512x768", "op": "grouped", "form": "forward",
         "tokens": 999, "top": 1, "experts": 8, "pad": 0, "skew": 0.5, "deal": 5, "N": 512,
         "K": 768, "dtype": "f32", "out": "f32"},
        # the gradient of the experts' weights over a training batch
        {"name": "grouped weight grad 16384 of 8, 4096x2048", "op": "wgrad", "tokens": 8192,
         "top": 2, "experts": 8, "pad": 0, "skew": 0.5, "deal": 6, "N": 4096, "K": 2048,
         "dtype": "bf16", "out": "f32"},
        # the same of a small batch over many experts: short sums, empty groups
        {"name": "grouped weight grad 301 of 24, 520x1000", "op": "wgrad", "tokens": 301,
         "top": 1, "experts": 24, "pad": 3, "skew": 1.5, "deal": 7, "N": 520, "K": 1000,
         "dtype": "f16", "out": "f16"},
        # a few requests' tokens, small ranks, some without an adapter
        {"name": "lora decode 5, 1000x2048, rank 8", "op": "lora", "tokens": 5, "run": 1,
         "adapters": 4, "none": 0.2, "deal": 8, "N": 1000, "K": 2048, "rank": 8,
         "dtype": "f16", "out": "f16"},
        # a decoding batch in which nearly every request has an adapter of its own
        {"name": "lora decode 64, 4096x4096, rank 16", "op": "lora", "tokens": 64, "run": 1,
         "adapters": 64, "none": 0.1, "deal": 9, "N": 4096, "K": 4096, "rank": 16,
         "dtype": "bf16", "out": "bf16"},
        # prompts of several requests
        {"name": "lora prompts 8192, 4096x4096, rank 64", "op": "lora", "tokens": 8192,
         "run": 700, "adapters": 12, "none": 0.1, "deal": 10, "N": 4096, "K": 4096, "rank": 64,
         "dtype": "bf16", "out": "bf16"},
        # training one adapter for each of a batch's tasks
        {"name": "lora backward 4096, 4096x4096, rank 16", "op": "lora_backward", "tokens": 4096,
         "run": 512, "adapters": 6, "none": 0.0, "deal": 11, "N": 4096, "K": 4096, "rank": 16,
         "dtype": "bf16", "out": "bf16"},
        # short mixed sequences, sizes and rank off the usual grid
        {"name": "lora backward 777, 1000x2000, rank 12", "op": "lora_backward", "tokens": 777,
         "run": 33, "adapters": 5, "none": 0.2, "deal": 12, "N": 1000, "K": 2000, "rank": 12,
         "dtype": "f16", "out": "f16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A layer's width: mostly a multiple of 8, now and then any number."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.15 else max(8, n // 8 * 8)


def draw(rng):
    op = rng.choice(["grouped", "grouped", "grouped", "wgrad", "lora", "lora", "lora_backward"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    case = {"op": op, "deal": rng.randrange(1, 1 << 30), "N": _width(rng, 128, 4096),
            "K": _width(rng, 128, 4096), "dtype": dtype, "out": dtype}
    if op in ("grouped", "wgrad"):
        experts = _log(rng, 2, 64)
        top = rng.randint(1, min(8, experts))
        most = 16384 if experts <= 16 else 8192
        case.update(tokens=max(1, _log(rng, 1, most) // top), top=top, experts=experts,
                    pad=rng.choice([0, 0, rng.randint(1, 200)]), skew=rng.uniform(0.0, 1.5))
        if op == "grouped":
            case["form"] = rng.choice(["forward", "forward", "input"])
            if rng.random() < 0.1:  # 32 bits: smaller layers
                case.update(dtype="f32", out="f32", N=min(case["N"], 1024), K=min(case["K"], 1024),
                            tokens=min(case["tokens"], 1024))
        else:
            case["out"] = rng.choice(["f32", dtype])
        return case
    tokens = _log(rng, 1, 8192) if op == "lora" else _log(rng, 64, 4096)
    case.update(tokens=tokens, run=1 if tokens <= 64 else _log(rng, 16, 1024),
                adapters=_log(rng, 1, 64 if tokens <= 64 else 16), none=rng.uniform(0.0, 0.3),
                rank=rng.choice([4, 8, 8, 12, 16, 16, 32, 64, 128, rng.randint(1, 64)]))
    return case


# ------------------------------------------------------------------- inputs

def _counts(case):
    """Rows of each expert: every token goes to its `top` experts of highest score."""
    deal = np.random.RandomState(case["deal"])
    score = case["skew"] * deal.standard_normal(case["experts"]) + deal.gumbel(
        size=(case["tokens"], case["experts"]))
    chosen = np.argsort(-score, axis=1)[:, :case["top"]]
    return [int(n) for n in np.bincount(chosen.ravel(), minlength=case["experts"])]


def _adapters(case):
    """The adapter of each token (-1: none): sequences of about `run` tokens, one after another."""
    deal = np.random.RandomState(case["deal"])
    of = []
    while len(of) < case["tokens"]:
        length = 1 if case["run"] == 1 else int(deal.randint(case["run"] // 2, case["run"] * 3 // 2 + 1))
        which = -1 if deal.uniform() < case["none"] else int(deal.randint(case["adapters"]))
        of += [which] * length
    return np.array(of[:case["tokens"]], dtype=np.int32)


def _activations(rows, cols, gen, dtype):
    """Normal values with a size of their own for each row and a few large columns."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x *= torch.exp(0.3 * torch.randn(rows, 1, generator=gen, device="cuda"))
    x *= torch.where(torch.rand(1, cols, generator=gen, device="cuda") < 0.01, 5.0, 1.0)
    return x.to(dtype)


def _weights(gen, dtype, size, *shape):
    w = torch.empty(shape, dtype=dtype, device="cuda")
    for part in (w if len(shape) == 3 else [w]):
        part.copy_(size * torch.randn(shape[-2:], generator=gen, device="cuda"))
    return w


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, N, K = DT[case["dtype"]], case["N"], case["K"]
    state = dict(case)
    if case["op"] in ("grouped", "wgrad"):
        counts = _counts(case)
        rows = sum(counts) + case["pad"]
        state["counts"] = counts
        state["offsets"] = torch.tensor(np.cumsum([0] + counts), dtype=torch.int32, device="cuda")
        if case["op"] == "wgrad":
            state["dy"] = _activations(rows, N, gen, dt)
            state["x"] = _activations(rows, K, gen, dt)
        else:
            state["x"] = _activations(rows, K if case["form"] == "forward" else N, gen, dt)
            state["w"] = _weights(gen, dt, 1 / math.sqrt(K), case["experts"], N, K)
        return state
    of, G, r = _adapters(case), case["adapters"], case["rank"]
    state["adapter"] = torch.from_numpy(of).cuda()
    state["rows"] = {int(g): torch.from_numpy(np.nonzero(of == g)[0]).cuda()
                     for g in np.unique(of) if g >= 0}
    state["x"] = _activations(case["tokens"], K, gen, dt)
    state["w"] = _weights(gen, dt, 1 / math.sqrt(K), N, K)
    state["a"] = _weights(gen, dt, 1 / math.sqrt(K), G, r, K)
    state["b"] = _weights(gen, dt, 0.5 / math.sqrt(r), G, N, r)
    state["scale"] = 0.5 + 1.5 * torch.rand(G, generator=gen, device="cuda")
    if case["op"] == "lora_backward":
        state["dy"] = _activations(case["tokens"], N, gen, dt)
    return state


# --------------------------------------------------------------- plain forms

def _plain_grouped(s):
    x, w = s["x"].float(), s["w"]
    forward = s["form"] == "forward"
    y = torch.zeros(x.shape[0], s["N"] if forward else s["K"], device=x.device)
    row = 0
    for g, n in enumerate(s["counts"]):
        if n:
            wg = w[g].float()
            y[row:row + n] = x[row:row + n] @ (wg.t() if forward else wg)
        row += n
    return y.to(DT[s["out"]])


def _plain_wgrad(s):
    out = torch.zeros(s["experts"], s["N"], s["K"], device=s["x"].device)
    row = 0
    for g, n in enumerate(s["counts"]):
        if n:
            out[g] = s["dy"][row:row + n].float().t() @ s["x"][row:row + n].float()
        row += n
    return out.to(DT[s["out"]])


def _plain_lora(s):
    x, a, b = s["x"].float(), s["a"], s["b"]
    y = x @ s["w"].float().t()
    if x.shape[0] <= 256:  # few tokens: each with its own copy of an adapter
        of = s["adapter"].long()
        g = of.clamp_min(0)
        t = torch.bmm(a[g].float(), x[:, :, None])
        d = torch.bmm(b[g].float(), t)[:, :, 0] * s["scale"][g][:, None]
        y += torch.where(of[:, None] >= 0, d, torch.zeros_like(d))
        return y.to(DT[s["out"]])
    for g, rows in s["rows"].items():
        t = (x[rows] @ a[g].float().t()) * s["scale"][g]
        y[rows] += t @ b[g].float().t()
    return y.to(DT[s["out"]])


def _plain_lora_backward(s):
    x, dy = s["x"].float(), s["dy"].float()
    a, b, scale = s["a"], s["b"], s["scale"]
    dx = dy @ s["w"].float()
    da, db = torch.zeros(a.shape, device=x.device), torch.zeros(b.shape, device=x.device)
    for g, rows in s["rows"].items():
        ag, bg, xr, dyr = a[g].float(), b[g].float(), x[rows], dy[rows]
        u = (dyr @ bg) * scale[g]
        dx[rows] += u @ ag
        da[g] = u.t() @ xr
        db[g] = dyr.t() @ ((xr @ ag.t()) * scale[g])
    return {"dx": dx.to(DT[s["out"]]), "da": da, "db": db}


_PLAIN = {"grouped": _plain_grouped, "wgrad": _plain_wgrad, "lora": _plain_lora,
          "lora_backward": _plain_lora_backward}


def run(state):
    s = state
    if not own:
        return _PLAIN[s["op"]](s)
    import tiled_matrix_multiplication_output_gb300 as tg
    out = DT[s["out"]]
    if s["op"] == "grouped":
        return tg.matmul_grouped(s["x"], s["w"], s["offsets"],
                                 op_b="t" if s["form"] == "forward" else "n", out_dtype=out)
    if s["op"] == "wgrad":
        return tg.matmul_grouped_wgrad(s["dy"], s["x"], s["offsets"], out_dtype=out)
    if s["op"] == "lora":
        return tg.matmul_lora(s["x"], s["w"], s["a"], s["b"], s["adapter"], scale=s["scale"],
                              out_dtype=out)
    dx, da, db = tg.matmul_lora_backward(s["dy"], s["x"], s["w"], s["a"], s["b"], s["adapter"],
                                         scale=s["scale"], out_dtype=out,
                                         grad_dtype=torch.float32)
    return {"dx": dx, "da": da, "db": db}


# --------------------------------------------------------------------- work

def work(case):
    N, K, el, out = case["N"], case["K"], SIZE[case["dtype"]], SIZE[case["out"]]
    if case["op"] in ("grouped", "wgrad"):
        counts = _counts(case)
        rows, hit = sum(counts), sum(n > 0 for n in counts)
        if case["op"] == "wgrad":
            moved = rows * (N + K) * el + case["experts"] * N * K * out
        else:
            n_in, n_out = (K, N) if case["form"] == "forward" else (N, K)
            moved = rows * n_in * el + hit * N * K * el + (rows + case["pad"]) * n_out * out
        return {"bytes": moved, "flops": 2 * rows * N * K}
    of = _adapters(case)
    M, r = case["tokens"], case["rank"]
    held, with_one = len(set(of[of >= 0].tolist())), int((of >= 0).sum())
    thin = 2 * with_one * r * (N + K)  # one pass of the rows through one pair of factors
    adapters = held * r * (N + K) * el
    if case["op"] == "lora":
        return {"bytes": (M * K + N * K) * el + adapters + M * N * out,
                "flops": 2 * M * N * K + thin}
    return {"bytes": (M * N + M * K + N * K) * el + adapters + M * K * out
            + case["adapters"] * r * (N + K) * 4,
            "flops": 2 * M * N * K + thin * 2 + 2 * with_one * r * K}


# -------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("grouped", "wgrad"):
        ends = s["offsets"].tolist()
        spans = [slice(b, e) for b, e in zip(ends, ends[1:])]
        if case["op"] == "wgrad":
            # a sum over each expert's rows, in parts
            out = s["x"].new_zeros((len(spans), case["N"], case["K"]), dtype=torch.float64)
            for g, span in enumerate(spans):
                for r0 in range(span.start, span.stop, 2048):
                    part = slice(r0, min(r0 + 2048, span.stop))
                    out[g].addmm_(s["dy"][part].double().mT, s["x"][part].double())
            return out
        eq = "mk,nk->mn" if case["form"] == "forward" else "mn,nk->mk"
        parts = [torch.einsum(eq, s["x"][span].double(), s["w"][g].double())
                 for g, span in enumerate(spans)]
        parts.append(parts[0].new_zeros(case["pad"], parts[0].shape[1]))
        return torch.cat(parts)
    # every token's weight is W + scale B A of its adapter: the change of one adapter at a time,
    # times rows that are zero for the tokens of the others
    x, w, of = s["x"].double(), s["w"].double(), s["adapter"]
    G = case["adapters"]
    mine = [(of == g)[:, None].double() for g in range(G)]
    if case["op"] == "lora":
        y = x @ w.mT
        for g in range(G):
            y += (x * mine[g]) @ s["a"][g].double().mT @ (s["b"][g].double().mT * s["scale"][g].double())
        return y
    dy = s["dy"].double()
    dx, da, db = dy @ w, [], []
    for g in range(G):
        a, b, k = s["a"][g].double(), s["b"][g].double(), s["scale"][g].double()
        d = dy * mine[g]
        dx += k * (d @ b) @ a
        da.append(k * torch.einsum("mr,mk->rk", d @ b, x))
        db.append(k * torch.einsum("mn,mr->nr", d, x @ a.mT))
    return {"dx": dx, "da": torch.stack(da), "db": torch.stack(db)}
