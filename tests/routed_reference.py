"""64-bit forms of the products grouped by rows and of the low-rank adapters,
from their definitions, with bounds on what FP32 sums and one rounding may
differ from them, for the tests (torch only; nothing of the package is used)."""
from __future__ import annotations

import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def sums_bound(terms: int) -> float:
    """Relative to the sum of magnitudes: an FP32 sum of `terms` products in any
    order, where a tensor-core step of 16 products counts as 17 additions."""
    return (1.1 * terms + 32) * 2.0 ** -24


def rounding_bound(ref, dtype):
    """Half a step of the type at each value (and half its least step)."""
    info = torch.finfo(dtype)
    return ref.abs() * (info.eps / 2) + info.smallest_normal * info.eps / 2


def clean(offsets, rows):
    """Ascending offsets within [0, rows]: each the largest of those up to it."""
    out, top = [], 0
    for v in offsets:
        top = max(top, min(max(int(v), 0), rows))
        out.append(top)
    return out


def grouped(x, w, offsets, w_t, alpha=1.0, beta=0.0, y=None):
    """(values, bound of the FP32 sums, rows of a group) in 64 bits."""
    x, w = x.double(), w.double()
    rows, n = x.shape[0], w.shape[1] if w_t else w.shape[2]
    out = torch.zeros(rows, n, dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(out)
    in_group = torch.zeros(rows, dtype=torch.bool, device=x.device)
    ends = clean(offsets, rows)
    for g, (b, e) in enumerate(zip(ends, ends[1:])):
        m = w[g].t() if w_t else w[g]
        out[b:e] = alpha * (x[b:e] @ m)
        mag[b:e] = abs(alpha) * (x[b:e].abs() @ m.abs())
        in_group[b:e] = True
    if beta != 0.0:
        out = out + beta * y.double()
        mag = mag + abs(beta) * y.double().abs()
    return out, mag * sums_bound(x.shape[1]), in_group


def wgrad(dy, x, offsets, alpha=1.0, beta=0.0, c=None):
    dy, x = dy.double(), x.double()
    ends = clean(offsets, x.shape[0])
    spans = list(zip(ends, ends[1:]))
    shape = (len(spans), dy.shape[1], x.shape[1])
    out = torch.zeros(shape, dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(out)
    for g, (b, e) in enumerate(spans):
        out[g] = alpha * (dy[b:e].t() @ x[b:e])
        mag[g] = abs(alpha) * (dy[b:e].abs().t() @ x[b:e].abs())
    if beta != 0.0:
        out = out + beta * c.double()
        mag = mag + abs(beta) * c.double().abs()
    terms = max([e - b for b, e in spans] + [0])
    return out, mag * sums_bound(terms)


def parts_bound(dtype, out_dtype) -> float:
    """Relative: what the rank values lose on entering the second product."""
    if dtype == torch.float32:
        return 0.0
    if dtype == torch.float16:
        return 2.0 ** -22
    return 2.0 ** -24 if out_dtype == torch.float32 else 2.0 ** -16


def _each(adapter, adapters):
    for g in range(adapters):
        rows = torch.nonzero(adapter == g)[:, 0]
        if len(rows):
            yield g, rows


def _values(x, f, scale, g):
    """Rank values of rows x through factor f (rank x in), and their magnitudes' sums."""
    s = 1.0 if scale is None else float(scale[g])
    return s * (x @ f.t()), abs(s) * (x.abs() @ f.abs().t())


def _beside(x, w, down, up, adapter, scale, dtype, out_dtype):
    """x w + (rank values) up, per row's adapter; w: in x out, down: rank x in, up: rank x out."""
    out, mag = x @ w, x.abs() @ w.abs()
    G, r = down.shape[:2]
    err = torch.zeros_like(mag)
    for g, rows in _each(adapter, G):
        t, tm = _values(x[rows], down[g], scale, g)
        out[rows] += t @ up[g]
        d = tm @ up[g].abs()
        mag[rows] += d
        err[rows] += (sums_bound(x.shape[1]) + 2.0 ** -23 + parts_bound(dtype, out_dtype)) * d
        if dtype == torch.float16:
            # the second part is a multiple of FP16's least step, 2^-24: it leaves up to half
            # of that of a rank value, however small the value is
            err[rows] += 2.0 ** -25 * up[g].abs().sum(0)
    return out, err + mag * sums_bound(x.shape[1] + 3 * r)


def lora(x, w, a, b, adapter, scale, out_dtype):
    dtype = x.dtype
    x, w, a, b = (t.double() for t in (x, w, a, b))
    return _beside(x, w.t(), a, b.transpose(1, 2), adapter, scale, dtype, out_dtype)


def lora_backward(dy, x, w, a, b, adapter, scale, out_dtype):
    """((dx, bound), (da, bound), (db, bound))."""
    dtype = x.dtype
    dy, x, w, a, b = (t.double() for t in (dy, x, w, a, b))
    dx = _beside(dy, w, b.transpose(1, 2), a, adapter, scale, dtype, out_dtype)
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    ea, eb = torch.zeros_like(a), torch.zeros_like(b)
    part = parts_bound(dtype, torch.float32) + 2.0 ** -23
    for g, rows in _each(adapter, a.shape[0]):
        u, um = _values(dy[rows], b[g].t(), scale, g)
        t, tm = _values(x[rows], a[g], scale, g)
        da[g], db[g] = u.t() @ x[rows], dy[rows].t() @ t
        n = sums_bound(3 * len(rows)) + part
        ea[g] = (n + sums_bound(dy.shape[1])) * (um.t() @ x[rows].abs())
        eb[g] = (n + sums_bound(x.shape[1])) * (dy[rows].abs().t() @ tm)
    return dx, (da, ea), (db, eb)


def check(got, ref, bound):
    """|got - ref| within the bound of the sums plus one rounding to got's type."""
    assert got.shape == ref.shape
    limit = bound * (1 + torch.finfo(got.dtype).eps) + rounding_bound(ref, got.dtype)
    err = (got.double() - ref).abs()
    bad = ~(err <= limit)
    if bad.any():
        at = torch.nonzero(bad)
        raise AssertionError(f"{len(at)} of {got.numel()} values out of bound, first at "
                             f"{at[0].tolist()}: {got[tuple(at[0])]} against {ref[tuple(at[0])]} "
                             f"(within {limit[tuple(at[0])]}), last at {at[-1].tolist()}")
