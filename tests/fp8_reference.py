"""Plain 64-bit forms of the block-scaled 8-bit operators, from their
definitions, for the tests (numpy; nothing of the package is used)."""
from __future__ import annotations

import numpy as np

F8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
MANTISSA = {"e4m3": (3, -6), "e5m2": (2, -14)}     # stored mantissa bits, least normal exponent
BLOCK = {"row": (1, 128), "col": (128, 1), "tile": (128, 128)}


def round8(v: np.ndarray, f8: str) -> np.ndarray:
    """Nearest 8-bit value, ties to even, saturating; NaN stays NaN."""
    bits, low = MANTISSA[f8]
    v = np.asarray(v, np.float64)
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(v)
        unit = np.ldexp(1.0, np.maximum(e - 1, low) - bits)
        return np.clip(np.rint(v / unit) * unit, -F8_MAX[f8], F8_MAX[f8])


def spread(s: np.ndarray, rows: int, cols: int, block: str) -> np.ndarray:
    """The scale of every element, from scales as the library stores them."""
    if block == "row":
        s = s.T
    br, bc = BLOCK[block]
    return np.repeat(np.repeat(s, br, 0), bc, 1)[:rows, :cols]


def quantize(x: np.ndarray, block: str, f8: str):
    """(code values, scales as stored) of a 2-D array whose values are exact
    in FP32.  Every rounding to FP32 of the definition is made explicitly."""
    x32 = np.asarray(x, np.float32)
    rows, cols = x32.shape
    br, bc = BLOCK[block]
    pad = np.pad(x32, ((0, -rows % br), (0, -cols % bc)))
    v = pad.reshape(pad.shape[0] // br, br, pad.shape[1] // bc, bc)
    amax = np.where(np.isfinite(v), np.abs(v), np.float32(0)).max(axis=(1, 3))
    inv_max = np.float32(1.0 / F8_MAX[f8])
    s = np.where(amax > 0, np.maximum(amax * inv_max, np.float32(2.0 ** -126)), np.float32(1))
    r = np.float32(1) / s
    with np.errstate(invalid="ignore", over="ignore"):
        t = v * r[:, None, :, None]
    t = np.where(np.isfinite(v), t, np.float32(np.nan)).astype(np.float64)
    q = round8(t, f8).reshape(pad.shape)[:rows, :cols]
    return q, (s.T if block == "row" else s)


def product(qa, sa, block_a, op_a, qb, sb, block_b, op_b):
    """(sum, sum of magnitudes) of op(A) @ op(B) in 64 bits."""
    a = qa.astype(np.float64) * spread(sa.astype(np.float64), *qa.shape, block_a)
    b = qb.astype(np.float64) * spread(sb.astype(np.float64), *qb.shape, block_b)
    a = a.T if op_a == "t" else a
    b = b.T if op_b == "t" else b
    return a @ b, np.abs(a) @ np.abs(b)


def product_bound(cabs: np.ndarray, cref: np.ndarray, K: int, half_ulp: float) -> np.ndarray:
    """How far an FP32-accumulated result may be off: a sum of 128 terms, the
    scales' product, its product with the block's sum, a sum over the blocks,
    alpha and beta -- each step at most one unit in the last place of FP32
    (2^-23, whether it rounds or truncates) of the sum of magnitudes -- and
    one rounding to the output type (plus the least subnormal of FP16)."""
    blocks = -(-K // 128)
    return (128 + blocks + 6) * 2.0 ** -23 * cabs + half_ulp * np.abs(cref) + 2.0 ** -25
