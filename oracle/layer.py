"""Plain 64-bit forms of the layer operators (test infrastructure only).

numpy binary64 throughout, from the definitions alone: the residual norm, the
8- and 4-bit row formats and the linear layer.  Nothing is shared with the
product.  Formats go by name: bf16, f16, f32, row8 (e4m3 codes, one binary32
scale a row), mx8 (e4m3 codes, one e8m0 scale for 32 elements), mx4 (e2m1).
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
# every non-negative value of the formats, by code
E4M3 = np.array([m / 512 for m in range(8)] +
                [2.0 ** (e - 7) * (1 + m / 8) for e in range(1, 16) for m in range(8)][:-1])
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
EMAX = {"mx8": 8, "mx4": 2}
GRID = {"row8": E4M3, "mx8": E4M3, "mx4": E2M1}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


def nearest_code(a, grid):
    """Code of the nearest grid value to each a >= 0 (ties: the even code; past
    the last value: the last)."""
    a = np.asarray(a, dtype=np.float64)
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = np.searchsorted(mid, a, "left"), np.searchsorted(mid, a, "right")
    return np.where(lo % 2 == 0, lo, hi)


def signed_codes(v, grid, sign_bit):
    code = nearest_code(np.abs(v), grid)
    return (code + np.where(np.signbit(v), sign_bit, 0)).astype(np.uint8)


def blocks_of(v):
    """[rows, cols] -> [rows, blocks, 32], zeros behind the last column."""
    rows, cols = v.shape
    nb = -(-cols // BLOCK)
    out = np.zeros((rows, nb * BLOCK))
    out[:, :cols] = v
    return out.reshape(rows, nb, BLOCK)


def scale_codes(amax, fmt):
    """e8m0 codes from the blocks' largest magnitudes."""
    amax = np.asarray(amax, dtype=np.float64)
    fine = np.isfinite(amax)
    _, e = np.frexp(np.where(fine & (amax > 0), amax, 1.0))      # amax = f * 2^e, f in [1/2, 1)
    code = np.where(amax > 0, np.clip(e - 1 - EMAX[fmt], -127, 127) + 127, 0)
    return np.where(fine, code, 255).astype(np.uint8)


def scale_values(codes):
    c = np.asarray(codes).astype(np.int64)
    return np.where(c == 255, np.nan, np.ldexp(1.0, np.where(c == 255, 0, c - 127)))


def codes_with_scales(v, codes, fmt):
    """Element codes (one a byte) of v for given scale codes, whole blocks."""
    b = blocks_of(v)
    nan = codes == 255
    s = np.where(nan, 1.0, scale_values(np.where(nan, 127, codes)))[..., None]
    bit = 128 if fmt == "mx8" else 8
    q = signed_codes(np.where(nan[..., None], 0.0, b) / s, GRID[fmt], bit)
    q = np.where(nan[..., None], 127 if fmt == "mx8" else 0, q).astype(np.uint8)
    return q.reshape(v.shape[0], -1)


def quantize(v, fmt):
    """(element codes one a byte, whole blocks; scale codes) of an MX format."""
    v = np.asarray(v, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        amax = np.abs(blocks_of(v)).max(-1)
    sc = scale_codes(np.where(np.isnan(amax), np.inf, amax), fmt)
    return codes_with_scales(v, sc, fmt), sc


def code_values(codes, fmt):
    """What element codes (one a byte) stand for, scales apart."""
    c = np.asarray(codes).astype(np.int64)
    if fmt == "mx4":
        return np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]
    mag = c & 127
    return np.where(mag == 127, np.nan, np.where(c & 128, -1.0, 1.0) * E4M3[np.minimum(mag, 126)])


def dequantize(codes, scales, fmt, cols):
    v = code_values(codes, fmt)
    if fmt == "row8":
        return v[:, :cols] * np.asarray(scales, dtype=np.float64)[:, None]
    return (v * np.repeat(scale_values(scales), BLOCK, axis=1))[:, :cols]


def pack4(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack4(packed):
    out = np.empty(packed.shape[:-1] + (2 * packed.shape[-1],), dtype=np.uint8)
    out[..., 0::2], out[..., 1::2] = packed & 15, packed >> 4
    return out


def norm(h, gamma, eps):
    """v of rows h (binary64)."""
    r = 1.0 / np.sqrt((h * h).sum(-1, keepdims=True) / h.shape[-1] + eps)
    return h * r * (1.0 if gamma is None else gamma)


def rank_sum_f32(x):
    """binary32 sum of rows [ranks, ...] in rank order."""
    acc = np.array(x[0], dtype=np.float32)
    for r in range(1, len(x)):
        acc = (acc + x[r].astype(np.float32)).astype(np.float32)
    return acc


def linear(x, w):
    """[ranks, m, k] x [ranks, n, k] -> [ranks, m, n]."""
    return np.stack([x[r] @ w[r].T for r in range(x.shape[0])])
