"""Helpers of the layer operators' tests: rows on the device in each format,
and the checks of outputs against the 64-bit forms of oracle/layer.py."""
import numpy as np
import torch

from collective_synchronization_amd import abi, buffers
from oracle import layer

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def to_type(v, fmt):
    """Values rounded to a float format, as binary64."""
    return torch.from_numpy(np.asarray(v, dtype=np.float32)).to(TORCH[fmt]).double().numpy()


def float_rows(v, fmt, extra=0, device="cuda"):
    """Rows of values on the device with `extra` * 8 elements of stride past
    the row; what lies past the row is NaN, which nothing may read."""
    rows, cols = v.shape
    r = buffers.FormatRows(rows, cols, fmt, device)
    if extra:
        r.stride += 8 * extra
        r.data = torch.zeros((rows, r.stride), dtype=TORCH[fmt], device=device)
    host = torch.full((rows, r.stride), float("nan"), dtype=TORCH[fmt])
    host[:, :cols] = torch.from_numpy(np.asarray(v, dtype=np.float64)).to(TORCH[fmt])
    r.data.copy_(host)
    return r


def code_rows(codes, scales, fmt, cols, extra=0, device="cuda"):
    """8- or 4-bit rows on the device from element codes (one a byte, whole
    blocks for the MX formats); what lies past the row's last element, in its
    last block and after it, and past the scales is the worst there is."""
    rows = codes.shape[0]
    r = buffers.FormatRows(rows, cols, fmt, device)
    r.stride += 16 * extra
    host = np.full((rows, r.stride), 0xFF, dtype=np.uint8)
    codes = codes.copy()
    codes[:, cols:] = 15 if fmt == "mx4" else 0x7F     # -6, or NaN: nobody may use them
    packed = layer.pack4(codes) if fmt == "mx4" else codes
    host[:, :packed.shape[1]] = packed
    r.data = torch.from_numpy(host).to(device)
    if fmt == "row8":
        r.scales = torch.from_numpy(np.asarray(scales, dtype=np.float32)).to(device)
    else:
        r.scale_stride += 4 * extra
        sc = np.full((rows, r.scale_stride), 0xFF, dtype=np.uint8)
        sc[:, :scales.shape[1]] = scales
        r.scales = torch.from_numpy(sc).to(device)
    return r


def out_rows(rows, cols, fmt, device="cuda"):
    """Output rows filled with a pattern that no output has, one stride step
    wider than a row."""
    r = buffers.FormatRows(rows, cols, fmt, device)
    if fmt in TORCH:
        r.stride += 8
        r.data = torch.full((rows, r.stride), -77.0, dtype=TORCH[fmt], device=device)
    else:
        r.stride += 16
        r.data = torch.full((rows, r.stride), 0xA5, dtype=torch.uint8, device=device)
        if fmt == "row8":
            r.scales.fill_(-77.0)
        else:
            r.scale_stride += 4
            r.scales = torch.full((rows, r.scale_stride), 0xA5, dtype=torch.uint8, device=device)
    return r


def untouched(r):
    """Nothing past what a row takes has been written."""
    fmt = {v: k for k, v in abi.FORMATS.items()}[r.fmt]
    if fmt in TORCH:
        return bool((r.data[:, r.cols:] == -77.0).all())
    nb = -(-r.cols // 32)
    taken = r.cols if fmt == "row8" else (16 * nb if fmt == "mx4" else 32 * nb)
    ok = bool((r.data[:, taken:] == 0xA5).all())
    if fmt != "row8":
        ok = ok and bool((r.scales[:, nb:] == 0xA5).all())
    return ok


def read_codes(r, fmt):
    """(element codes one a byte, scales) of device rows."""
    nb = -(-r.cols // 32)
    d = r.data.cpu().numpy()
    if fmt == "row8":
        return d[:, :r.cols], r.scales.cpu().numpy()
    sc = r.scales.cpu().numpy()[:, :nb]
    return (layer.unpack4(d[:, :16 * nb]) if fmt == "mx4" else d[:, :32 * nb]), sc


def check_float(got, want, fmt, rel, absolute=0.0):
    """got within one rounding of its type and `rel` of the 64-bit result."""
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want)
    lim = {"bf16": 2.0 ** 128 - 2.0 ** 119, "f16": 65520.0, "f32": 2.0 ** 128 - 2.0 ** 103}[fmt]
    inside = np.isfinite(want) & (np.abs(want) * (1 + rel) < lim)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    tiny = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}[fmt]
    tol = np.abs(want) * (rel + (1 + rel) * layer.HALF_STEP[fmt]) + tiny + absolute
    bad = inside & ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


def _signed_key(codes, fmt):
    """Element codes in the order of their values (-0 and 0 equal)."""
    c = codes.astype(np.int64)
    mag = c & (7 if fmt == "mx4" else 127)
    return np.where(c & (8 if fmt == "mx4" else 128), -mag, mag)


def check_quantized(r, fmt, v, rel):
    """8- or 4-bit rows of values known to `rel`: every scale lies between
    those of the smallest and the largest value it may come from, and every
    code between those of the smallest and largest value for that scale."""
    got, sc = read_codes(r, fmt)
    cols = r.cols
    assert untouched(r)
    small, large = v - np.abs(v) * rel, v + np.abs(v) * rel
    if fmt == "row8":
        amax = np.abs(v).max(-1)
        nan = ~np.isfinite(amax)
        assert np.array_equal(np.isnan(sc), nan)
        assert (got[nan] == 0x7F).all()
        ok = ~nan
        want = np.maximum(amax[ok] / 448.0, 2.0 ** -126)
        # one division, the row's maximum, then 1/s and the product with it
        assert (np.abs(sc[ok] - want) <= want * (rel + 2.0 ** -23)).all()
        s = sc[ok].astype(np.float64)[:, None]
        lo = layer.signed_codes((small[ok] - np.abs(v[ok]) * 2.0 ** -22) / s, layer.E4M3, 128)
        hi = layer.signed_codes((large[ok] + np.abs(v[ok]) * 2.0 ** -22) / s, layer.E4M3, 128)
        got = got[ok]
    else:
        b = np.abs(layer.blocks_of(v))
        with np.errstate(invalid="ignore"):
            amax = b.max(-1)
        amax = np.where(np.isnan(amax), np.inf, amax)
        first, last = (layer.scale_codes(amax * (1 - rel), fmt), layer.scale_codes(amax * (1 + rel), fmt))
        assert ((sc >= first) & (sc <= last)).all(), (sc, first, last)
        nan = np.repeat(sc == 255, 32, axis=1)
        assert (got[nan] == (0 if fmt == "mx4" else 0x7F)).all()
        assert (got[:, cols:][~nan[:, cols:]] == 0).all()
        safe = np.where(nan[:, :cols], 0.0, v)
        lo = layer.codes_with_scales(np.where(nan[:, :cols], 0.0, small) if rel else safe, sc, fmt)
        hi = layer.codes_with_scales(np.where(nan[:, :cols], 0.0, large) if rel else safe, sc, fmt)
        lo, hi, got = (np.where(nan, 0, x) for x in (lo, hi, got))
    k, l, h = (_signed_key(x, fmt) for x in (got, lo, hi))
    bad = (k < l) | (k > h)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], lo[bad][:5], hi[bad][:5])
