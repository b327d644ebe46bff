"""The residual norm where single roundings show: the ends of the range, and
values beside the border between two codes.

The kernel's r is right to 2^-50 and its products to 2^-46 before they are
rounded (to binary32, or for the MX formats to odd, which keeps every border
between two codes), so its outputs, those of 16-bit types apart, are those of the
64-bit form but where that lies within 2^-46 of a border.  The 64-bit form's own sum and products are off by
less than 2^-48.  NEAR covers both.
"""
import numpy as np
import pytest
import torch

from collective_synchronization_amd import abi
from layer_cases import TORCH, check_float, check_quantized, float_rows, out_rows, to_type, untouched
from oracle import layer

pytestmark = pytest.mark.gpu

NEAR = 2.0 ** -46
REL = 64 * 2.0 ** -24            # a row's steps when each is a binary32 one


def run(x, fmt, y_fmt, gamma=None, eps=0.0, res=None, res_fmt=None):
    """y rows of the norm of x (+ res), with gamma."""
    rows, cols = x.shape
    xd = float_rows(x, fmt)
    rd = float_rows(res, res_fmt) if res is not None else None
    y = out_rows(rows, cols, y_fmt)
    g = torch.from_numpy(np.asarray(gamma)).to(TORCH[fmt]).to("cuda") if gamma is not None else None
    p = abi.norm_params(rows, cols, eps, fmt, g, res_fmt or fmt, rd.data if rd else None,
                        rd.stride if rd else 0, None, 0, y_fmt, y.data, y.stride, y.scales,
                        y.scale_stride)
    abi.ar_residual_norm(p, xd.data, xd.stride)
    torch.cuda.synchronize()
    return y


@pytest.mark.parametrize("y_fmt", ("same", "row8", "mx8", "mx4"))
@pytest.mark.parametrize("fmt", ("f32", "bf16"))
@pytest.mark.parametrize("cols", (40, 4096, 12000))
def test_rows_at_the_ends_of_the_range(cols, fmt, y_fmt):
    """Rows whose mean square leaves binary32's range either way: v is of
    the order of 1 all the same."""
    rng = np.random.default_rng(cols)
    sizes = np.array([1e19, 3e19, 1e25, 5e37, 1e-18, 1e-19, 3e-21, 1e-22, 1e-23, 1e-30, 2e-37, 1.0])
    x = to_type(np.clip(rng.standard_normal((len(sizes), cols)), -6, 6) * sizes[:, None], fmt)
    y_fmt = fmt if y_fmt == "same" else y_fmt
    y = run(x, fmt, y_fmt)
    v = layer.norm(x, None, 0.0)
    if y_fmt in TORCH:
        check_float(y.data[:, :cols].double().cpu().numpy(), v, y_fmt, REL)
    else:
        check_quantized(y, y_fmt, v, REL)
    assert untouched(y)


def test_subnormal_rows():
    """Rows of binary32's smallest numbers, eps 0."""
    x = np.ldexp(np.arange(1.0, 65.0)[None], np.array([[-149], [-140], [-131]]))
    y = run(x, "f32", "f32")
    check_float(y.data[:, :64].double().cpu().numpy(), layer.norm(x, None, 0.0), "f32", REL)


def test_eps_beside_a_small_mean_square():
    """A mean square below binary32's range and an eps like it."""
    rng = np.random.default_rng(2)
    x = to_type(rng.standard_normal((4, 300)) * 1e-20, "f32")
    eps = np.float32(1e-40)
    y = run(x, "f32", "f32", eps=float(eps))
    check_float(y.data[:, :300].double().cpu().numpy(), layer.norm(x, None, float(eps)), "f32", REL)


def _beside_borders(rng, cols, fmt, s):
    """(x, gamma) of one binary32 row, eps 0, whose values in units of 2^s lie
    within half a binary32 step of the format's borders, on either side; the
    first of each 32 is the block's largest.  gamma is the binary32 number
    nearest to border / (h * r)."""
    grid = layer.GRID[fmt]
    borders = (grid[1:] + grid[:-1]) / 2
    x = to_type(rng.uniform(1.0, 2.0, (1, cols)) * rng.choice([-1.0, 1.0], (1, cols)), "f32")
    b = rng.choice(borders, cols)
    b[::32] = 1.25 * 2.0 ** layer.EMAX[fmt]
    r = 1.0 / np.sqrt((x * x).sum() / cols)
    return x, to_type(np.ldexp(b / (np.abs(x[0]) * r), s), "f32")


@pytest.mark.parametrize("fmt", ("mx8", "mx4"))
@pytest.mark.parametrize("s", (0, 60, -20, -58, -61, -70, -95, -110, -118, -125, -127))
def test_codes_beside_borders(s, fmt):
    rng = np.random.default_rng(200 + s)
    cols = 16384
    x, gamma = _beside_borders(rng, cols, fmt, s)
    y = run(x, "f32", fmt, gamma=gamma)
    check_quantized(y, fmt, layer.norm(x, gamma, 0.0), NEAR)


@pytest.mark.parametrize("y_fmt", ("mx8", "mx4"))
@pytest.mark.parametrize("fmt,res_fmt", (("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32")))
@pytest.mark.parametrize("rows,cols", ((400, 4096), (60, 8200), (2000, 520), (70, 30011)))
def test_codes_of_ordinary_rows(rows, cols, fmt, res_fmt, y_fmt):
    """Every code and scale is the 64-bit form's."""
    rng = np.random.default_rng(rows + cols)
    x = to_type(rng.standard_normal((rows, cols)), fmt)
    res = to_type(rng.standard_normal((rows, cols)) * 2, res_fmt)
    gamma = to_type(rng.uniform(0.5, 1.5, cols), fmt)
    eps = np.float32(1e-5)
    y = run(x, fmt, y_fmt, gamma=gamma, eps=float(eps), res=res, res_fmt=res_fmt)
    h = (res.astype(np.float32) + x.astype(np.float32)).astype(np.float64)
    check_quantized(y, y_fmt, layer.norm(h, gamma, float(eps)), NEAR)


@pytest.mark.parametrize("y_fmt", ("mx8", "mx4", "row8"))
def test_zeros_among_values(y_fmt):
    """Zeros in the row and in gamma, small products and a gamma that takes a
    value past binary32's range: the block of that one is NaN."""
    cols = 320
    rng = np.random.default_rng(5)
    x = to_type(rng.standard_normal((3, cols)), "f32")
    x[0, ::3] = 0.0
    x[1, 64:] = -0.0
    x[2, 5] = 2.0 ** -140
    gamma = to_type(rng.uniform(0.5, 1.5, cols), "f32")
    gamma[::5] = 0.0
    gamma[5], gamma[100], gamma[130] = 2.0 ** 100, 2.0 ** -120, 2.0 ** 126
    x[2, 130] = 60.0
    y = run(x, "f32", y_fmt, gamma=gamma)
    with np.errstate(over="ignore"):
        v = layer.norm(x, gamma, 0.0)
    v = np.where(np.abs(v) >= 2.0 ** 128, np.inf, v)
    assert np.isinf(v[2, 130])
    check_quantized(y, y_fmt, v, NEAR)


# significant bits, exponent of the smallest normal number, largest finite value
TYPES = {"bf16": (8, -126, 2.0 ** 128 - 2.0 ** 120), "f16": (11, -14, 65504.0), "f32": (24, -126, 2.0 ** 128 - 2.0 ** 104)}


def rounded(v, fmt):
    """binary64 values to a float type, nearest even, in one rounding."""
    bits, emin, largest = TYPES[fmt]
    _, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(e - 1, emin) - bits + 1)
    q = np.rint(v / step) * step                       # exact: a power of two
    return np.where(np.abs(q) > largest, np.copysign(np.inf, q), q)


def check_float_rows(y, v):
    """Every output lies between the roundings of v a little smaller and larger:
    for binary32 by the 64-bit form's own error, for 16-bit types by r's
    rounding to binary32 and that of two products, 3 * 2^-24.  Below 2^-100 the
    correction of binary32's last bit is lost: one step more."""
    fmt = {k: f for f, k in abi.FORMATS.items()}[y.fmt]
    got = y.data[:, :y.cols].double().cpu().numpy()
    rel = np.where(np.abs(v) < 2.0 ** -100, 2.0 ** -22, NEAR) if fmt == "f32" else 3 * 2.0 ** -24
    off = np.abs(v) * rel + np.where(np.abs(v) < 2.0 ** -100, 2.0 ** -149, 0.0)
    with np.errstate(invalid="ignore"):
        lo, hi = rounded(v - off, fmt), rounded(v + off, fmt)
    bad = ~((got >= lo) & (got <= hi)) & ~(np.isnan(got) & np.isnan(v))
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], v[bad][:5])
    assert untouched(y)


@pytest.mark.parametrize("fmt,res_fmt", (("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32")))
@pytest.mark.parametrize("rows,cols", ((400, 4096), (60, 8200), (2000, 523), (70, 30011)))
def test_float_rows(rows, cols, fmt, res_fmt):
    rng = np.random.default_rng(rows + cols)
    x = to_type(rng.standard_normal((rows, cols)), fmt)
    res = to_type(rng.standard_normal((rows, cols)) * 2, res_fmt)
    gamma = to_type(rng.uniform(0.5, 1.5, cols), fmt)
    eps = np.float32(1e-5)
    y = run(x, fmt, fmt, gamma=gamma, eps=float(eps), res=res, res_fmt=res_fmt)
    h = (res.astype(np.float32) + x.astype(np.float32)).astype(np.float64)
    check_float_rows(y, layer.norm(h, gamma, float(eps)))


@pytest.mark.parametrize("s", (0, 100, -30, -95, -110, -124, -128, -134))
@pytest.mark.parametrize("fmt", ("bf16", "f16", "f32"))
def test_float_values_beside_borders(fmt, s):
    """Of 40 gammas for each element the one whose product comes nearest to the
    border between two neighbours of the type, in sizes from 2^100 to its
    subnormal numbers."""
    if fmt == "f16":
        if s > 0 or s < -30:
            pytest.skip("past the type's range")
        s = max(s, -16)
    rng = np.random.default_rng(300 + s)
    cols = 32768
    x = to_type(rng.uniform(1.0, 2.0, (1, cols)) * rng.choice([-1.0, 1.0], (1, cols)), fmt)
    r = 1.0 / np.sqrt((x * x).sum() / cols)
    bits, emin, _ = TYPES[fmt]
    g = to_type(np.ldexp(rng.uniform(0.7, 1.4, (40, cols)), s), fmt)
    step = np.ldexp(1.0, np.maximum(np.frexp(x * r * g)[1] - 1, emin) - bits + 1)
    off = np.abs(x * r * g / step % 1.0 - 0.5)
    gamma = g[off.argmin(0), np.arange(cols)]
    y = run(x, fmt, fmt, gamma=gamma)
    check_float_rows(y, layer.norm(x, gamma, 0.0))


def test_infinite_products_are_infinite():
    """v past the type's range, next to zeros."""
    x = np.ones((1, 64))
    x[0, 0], x[0, 1], x[0, 2] = 4.0, 0.0, -4.0
    gamma = np.ones(64)
    gamma[[0, 2, 5]] = 3.3e38
    for fmt in ("bf16", "f32"):
        xs, gs = to_type(x, fmt), to_type(gamma, fmt)
        y = run(xs, fmt, fmt, gamma=gs)
        check_float_rows(y, layer.norm(xs, gs, 0.0))
        got = y.data[0, :64].double().cpu().numpy()
        assert got[0] == np.inf and got[2] == -np.inf and got[1] == 0.0 and np.isfinite(got[5])
