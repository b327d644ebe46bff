"""The residual norm and the microscaled formats on the GPU, against the
64-bit forms of oracle/layer.py.

Tolerances, derived from the arithmetic:
* quantisation and its inverse round once from exact inputs: equal bits;
* the norm: h is one binary32 addition (2^-24 of h).  The sum of squares has
  only positive terms and its relative error is at most the longest chain of
  additions (64 in a thread, 6 levels of lanes, 16 waves) plus the squares' own,
  90 steps, halved by the square root; the division by hidden, eps, root,
  reciprocal and the two products add 6 more.  With every one of them a
  binary32 step, the worst that is allowed, that is at most 51 + 2 <= 64 steps of
  2^-24; then the output's own rounding.
"""
import numpy as np
import pytest
import torch

from collective_synchronization_amd import abi, buffers
from layer_cases import (check_float, check_quantized, code_rows, float_rows, out_rows, read_codes,
                         to_type, untouched)
from oracle import layer

pytestmark = pytest.mark.gpu

REL = 64 * 2.0 ** -24
QUANT = ("row8", "mx8", "mx4")


def _rows(rng, rows, cols, fmt):
    v = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-3, 4, (rows, 1)))
    return to_type(v, fmt)


def _norm(x, fmt, res, res_fmt, gamma, y_fmt, eps=1e-5, extra=0, in_place=False, want_h=True):
    """Runs the norm; returns (residual_out rows, y rows)."""
    rows, cols = x.shape
    xd = float_rows(x, fmt, extra)
    rd = float_rows(res, res_fmt, extra) if res is not None else None
    h = rd if in_place else (out_rows(rows, cols, res_fmt) if want_h else None)
    y = out_rows(rows, cols, y_fmt)
    g = torch.from_numpy(gamma).to(xd.data.dtype).to("cuda") if gamma is not None else None
    p = abi.norm_params(rows, cols, eps, fmt, g, res_fmt, rd.data if rd else None,
                        rd.stride if rd else 0, h.data if h else None, h.stride if h else 0, y_fmt,
                        y.data, y.stride, y.scales, y.scale_stride)
    abi.ar_residual_norm(p, xd.data, xd.stride)
    torch.cuda.synchronize()
    return h, y


def _check(h, y, x, res, res_fmt, gamma, y_fmt, eps=1e-5):
    hs = x if res is None else x + res
    if h is not None:
        got = h.data[:, :h.cols].double().cpu().numpy()
        check_float(got, hs, res_fmt, 2.0 ** -24)
    v = layer.norm(hs, gamma, eps)
    if y_fmt in QUANT:
        check_quantized(y, y_fmt, v, REL)
    else:
        check_float(y.data[:, :y.cols].double().cpu().numpy(), v, y_fmt, REL)
        assert untouched(y)


@pytest.mark.parametrize("y_fmt", ["same", "row8", "mx8", "mx4"])
@pytest.mark.parametrize("fmt,res_fmt", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"),
                                         ("f16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("rows,cols", [(1, 4096), (3, 1), (2, 7), (5, 33), (4, 250), (300, 520),
                                       (2, 8200), (1, 16384), (2, 30011), (1, 32768)])
def test_residual_norm(rows, cols, fmt, res_fmt, y_fmt):
    print(f"[norm] {rows}x{cols} {fmt} {res_fmt} {y_fmt}", flush=True)
    rng = np.random.default_rng(rows * 100003 + cols)
    x, res = _rows(rng, rows, cols, fmt), _rows(rng, rows, cols, res_fmt)
    gamma = to_type(rng.uniform(0.5, 1.5, cols), fmt)
    y_fmt = fmt if y_fmt == "same" else y_fmt
    h, y = _norm(x, fmt, res, res_fmt, gamma, y_fmt, extra=rows % 2)
    assert untouched(h)
    _check(h, y, x, res, res_fmt, gamma, y_fmt)


@pytest.mark.parametrize("y_fmt", ["bf16", "row8", "mx8", "mx4"])
def test_norm_without_residual_gamma_or_output(y_fmt):
    rng = np.random.default_rng(5)
    x = _rows(rng, 6, 1000, "bf16")
    h, y = _norm(x, "bf16", None, "bf16", None, y_fmt, want_h=False)
    _check(None, y, x, None, "bf16", None, y_fmt)
    # the residual stream updated in place
    res = _rows(rng, 6, 1000, "f32")
    h, y = _norm(x, "bf16", res, "f32", None, y_fmt, in_place=True)
    _check(h, y, x, res, "f32", None, y_fmt)


@pytest.mark.parametrize("y_fmt", ["f32", "row8", "mx8", "mx4"])
def test_norm_of_zeros_and_extremes(y_fmt):
    x = np.zeros((6, 100))
    x[1, 3] = np.nan
    x[2, 50] = np.inf
    x[3, :] = 1e-30
    x[4, :] = -0.0
    x[5, 99] = 2.0 ** 40
    h, y = _norm(x, "f32", None, "f32", None, y_fmt, eps=1e-6)
    v = np.empty_like(x)
    with np.errstate(invalid="ignore", divide="ignore"):
        v[:] = layer.norm(x, None, 1e-6)
    if y_fmt == "f32":
        check_float(y.data[:, :100].double().cpu().numpy(), v, "f32", REL)
    elif y_fmt == "row8":
        check_quantized(y, y_fmt, v, REL)
        codes, sc = read_codes(y, y_fmt)
        assert (codes[0] == 0).all() and sc[0] == np.float32(2.0 ** -126)
    else:
        # row 2: zeros but for the block that holds inf * 0
        assert np.isnan(v[2, 50])
        check_quantized(y, y_fmt, v, REL)
    # eps 0 on a zero row: 0 * inf is NaN everywhere
    h, y = _norm(np.zeros((1, 40)), "f32", None, "f32", None, y_fmt, eps=0.0)
    if y_fmt == "f32":
        assert np.isnan(y.data[:, :40].cpu().numpy()).all()
    else:
        codes, sc = read_codes(y, y_fmt)
        assert np.isnan(sc).all() if y_fmt == "row8" else (sc == 255).all()


def test_norm_in_place_and_many_rows():
    """y over x, residual_out over the residual; more rows than 2^16."""
    rng = np.random.default_rng(6)
    rows, cols = 70001, 40
    x, res = _rows(rng, rows, cols, "bf16"), _rows(rng, rows, cols, "bf16")
    xd, rd = float_rows(x, "bf16"), float_rows(res, "bf16")
    p = abi.norm_params(rows, cols, 1e-5, "bf16", None, "bf16", rd.data, rd.stride, rd.data, rd.stride,
                        "bf16", xd.data, xd.stride)
    abi.ar_residual_norm(p, xd.data, xd.stride)
    torch.cuda.synchronize()
    check_float(rd.data[:, :cols].double().cpu().numpy(), x + res, "bf16", 2.0 ** -24)
    check_float(xd.data[:, :cols].double().cpu().numpy(), layer.norm(x + res, None, 1e-5), "bf16", REL)


def test_norm_rows_past_32_bits():
    """Rows whose offsets pass 2^32 bytes."""
    cols, stride, rows = 64, 1 << 20, 2100
    x = torch.zeros((rows, stride), dtype=torch.bfloat16, device="cuda")
    x[:, :cols] = torch.randn((rows, cols), device="cuda").to(torch.bfloat16)
    y = out_rows(rows, cols, "bf16")
    p = abi.norm_params(rows, cols, 1e-5, "bf16", None, "bf16", None, 0, None, 0, "bf16", y.data,
                        y.stride)
    abi.ar_residual_norm(p, x, stride)
    torch.cuda.synchronize()
    xs = x[:, :cols].double().cpu().numpy()
    check_float(y.data[:, :cols].double().cpu().numpy(), layer.norm(xs, None, 1e-5), "bf16", REL)


def test_empty_calls_write_nothing():
    y = out_rows(4, 64, "mx8")
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    for rows, cols in ((0, 64), (4, 0)):
        p = abi.norm_params(rows, cols, 1e-5, "bf16", None, "bf16", None, 0, None, 0, "mx8", y.data,
                            y.stride, y.scales, y.scale_stride)
        abi.ar_residual_norm(p, x, 64)
        abi.ar_quantize_mx(rows, cols, "bf16", x, 64, "mx8", y.data, y.stride, y.scales, y.scale_stride)
        abi.ar_dequantize_mx(rows, cols, "mx8", y.data, y.stride, y.scales, y.scale_stride, "bf16", x, 64)
    torch.cuda.synchronize()
    assert bool((y.data == 0xA5).all()) and bool((y.scales == 0xA5).all())


# ------------------------------------------------------------ quantisation --

def _edge_values(fmt):
    """Blocks of ties, limits, signed zeros, subnormals, NaN and infinities."""
    t = []
    for e in (-126, -20, -1, 0, 5, 14):
        s = 2.0 ** e
        t.append([k * 0.25 * s for k in range(-16, 16)])
        t.append([(1 + k / 16) * s * (-1) ** k for k in range(32)])
        t.append([4 * s * (1 + k / 64) for k in range(32)])
    t.append([0.0, -0.0] * 16)
    t.append([2.0 ** -149 * k for k in range(32)])
    t.append([1.0] * 31 + [float("nan")])
    t.append([float("inf")] + [0.5] * 31)
    t.append([-float("inf"), float("nan")] + [0.0] * 30)
    t.append([3.3895313892515355e38 * (1 - k / 40) for k in range(32)])
    v = np.array(t)
    if fmt == "f16":
        v = np.where(np.abs(v) < 65520, v, np.where(np.isfinite(v), 60000.0, v))
    return to_type(v.reshape(-1), fmt).reshape(v.shape)


@pytest.mark.parametrize("q", ["mx8", "mx4"])
@pytest.mark.parametrize("fmt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (2, 32), (7, 33), (17, 4100), (2500, 72), (0, 0)])
def test_quantize_and_back_exact(rows, cols, fmt, q):
    print(f"[quant] {rows}x{cols} {fmt} {q}", flush=True)
    if rows == 0:                                   # the edge values
        v = _edge_values(fmt)
        rows, cols = v.shape
    else:
        rng = np.random.default_rng(rows * 31 + cols)
        v = to_type(rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-8, 9, (rows, cols))), fmt)
    xd = float_rows(v, fmt, rows % 3)
    out = out_rows(rows, cols, q)
    abi.ar_quantize_mx(rows, cols, fmt, xd.data, xd.stride, q, out.data, out.stride, out.scales,
                       out.scale_stride)
    torch.cuda.synchronize()
    want, want_sc = layer.quantize(v, q)
    got, sc = read_codes(out, q)
    assert np.array_equal(sc, want_sc)
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]
    assert untouched(out)
    back = layer.dequantize(want, want_sc, q, cols)
    for f in ("bf16", "f16", "f32"):
        y = out_rows(rows, cols, f)
        abi.ar_dequantize_mx(rows, cols, q, out.data, out.stride, out.scales, out.scale_stride, f,
                             y.data, y.stride)
        torch.cuda.synchronize()
        want_f = torch.from_numpy(back).to(y.data.dtype)
        got_f = y.data[:, :cols].cpu()
        same = (got_f == want_f) | (got_f.isnan() & want_f.isnan())
        assert bool(same.all()), f
        assert untouched(y)


@pytest.mark.parametrize("q", ["mx8", "mx4"])
def test_every_code_and_scale_back(q):
    """All element codes under all 256 scales."""
    n = 256 if q == "mx8" else 32
    codes = np.tile(np.arange(n) % (256 if q == "mx8" else 16), (256, 1)).astype(np.uint8)
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], n // 32, axis=1)
    r = code_rows(codes, scales, q, n)
    want = torch.from_numpy(layer.dequantize(codes, scales, q, n))
    for f, t in (("f32", torch.float32), ("bf16", torch.bfloat16)):
        y = out_rows(256, n, f)
        abi.ar_dequantize_mx(256, n, q, r.data, r.stride, r.scales, r.scale_stride, f, y.data, y.stride)
        torch.cuda.synchronize()
        got, w = y.data[:, :n].cpu(), want.to(torch.float32).to(t)
        assert bool(((got == w) | (got.isnan() & w.isnan())).all()), f


def test_rows_on_another_stream_and_in_a_graph():
    """Both operators on a side stream, captured and replayed with eager work
    between the replays."""
    rng = np.random.default_rng(9)
    x = _rows(rng, 9, 777, "bf16")
    xd = float_rows(x, "bf16")
    y = out_rows(9, 777, "row8")
    q = out_rows(9, 777, "mx4")
    p = abi.norm_params(9, 777, 1e-5, "bf16", None, "bf16", None, 0, None, 0, "row8", y.data, y.stride,
                        y.scales, 0)

    def both():
        abi.ar_residual_norm(p, xd.data, xd.stride)
        abi.ar_quantize_mx(9, 777, "bf16", xd.data, xd.stride, "mx4", q.data, q.stride, q.scales,
                           q.scale_stride)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for k in range(3):
        x = _rows(rng, 9, 777, "bf16")
        xd.data[:, :777] = torch.from_numpy(x).to(torch.bfloat16).to("cuda")
        y.data.fill_(0xA5)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        check_quantized(y, "row8", layer.norm(x, None, 1e-5), REL)
        got, sc = read_codes(q, "mx4")
        want, want_sc = layer.quantize(x, "mx4")
        assert np.array_equal(got, want) and np.array_equal(sc, want_sc), k
