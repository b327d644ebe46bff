"""The linear layer on 4-bit weights on the GPU, against 64-bit products.

Two kinds of inputs:
* small dyadic numbers whose every partial sum is a binary32 value, so that
  any order of the sum gives the same bits: binary32 outputs are equal to the
  64-bit product, bf16 outputs to its one rounding;
* random numbers: binary32 accumulation of K products in any order is off by
  at most K * 2^-24 * sum|x w|; the matrix cores' own additions may truncate
  instead of round, which doubles a step.
"""
import numpy as np
import pytest
import torch

from collective_synchronization_amd import abi, buffers
from layer_cases import code_rows, float_rows, to_type
from oracle import layer

pytestmark = pytest.mark.gpu

XF = ("bf16", "row8", "mx8", "mx4")
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def _dyadic(rng, rows, k, fmt):
    """(values, device rows): magnitudes at most 12, multiples of 1/4, so
    a product is a multiple of 2^-4."""
    if fmt == "bf16":
        v = rng.integers(-12, 13, (rows, k)) / 2.0
        return v, float_rows(v, "bf16")
    nb = -(-k // 32)
    if fmt == "row8":
        c = layer.signed_codes(rng.integers(-8, 9, (rows, k)) / 2.0, layer.E4M3, 128)
        s = np.exp2(rng.integers(-1, 2, rows))
        return layer.dequantize(c, s, fmt, k), code_rows(c, s, fmt, k)
    sc = rng.integers(126, 129, (rows, nb)).astype(np.uint8)
    if fmt == "mx8":
        c = layer.signed_codes(rng.integers(-8, 9, (rows, 32 * nb)) / 2.0, layer.E4M3, 128)
    else:
        c = rng.integers(0, 16, (rows, 32 * nb)).astype(np.uint8)
    c[:, k:] = 0
    return layer.dequantize(c, sc, fmt, k), code_rows(c, sc, fmt, k, extra=rows % 2)


def _random(rng, rows, k, fmt, scale):
    v = rng.standard_normal((rows, k)) * scale
    if fmt == "bf16":
        v = to_type(v, "bf16")
        return v, float_rows(v, "bf16")
    if fmt == "row8":
        s = (np.abs(v).max(-1) / 448).astype(np.float32)
        c = layer.signed_codes(v / s[:, None].astype(np.float64), layer.E4M3, 128)
        return layer.dequantize(c, s, fmt, k), code_rows(c, s, fmt, k)
    c, sc = layer.quantize(v, fmt)
    return layer.dequantize(c, sc, fmt, k), code_rows(c, sc, fmt, k)


def _run(ranks, m, n, k, xf, xd, wd, yf, y_stride=None, y_rank=None):
    y_stride = n if y_stride is None else y_stride
    y_rank = m * y_stride if y_rank is None else y_rank
    y = torch.full((ranks * y_rank + 8,), -77.0, dtype=TORCH[yf], device="cuda")
    xs_rank = m if xf == "row8" else m * xd.scale_stride
    p = abi.linear_params(ranks, m, n, k, xf, xd.data, xd.stride, m * xd.stride, xd.scales,
                          xd.scale_stride, xs_rank, wd.data, wd.stride, n * wd.stride, wd.scales,
                          wd.scale_stride, n * wd.scale_stride, yf, y, y_stride, y_rank)
    abi.ar_mx4_linear(p)
    torch.cuda.synchronize()
    flat = y.double().cpu().numpy()
    got = np.stack([flat[r * y_rank: r * y_rank + m * y_stride].reshape(m, y_stride) for r in range(ranks)])
    assert (got[:, :, n:] == -77.0).all() and (flat[ranks * y_rank:] == -77.0).all()
    return got[:, :, :n]


SIZES = [(1, 1, 16, 32), (1, 1, 1, 1), (2, 3, 17, 33), (8, 1, 4096, 512), (1, 16, 64, 512), (1, 17, 100, 1000),
         (4, 5, 33, 544), (1, 33, 48, 2080), (2, 64, 80, 1536), (1, 65, 130, 640), (1, 200, 300, 1056),
         (2, 130, 520, 288), (1, 257, 260, 2048), (1, 300, 1030, 160),
         # each of the tile kernels, by its number of tiles; K in whole steps and not
         (16, 300, 2000, 544), (16, 257, 2050, 96), (8, 700, 2500, 1100), (16, 100, 2000, 1100),
         (16, 20, 2000, 1100), (16, 32, 1100, 64), (16, 60, 2000, 300), (1, 40, 100, 3500), (3, 100, 200, 2560),
         # either side of where the kernel for a few tokens and the largest tiles take over
         (16, 8, 1100, 544), (16, 9, 1100, 544), (16, 16, 2000, 1100), (8, 13, 2500, 300), (16, 128, 2050, 288),
         (16, 129, 2050, 288)]


@pytest.mark.parametrize("yf", ("bf16", "f32"))
@pytest.mark.parametrize("xf", XF)
@pytest.mark.parametrize("ranks,m,n,k", SIZES)
def test_dyadic_products_exact(ranks, m, n, k, xf, yf):
    print(f"[linear] R={ranks} {m}x{n}x{k} {xf} -> {yf}", flush=True)
    rng = np.random.default_rng(m * 7 + n * 3 + k)
    xv, xd = _dyadic(rng, ranks * m, k, xf)
    wv, wd = _dyadic(rng, ranks * n, k, "mx4")
    want = layer.linear(xv.reshape(ranks, m, k), wv.reshape(ranks, n, k))
    # products are multiples of 2^-4, partial sums below 2^19: 23 bits
    assert k * 12 * 12 < 2 ** 19
    got = _run(ranks, m, n, k, xf, xd, wd, yf, y_stride=n + (n + m) % 3)
    if yf == "bf16":
        want = to_type(want, "bf16")
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]


@pytest.mark.parametrize("xf", XF)
@pytest.mark.parametrize("ranks,m,n,k", [(2, 1, 512, 2048), (1, 16, 256, 8192), (1, 150, 384, 4100)])
def test_random_products(ranks, m, n, k, xf):
    rng = np.random.default_rng(k + m)
    xv, xd = _random(rng, ranks * m, k, xf, 1.0)
    wv, wd = _random(rng, ranks * n, k, "mx4", k ** -0.5)
    x3, w3 = xv.reshape(ranks, m, k), wv.reshape(ranks, n, k)
    want, size = layer.linear(x3, w3), layer.linear(np.abs(x3), np.abs(w3))
    got = _run(ranks, m, n, k, xf, xd, wd, "f32")
    tol = 2 * k * 2.0 ** -24 * size + 2.0 ** -24 * np.abs(want)
    assert (np.abs(got - want) <= tol).all()
    got = _run(ranks, m, n, k, xf, xd, wd, "bf16")
    assert (np.abs(got - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol)).all()


@pytest.mark.parametrize("m", (1, 100))
@pytest.mark.parametrize("xf", XF)
def test_every_weight_scale(xf, m):
    """Output n's weights have scale code n: 2^-127 to 2^127, then NaN."""
    codes = np.full((256, 32), 2, dtype=np.uint8)                  # ones
    wd = code_rows(codes, np.arange(256, dtype=np.uint8)[:, None], "mx4", 32)
    one = np.zeros((m, 32))
    one[:, 3] = 1.0
    if xf == "bf16":
        xd = float_rows(one, "bf16")
    elif xf == "row8":
        xd = code_rows(layer.signed_codes(one, layer.E4M3, 128), np.ones(m), xf, 32)
    else:
        c = layer.signed_codes(one, layer.GRID[xf], 128)
        xd = code_rows(c, np.full((m, 1), 127, dtype=np.uint8), xf, 32)
    got = _run(1, m, 256, 32, xf, xd, wd, "f32")[0]
    want = np.ldexp(1.0, np.arange(255) - 127)
    # the smallest scale makes a binary32 subnormal, which the matrix cores may flush
    assert np.array_equal(got[:, 1:255], np.tile(want[1:], (m, 1)))
    assert ((got[:, 0] == want[0]) | (got[:, 0] == 0)).all()
    assert np.isnan(got[:, 255]).all()


@pytest.mark.parametrize("xf", ("mx8", "mx4", "row8"))
@pytest.mark.parametrize("m", (2, 80))
def test_scale_nan_of_an_input_row_stays_in_its_row(xf, m):
    rng = np.random.default_rng(3)
    xv, xd = _dyadic(rng, m, 96, xf)
    wv, wd = _dyadic(rng, 40, 96, "mx4")
    if xf == "row8":
        xd.scales[1] = float("nan")
    else:
        xd.scales[1, 1] = 255
    got = _run(1, m, 40, 96, xf, xd, wd, "f32")[0]
    want = xv @ wv.T
    keep = np.arange(m) != 1
    assert np.isnan(got[1]).all() and np.array_equal(got[keep], want[keep])


@pytest.mark.parametrize("m", (3, 40, 300))
@pytest.mark.parametrize("xf", XF)
def test_no_inputs_gives_zeros(xf, m):
    y = torch.full((m, 24), -77.0, device="cuda")
    p = abi.linear_params(1, m, 20, 0, xf, None, 0, 0, None, 0, 0, None, 0, 0, None, 0, 0, "f32", y, 24, 0)
    abi.ar_mx4_linear(p)
    for rows, outs in ((0, 20), (m, 0)):
        q = abi.linear_params(1, rows, outs, 64, xf, None, 0, 0, None, 0, 0, None, 0, 0, None, 0, 0, "f32",
                              None, 24, 0)
        abi.ar_mx4_linear(q)
    torch.cuda.synchronize()
    assert bool((y[:, :20] == 0).all()) and bool((y[:, 20:] == -77.0).all())


def test_ranks_take_slices_of_one_row():
    """Row-parallel: rank r's inputs are columns [r*kr, (r+1)*kr) of the same rows."""
    ranks, m, n, kr = 4, 5, 64, 256
    rng = np.random.default_rng(8)
    xv, xd = _dyadic(rng, m, ranks * kr, "mx8")
    wv, wd = _dyadic(rng, ranks * n, kr, "mx4")
    y = torch.zeros((ranks, m, n), device="cuda")
    p = abi.linear_params(ranks, m, n, kr, "mx8", xd.data, xd.stride, kr, xd.scales, xd.scale_stride,
                          kr // 32, wd.data, wd.stride, n * wd.stride, wd.scales, wd.scale_stride,
                          n * wd.scale_stride, "f32", y, n, m * n)
    abi.ar_mx4_linear(p)
    torch.cuda.synchronize()
    want = layer.linear(np.stack([xv[:, r * kr:(r + 1) * kr] for r in range(ranks)]), wv.reshape(ranks, n, kr))
    assert np.array_equal(y.double().cpu().numpy(), want)


def test_rows_far_apart():
    """Row strides of 8 MiB, at any number of tokens."""
    m, n, k, far = 40, 70, 600, 1 << 23
    rng = np.random.default_rng(11)
    wv, wd = _dyadic(rng, n, k, "mx4")
    xv, xn = _dyadic(rng, m, k, "row8")
    x = torch.zeros((m, far), dtype=torch.uint8, device="cuda")
    x[:, :k] = xn.data[:, :k]
    y = torch.zeros((m, n), device="cuda")
    p = abi.linear_params(1, m, n, k, "row8", x, far, 0, xn.scales, 0, 0, wd.data, wd.stride, 0, wd.scales,
                          wd.scale_stride, 0, "f32", y, n, 0)
    abi.ar_mx4_linear(p)
    torch.cuda.synchronize()
    assert np.array_equal(y.double().cpu().numpy(), xv @ wv.T)


def test_two_streams_at_once():
    """Calls on two streams, tiles of different kernels, beside each other."""
    rng = np.random.default_rng(12)
    cases = []
    for m, n, k in ((1, 4096, 1024), (200, 2000, 1100)):
        xv, xd = _dyadic(rng, m, k, "mx8")
        wv, wd = _dyadic(rng, n, k, "mx4")
        y = torch.zeros((m, n), device="cuda")
        p = abi.linear_params(1, m, n, k, "mx8", xd.data, xd.stride, 0, xd.scales, xd.scale_stride, 0,
                              wd.data, wd.stride, 0, wd.scales, wd.scale_stride, 0, "f32", y, n, 0)
        cases.append((p, y, xv @ wv.T, (xd, wd), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for p, _, _, _, s in cases:
            abi.ar_mx4_linear(p, stream=s)
    torch.cuda.synchronize()
    for _, y, want, _, _ in cases:
        assert np.array_equal(y.double().cpu().numpy(), want)


@pytest.mark.parametrize("m", (1, 90))
def test_same_bits_every_time_and_in_a_graph(m):
    rng = np.random.default_rng(4)
    xv, xd = _random(rng, m, 2048, "mx8", 1.0)
    wv, wd = _random(rng, 256, 2048, "mx4", 0.02)
    y = torch.zeros((m, 256), device="cuda")
    p = abi.linear_params(1, m, 256, 2048, "mx8", xd.data, xd.stride, 0, xd.scales, xd.scale_stride, 0,
                          wd.data, wd.stride, 0, wd.scales, wd.scale_stride, 0, "f32", y, 256, 0)
    abi.ar_mx4_linear(p)
    torch.cuda.synchronize()
    first = y.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        abi.ar_mx4_linear(p)
    for _ in range(3):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, first)
        abi.ar_mx4_linear(p)
        torch.cuda.synchronize()
        assert torch.equal(y, first)


@pytest.mark.parametrize("proto", ("ll", "sentinel"))
@pytest.mark.parametrize("rows", (1, 4))
def test_layers_in_a_row(proto, rows):
    """As they are used: reduce + norm to 8 bits, the ranks' linear shards of
    the normed row, their payloads packed, reduced and normed again.  Each
    step is checked against the 64-bit form of the values it was given."""
    ranks, hidden = 4, 1024
    kr = hidden // ranks
    rng = np.random.default_rng(rows)
    ws = buffers.Workspace(ranks, rows * hidden, proto)
    wv, wd = _random(rng, ranks * hidden, kr, "mx4", hidden ** -0.5)
    res = buffers.FormatRows(rows, hidden, "f32")
    res.data.copy_(torch.from_numpy(rng.standard_normal((rows, hidden))))
    y = buffers.FormatRows(rows, hidden, "mx8")
    pay = torch.zeros((ranks, rows * hidden), dtype=torch.bfloat16, device="cuda")
    pay.copy_(torch.from_numpy(rng.standard_normal((ranks, rows * hidden))))
    norm = abi.norm_params(rows, hidden, 1e-5, "bf16", None, "f32", res.data, res.stride, res.data,
                           res.stride, "mx8", y.data, y.stride, y.scales, y.scale_stride)
    lin = abi.linear_params(ranks, rows, hidden, kr, "mx8", y.data, y.stride, kr, y.scales,
                            y.scale_stride, kr // 32, wd.data, wd.stride, hidden * wd.stride, wd.scales,
                            wd.scale_stride, hidden * wd.scale_stride, "bf16", pay, hidden, rows * hidden)
    for step in range(5):
        before = res.data.cpu().numpy().copy()
        sent = pay.double().cpu().numpy().astype(np.float32)
        ws.pack(pay, rows * hidden)
        ws.reduce_norm(norm, timeout_ns=2_000_000_000)
        ws.flip()
        abi.ar_mx4_linear(lin)
        torch.cuda.synchronize()
        assert ws.status() == 0
        h = (before + layer.rank_sum_f32(sent).reshape(rows, hidden)).astype(np.float32)
        assert np.array_equal(res.data.cpu().numpy(), h)
        v = layer.norm(h.astype(np.float64), None, 1e-5)
        codes, sc = y.data.cpu().numpy(), y.scales.cpu().numpy()[:, :hidden // 32]
        want_codes, want_sc = layer.quantize(v, "mx8")
        assert (sc == want_sc).mean() > 0.99 and (codes == want_codes).mean() > 0.99
        x = layer.dequantize(codes, sc, "mx8", hidden)
        xr = np.stack([x[:, r * kr:(r + 1) * kr] for r in range(ranks)])
        w3 = wv.reshape(ranks, hidden, kr)
        want, size = layer.linear(xr, w3), layer.linear(np.abs(xr), np.abs(w3))
        got = pay.double().cpu().numpy().reshape(ranks, rows, hidden)
        tol = 2 * kr * 2.0 ** -24 * size
        assert (np.abs(got - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol)).all(), step
