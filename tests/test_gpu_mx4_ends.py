"""The linear layer on 4-bit weights at the ends of K and of the scales, on
each of its kernels.  Everything is a power of two or a small sum: exact."""
import numpy as np
import pytest
import torch

from collective_synchronization_amd import abi
from layer_cases import code_rows, float_rows
from oracle import layer

pytestmark = pytest.mark.gpu

XF = ("bf16", "row8", "mx8", "mx4")
# waves on rows (K whole or not, one part or eight), and each of the tiles
SIZES = ((1, 64, 90), (1, 64, 96), (16, 64, 1100), (3, 40, 4100), (30, 64, 90), (30, 33000, 90), (64, 16384, 90),
         (100, 200, 1100), (70, 33000, 96), (300, 33000, 90))


def _x(v, xf):
    """Device rows of values that every format holds as they are."""
    m, k = v.shape
    if xf == "bf16":
        return float_rows(v, xf)
    if xf == "row8":
        return code_rows(layer.signed_codes(v, layer.E4M3, 128), np.ones(m), xf, k)
    c, s = layer.quantize(v, xf)
    return code_rows(c, s, xf, k)


def _run(m, n, k, xf, xd, wd):
    y = torch.empty((m, n), device="cuda")
    p = abi.linear_params(1, m, n, k, xf, xd.data, xd.stride, 0, xd.scales, xd.scale_stride, 0, wd.data, wd.stride,
                          0, wd.scales, wd.scale_stride, 0, "f32", y, n, 0)
    abi.ar_mx4_linear(p)
    torch.cuda.synchronize()
    return y


@pytest.mark.parametrize("xf", XF)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_weights_past_k_under_the_largest_scale(m, n, k, xf):
    """The block that K ends in has the scale 2^127 and zeros below K; what
    code_rows puts past K would be infinite in bf16."""
    nb = -(-k // 32)
    codes, scales = np.zeros((n, nb * 32), dtype=np.uint8), np.full((n, nb), 127, dtype=np.uint8)
    codes[:, 0], scales[:, nb - 1] = 2, 254
    y = _run(m, n, k, xf, _x(np.ones((m, k)), xf), code_rows(codes, scales, "mx4", k))
    assert bool((y == 1.0).all())


@pytest.mark.parametrize("xf", XF)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_every_code_under_the_first_and_last_scales(m, n, k, xf):
    nb = -(-k // 32)
    codes, scales = np.zeros((n, nb * 32), dtype=np.uint8), np.full((n, nb), 127, dtype=np.uint8)
    codes[:, 0] = np.arange(n) % 16
    scales[:, 0] = np.array([0, 1, 252, 253, 254])[np.arange(n) // 16 % 5]
    x = np.zeros((m, k))
    x[:, 0] = 2.0 ** -6
    y = _run(m, n, k, xf, _x(x, xf), code_rows(codes, scales, "mx4", k)).double().cpu().numpy()
    w = layer.dequantize(codes, scales, "mx4", k)[:, 0]
    if xf == "bf16":                                    # past its range: infinite
        w = np.where(np.abs(w) >= 2.0 ** 128, np.copysign(np.inf, w), w)
    assert np.array_equal(y, np.tile(w * 2.0 ** -6, (m, 1)))


@pytest.mark.parametrize("xf", XF)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_scale_nan_over_zero_codes(m, n, k, xf):
    """What the quantisation makes of a 4-bit block with a NaN: zeros under
    the scale NaN.  Their products are NaN all the same."""
    nb = -(-k // 32)
    codes, scales = np.zeros((n, nb * 32), dtype=np.uint8), np.full((n, nb), 127, dtype=np.uint8)
    scales[3, 1], scales[4, nb - 1] = 255, 255
    xd = _x(np.ones((m, k)), xf)
    nan = _run(m, n, k, xf, xd, code_rows(codes, scales, "mx4", k)).isnan()
    assert bool(nan[:, 3:5].all()) and int(nan.sum()) == 2 * m
    if xf not in ("mx8", "mx4"):
        return
    codes[:], scales[:] = 2, 127
    xc, xs = np.zeros((m, nb * 32), dtype=np.uint8), np.full((m, nb), 127, dtype=np.uint8)
    xs[0, 1] = xs[m - 1, nb - 1] = 255
    nan = _run(m, n, k, xf, code_rows(xc, xs, xf, k), code_rows(codes, scales, "mx4", k)).isnan()
    assert bool(nan[0].all()) and bool(nan[m - 1].all()) and int(nan.sum()) == n * len({0, m - 1})
