"""Attention over a shared prefix and paged own tokens on the GPU: infinities and
NaNs among the values that a token sees, and fp16 weights far below the largest."""
import numpy as np
import pytest
import torch

from collective_synchronization_amd import abi
from test_gpu_attention import Batch, U, _round
from oracle import cache as oc

pytestmark = pytest.mark.gpu

# the places of a key with odd values, and of one with others: token of the prefix, or of a sequence's own ones
PLACES = [("prefix", 0, 5), ("prefix", 99, 2), ("own", 0, 1), ("own", 40, 39), ("own", 61, 3)]


@pytest.mark.parametrize("fmt,cache", [("bf16", "same"), ("f16", "same"), ("bf16", "row8"), ("f16", "row8")])
@pytest.mark.parametrize("queries,heads", [(1, 4), (1, 40), (3, 4), (9, 4), (40, 2)])
@pytest.mark.parametrize("dim", [64, 96])
@pytest.mark.parametrize("where,first,second", PLACES, ids=[f"{w}{a}" for w, a, _ in PLACES])
def test_infinite_and_nan_values_that_are_seen(where, first, second, dim, queries, heads, fmt, cache):
    """A weight is above zero, so an infinity among the values that a token sees makes its output that infinity, two of
    different signs or a NaN make it NaN, and other columns and other sequences are as they are without it."""
    b = Batch(13, (70, 64 + queries, 30), queries, heads, 2, dim, 16, 100, fmt, cache, poison=False)
    table = b.prefix_pages if where == "prefix" else b.pages[0]
    (p, s), (p2, s2) = ((int(table[t // 16]), t % 16) for t in (first, second))
    inf = float("inf")
    if cache == "same":
        for pl, sl, col, v in ((p, s, 0, inf), (p, s, 1, -inf), (p, s, 2, inf), (p2, s2, 2, -inf), (p2, s2, 3, float("nan")),
                               (p, s, dim - 1, inf), (p2, s2, dim - 1, inf), (p2, s2, 17, -inf)):
            b.v[pl, sl, :, col] = v
            b.vd[pl, sl, :, col] = v
    else:
        # an infinite scale: infinities with the codes' signs, and NaN where a code is 0; a NaN scale elsewhere
        b.vd[p, s, :, 3] = 0
        b.v[p, s, :, 3] = 0.0
        b.vd[p, s, :, 4] = 0x7F
        b.v[p, s, :, 4] = np.nan
        with np.errstate(invalid="ignore"):
            b.v[p, s] = b.v[p, s] * np.inf
        b.cache.tensors[3][p, s] = inf
        b.vd[p2, s2, :, 7] = 0x7F
        b.v[p2, s2, :, 7] = np.nan
    prm = b.params()
    abi.ar_prefix_attention(prm, b.work(prm))
    torch.cuda.synchronize()
    got = b.out[:3 * queries].double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        want, _, _, top, mass = oc.attention(b.q, b.k, b.v, b.scale, b.prefix, b.prefix_pages, b.lengths, b.pages, queries)
        fine = np.where(np.isfinite(b.v), b.v, 0.0)
    size = oc.attention(b.q, b.k, fine, b.scale, b.prefix, b.prefix_pages, b.lengths, b.pages, queries)[2]
    assert not np.isfinite(want).all()
    assert (np.isnan(got) == np.isnan(want)).all(), np.argwhere(np.isnan(got) != np.isnan(want))[:5]
    odd = np.isinf(want)
    assert (np.isinf(got) == odd).all() and (got[odd] == want[odd]).all()
    rest = np.isfinite(want)
    e = dim * 2.0 ** -23 * mass + 2 * 2.0 ** -24 * top * 1.4427 + 2.0 ** -22
    keys = b.prefix + max(b.lengths)
    tol = size * (U[fmt] + 2 * e[..., None] + keys * 2.0 ** -23) + keys * 2.0 ** -31 * np.abs(fine).max() + 2.0 ** -25
    tol[rest] += U[fmt] * np.abs(want[rest])
    assert (np.abs(got[rest] - want[rest]) <= tol[rest]).all()


@pytest.mark.parametrize("queries", [1, 9])
@pytest.mark.parametrize("cache", ["same", "row8"])
def test_fp16_weights_far_below_the_largest(cache, queries):
    """One key has almost all the weight and values of zero, the others about 2^-28 each and values of 6e4: weights
    below 2^-20 of the largest lose bits in fp16, by 2^-31 of it at most, which is this test's tolerance (Batch.check)."""
    b = Batch(14, (90, 40), queries, 4, 2, 64, 16, 50, "f16", poison=False)
    b.q[:] = 1.0
    b.qd.fill_(1.0)
    b.k[:] = 0.0
    p, s = int(b.prefix_pages[0]), 7
    b.k[p, s] = _round(28 * np.log(2.0) / 8, "f16")
    b.v[:] = 6e4
    b.v = _round(b.v, "f16")
    b.v[p, s] = 0.0
    if cache == "row8":
        # 60000 as 448 times a scale; keys by their scale, too
        sc = {n: np.ones(b.k.shape[:3], dtype=np.float32) for n in "kv"}
        sc["v"][:] = 60000 / 448
        sc["k"][p, s] = 28 * np.log(2.0) / 8
        codes = {"k": np.zeros(b.k.shape, dtype=np.uint8), "v": np.full(b.v.shape, 0x7E, dtype=np.uint8)}
        codes["k"][p, s] = 0x38                            # 1.0
        codes["v"][p, s] = 0
        value = {0: 0.0, 0x38: 1.0, 0x7E: 448.0}
        dev = {n: torch.from_numpy(codes[n]).cuda() for n in "kv"}
        scd = {n: torch.from_numpy(sc[n]).cuda() for n in "kv"}
        b.k, b.v = (np.vectorize(value.get)(codes[n]) * sc[n][..., None].astype(np.float64) for n in "kv")
        b.cache = abi.cache_params("row8", b.k.shape[0], 16, 2, 64, dev["k"], dev["v"], *dev["k"].stride()[:3],
                                   scd["k"], scd["v"], *scd["k"].stride())
    else:
        b.kd.copy_(torch.from_numpy(b.k).to(torch.float16))
        b.vd.copy_(torch.from_numpy(b.v).to(torch.float16))
    b.run()
    assert float(b.out[0, 0, 0]) > 0.0


@pytest.mark.parametrize("cache", ["same", "row8"])
@pytest.mark.parametrize("queries", [1, 9])
@pytest.mark.parametrize("width", [7, 300, 20000])
def test_tables_wider_than_the_lengths(width, queries, cache):
    """A table with room for far more tokens than there are cuts the keys otherwise and changes nothing."""
    Batch(15, (40, 100, 0, 77), queries, 8, 2, 64, 16, 1500, "bf16", cache, width=width).run()
