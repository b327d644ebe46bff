"""The linear layer on 4-bit weights with each token's low-rank adapter, against
64-bit products.

Two kinds of inputs, as for the layer alone: small dyadic numbers, whose every
partial sum is a binary32 value (t at most 16 bits, so that it is the sum of two
bf16 values), give outputs equal to the 64-bit ones; of random numbers the
layer's own sum is off by 2 * K * 2^-24 * sum|x w| (and 2^-13 of it for 8-bit x with
bf16 y, as the header says), t by 2 * K * 2^-24 * sum|x a| and by 2^-15 (binary32 y: 2^-23) of itself
and 2^-23 for its two scales, its second product by 2 * 3 * rank * 2^-24, all
of these times sum |t||b|; the output is rounded once.
"""
import numpy as np
import pytest
import torch

from collective_synchronization_amd import abi
from layer_cases import code_rows, float_rows
from oracle import layer

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def _x(rng, rows, k, fmt, dyadic):
    nb = -(-k // 32)
    if dyadic:
        if fmt == "bf16":
            v = rng.integers(-4, 5, (rows, k)) / 2.0
            return v, float_rows(v, "bf16")
        if fmt == "row8":
            c, s = layer.signed_codes(rng.integers(-4, 5, (rows, k)) / 2.0, layer.E4M3, 128), np.exp2(rng.integers(-1, 2, rows))
        elif fmt == "mx8":
            c, s = layer.signed_codes(rng.integers(-4, 5, (rows, 32 * nb)) / 2.0, layer.E4M3, 128), rng.integers(127, 129, (rows, nb)).astype(np.uint8)
        else:
            c, s = rng.integers(0, 16, (rows, 32 * nb)).astype(np.uint8), rng.integers(126, 128, (rows, nb)).astype(np.uint8)
    else:
        v = rng.standard_normal((rows, k))
        if fmt == "bf16":
            d = float_rows(v, "bf16")
            return d.data[:, :k].double().cpu().numpy(), d
        if fmt == "row8":
            s = (np.abs(v).max(-1) / 448).astype(np.float32)
            c = layer.signed_codes(v / s[:, None].astype(np.float64), layer.E4M3, 128)
        else:
            c, s = layer.quantize(v, fmt)
    if fmt != "row8":
        c[:, k:] = 0
    return layer.dequantize(c, s, fmt, k), code_rows(c, s, fmt, k)


def _matrices(rng, shape, dyadic, scale):
    """bf16 [..., rows, cols] with strides past the row; NaN behind it."""
    cols = shape[-1]
    wide = (cols + 7) // 8 * 8 + 8
    v = rng.integers(-2, 3, shape) / 2.0 if dyadic else rng.standard_normal(shape) * scale
    host = torch.full(shape[:-1] + (wide,), float("nan"), dtype=torch.bfloat16)
    host[..., :cols] = torch.from_numpy(v).to(torch.bfloat16)
    return host[..., :cols].double().numpy(), host.cuda()


class Case:
    def __init__(self, seed, ranks, m, n, k, xf, yf, count, rank, index, columns=False, dyadic=False, scales=True):
        rng = np.random.default_rng(seed)
        self.sizes, self.xf, self.yf, self.columns, self.dyadic = (ranks, m, n, k), xf, yf, columns, dyadic
        nb = -(-k // 32)
        xr = 1 if columns else ranks
        self.x, self.xd = _x(rng, xr * m, k, xf, dyadic)
        self.x = self.x.reshape(xr, m, k)
        if dyadic:
            wc, ws = rng.integers(0, 16, (ranks * n, 32 * nb)).astype(np.uint8), rng.integers(126, 128, (ranks * n, nb)).astype(np.uint8)
        else:
            wc, ws = layer.quantize(rng.standard_normal((ranks * n, k)) * k ** -0.5, "mx4")
        wc[:, k:] = 0
        self.w = layer.dequantize(wc, ws, "mx4", k).reshape(ranks, n, k)
        self.wd = code_rows(wc, ws, "mx4", k)
        self.a, self.ad = _matrices(rng, (1 if columns else ranks, count, rank, k), dyadic, k ** -0.5)
        self.b, self.bd = _matrices(rng, (ranks if columns else 1, count, n, rank), dyadic, rank ** -0.5)
        self.index = np.asarray(index, dtype=np.int64)
        self.scale = (np.exp2(rng.integers(-1, 2, count)) if dyadic else rng.uniform(0.2, 3, count).astype(np.float32)) if scales else np.ones(count)
        self.count, self.rank = count, rank
        self.idx = torch.from_numpy(self.index.astype(np.int32)).cuda()
        self.sc = torch.tensor(self.scale, dtype=torch.float32).cuda() if scales else None
        self.y = torch.full((ranks, m, n + 4), -77.0, dtype=TORCH[yf], device="cuda")

    def params(self):
        ranks, m, n, k = self.sizes
        xd, wd, a, b, y = self.xd, self.wd, self.ad, self.bd, self.y
        xs_rank = m if self.xf == "row8" else m * xd.scale_stride
        lin = abi.linear_params(ranks, m, n, k, self.xf, xd.data, xd.stride, 0 if self.columns else m * xd.stride, xd.scales,
                                xd.scale_stride, 0 if self.columns else xs_rank, wd.data, wd.stride, n * wd.stride,
                                wd.scales, wd.scale_stride, n * wd.scale_stride, self.yf, y, y.stride(1), y.stride(0))
        ad = abi.adapter_params(self.count, self.rank, self.idx, self.sc, a, a.stride(2), a.stride(1),
                                0 if self.columns else a.stride(0), b, b.stride(2), b.stride(1),
                                b.stride(0) if self.columns else 0)
        return lin, ad

    def work(self, lin, ad):
        return torch.full((max(64, abi.ar_adapter_work_bytes(lin, ad) // 4),), float("nan"), device="cuda")

    def run(self):
        lin, ad = self.params()
        abi.ar_mx4_linear_adapters(lin, ad, self.work(lin, ad))
        torch.cuda.synchronize()
        self.check()

    def check(self):
        ranks, m, n, k = self.sizes
        got = self.y.double().cpu().numpy()
        assert (got[:, :, n:] == -77.0).all()
        u = 2.0 ** -8 if self.yf == "bf16" else 2.0 ** -24
        for r in range(ranks):
            x, a, b = self.x[r % len(self.x)], self.a[r % len(self.a)], self.b[r % len(self.b)]
            y = x @ self.w[r].T
            err = np.abs(x) @ np.abs(self.w[r]).T * (2 * k * 2.0 ** -24 + (2.0 ** -13 if self.xf in ("row8", "mx8") and self.yf == "bf16" else 0) + 2.0 ** -23)
            for i in set(self.index.tolist()):
                if not 0 <= i < self.count:
                    continue
                at = np.flatnonzero(self.index == i)
                t = x[at] @ a[i].T * self.scale[i]
                y[at] += t @ b[i].T
                te = (np.abs(x[at]) @ np.abs(a[i]).T * abs(self.scale[i]) * (2 * k * 2.0 ** -24) +
                      np.abs(t) * ((2.0 ** -15 if self.yf == "bf16" else 2.0 ** -23) + 2.0 ** -23))
                err[at] += te @ np.abs(b[i]).T + np.abs(t) @ np.abs(b[i]).T * (6 * self.rank * 2.0 ** -24)
            out = got[r, :, :n]
            if self.dyadic:
                want = torch.from_numpy(y).to(TORCH[self.yf]).double().numpy()
                assert np.array_equal(out, want), np.argwhere(out != want)[:5]
            else:
                tol = err * (1 + u) + u * np.abs(y)
                assert (np.abs(out - y) <= tol).all(), (np.argwhere(np.abs(out - y) > tol)[:5], (np.abs(out - y) / tol).max())


def _index(kind, m, count, seed=0):
    rng = np.random.default_rng(seed)
    if kind == "each":
        return np.arange(m) % count
    if kind == "runs":
        return np.arange(m) * count // m
    if kind == "mixed":
        return rng.integers(-1, count + 1, m)         # -1 and `count` are none
    if kind == "wild":
        return rng.choice([0, -1, -2 ** 31, 2 ** 31 - 1, count, count - 1], m)
    return np.full(m, -1)


SIZES = [
    # ranks, m, n, k, adapters, rank, index
    (1, 1, 1, 1, 1, 1, "each"), (1, 1, 16, 32, 1, 16, "each"), (2, 3, 17, 33, 2, 5, "mixed"), (8, 1, 300, 512, 4, 16, "each"),
    (1, 16, 64, 1100, 16, 8, "each"), (4, 16, 2100, 544, 5, 16, "wild"), (1, 9, 5000, 96, 9, 33, "each"),
    (1, 17, 100, 1000, 17, 24, "each"), (2, 33, 48, 300, 3, 128, "mixed"), (1, 70, 130, 640, 2, 100, "runs"),
    (16, 20, 2000, 160, 3, 16, "mixed"), (2, 130, 520, 288, 9, 64, "mixed"), (1, 300, 300, 1056, 40, 31, "each"),
    (8, 700, 2500, 200, 4, 17, "runs"), (16, 260, 2050, 96, 2, 16, "runs"), (1, 40, 100, 3500, 2, 7, "none"),
    (3, 5, 30, 2080, 1, 40, "each"), (16, 100, 2000, 224, 3, 48, "mixed"),
]


@pytest.mark.parametrize("yf", ["bf16", "f32"])
@pytest.mark.parametrize("xf", ["bf16", "row8", "mx8", "mx4"])
@pytest.mark.parametrize("size", SIZES, ids=[str(i) for i in range(len(SIZES))])
def test_random(size, xf, yf):
    ranks, m, n, k, count, rank, kind = size
    Case(1, ranks, m, n, k, xf, yf, count, rank, _index(kind, m, count), columns=m % 2 == 1).run()


@pytest.mark.parametrize("yf", ["bf16", "f32"])
@pytest.mark.parametrize("xf", ["bf16", "row8", "mx8", "mx4"])
@pytest.mark.parametrize("size", [(1, 1, 40, 64, 2, 16, "each"), (2, 16, 100, 130, 7, 9, "mixed"), (1, 130, 200, 128, 3, 40, "mixed"),
                                  (4, 300, 300, 96, 2, 17, "runs"), (1, 300, 600, 64, 300, 3, "each")])
def test_dyadic_numbers_are_exact(size, xf, yf):
    """x and w within 12 * 2, a within 1: t is a multiple of 2^-5 below 2^11, so all of it is in two parts."""
    ranks, m, n, k, count, rank, kind = size
    Case(2, ranks, m, n, k, xf, yf, count, rank, _index(kind, m, count), dyadic=True, columns=ranks == 2).run()


@pytest.mark.parametrize("m", [5, 40])
def test_without_scales_and_without_adapters(m):
    Case(3, 2, m, 70, 200, "mx8", "bf16", 3, 16, _index("mixed", m, 3), scales=False).run()
    c = Case(4, 2, m, 70, 200, "mx8", "bf16", 3, 16, _index("mixed", m, 3))
    lin, ad = c.params()
    abi.ar_mx4_linear(lin)
    torch.cuda.synchronize()
    alone = c.y.view(torch.int16).clone()
    for name in ("adapters", "rank"):
        lin, ad = c.params()
        setattr(ad, name, 0)
        c.y.fill_(-77.0)
        abi.ar_mx4_linear_adapters(lin, ad, None)
        torch.cuda.synchronize()
        assert torch.equal(c.y.view(torch.int16), alone)


@pytest.mark.parametrize("m,n", [(7, 100), (16, 5000), (100, 200)])
def test_tokens_without_an_adapter_keep_the_layers_bits(m, n):
    """... and those of one adapter do not depend on their neighbours'."""
    c = Case(5, 2, m, n, 300, "mx4" if m == 7 else "bf16", "f32", 4, 16, _index("mixed", m, 4, 9))
    lin, ad = c.params()
    abi.ar_mx4_linear(lin)
    torch.cuda.synchronize()
    alone = c.y.clone()
    c.run()
    both = c.y.clone()
    none = torch.from_numpy((c.index < 0) | (c.index >= 4)).cuda()
    assert torch.equal(both[:, none], alone[:, none])
    c.idx.fill_(2)
    abi.ar_mx4_linear_adapters(lin, ad, c.work(lin, ad))
    torch.cuda.synchronize()
    two = torch.from_numpy(c.index == 2).cuda()
    assert torch.equal(c.y[:, two], both[:, two])


@pytest.mark.parametrize("m", [4, 50])
def test_infinite_and_nan_adapters_stay_with_their_tokens(m):
    c = Case(6, 1, m, 90, 200, "bf16", "f32", 4, 20, np.arange(m) % 4)
    c.ad[0, 1] = float("nan")
    c.bd[0, 2] = float("inf")
    lin, ad = c.params()
    abi.ar_mx4_linear_adapters(lin, ad, c.work(lin, ad))
    torch.cuda.synchronize()
    y = c.y[0, :, :90]
    kind = torch.arange(m, device="cuda") % 4
    assert y[kind == 1].isnan().all() and not y[kind == 2].isfinite().any()
    assert y[(kind == 0) | (kind == 3)].isfinite().all()


@pytest.mark.parametrize("rank", [7, 16, 40])
@pytest.mark.parametrize("ranks,m,n", [(16, 200, 2050), (8, 520, 2600)])       # tiles of 128 and 256
def test_tokens_of_large_tiles_keep_to_themselves(ranks, m, n, rank):
    """Neither a neighbour's adapter nor infinities and NaNs in it change a bit
    of a token, with one and two adapters to a matrix instruction."""
    c = Case(11, ranks, m, n, 96, "bf16", "f32", 5, rank, _index("mixed", m, 5, 3))
    lin, ad = c.params()
    abi.ar_mx4_linear(lin)
    torch.cuda.synchronize()
    alone = c.y.clone()
    abi.ar_mx4_linear_adapters(lin, ad, c.work(lin, ad))
    torch.cuda.synchronize()
    c.check()
    both = c.y.clone()
    index = c.idx.clone()
    none, other = (index < 0) | (index >= 5), (index != 1) & (index != 2)
    assert torch.equal(both[:, none], alone[:, none])
    c.ad[0, 1] = float("nan")
    c.bd[0, 2, :, rank - 1] = float("inf")
    c.bd[0, 2, 5] = float("nan")
    abi.ar_mx4_linear_adapters(lin, ad, c.work(lin, ad))
    torch.cuda.synchronize()
    assert torch.equal(c.y[:, other], both[:, other])
    assert c.y[0, index == 1, :n].isnan().all()          # a is a rank's own, b all ranks'
    assert not c.y[:, index == 2, :n].isfinite().any()
    c.idx[other] = -1
    abi.ar_mx4_linear_adapters(lin, ad, c.work(lin, ad))
    torch.cuda.synchronize()
    assert torch.equal(c.y[:, other], alone[:, other])
    c.idx.copy_(index)
    c.idx[~other] = -1
    abi.ar_mx4_linear_adapters(lin, ad, c.work(lin, ad))
    torch.cuda.synchronize()
    assert torch.equal(c.y[:, other], both[:, other])


def test_far_adapters():
    """Adapters more than 2^31 elements apart from the first."""
    c = Case(7, 1, 6, 70, 200, "mx8", "bf16", 2, 16, [0, 1, 1, 0, 1, 0])
    step = (1 << 31) + 64
    lin, ad = c.params()
    a = torch.empty(step + c.ad[0, 1].numel(), dtype=torch.bfloat16, device="cuda")
    b = torch.empty(step + c.bd[0, 1].numel(), dtype=torch.bfloat16, device="cuda")
    for far, near in ((a, c.ad[0]), (b, c.bd[0])):
        far[:near[0].numel()] = near[0].flatten()
        far[step:] = near[1].flatten()
    far = abi.adapter_params(2, 16, c.idx, c.sc, a, c.ad.stride(2), step, 0, b, c.bd.stride(2), step, 0)
    abi.ar_mx4_linear_adapters(lin, far, c.work(lin, far))
    torch.cuda.synchronize()
    c.check()


def test_rows_of_more_than_2_31_bits():
    """Inputs whose number times 16 passes 31 bits: of zeros but for a few places
    near both ends and around 2^26 and 2^27 (the sums are exact)."""
    m, n, k, rank = 33, 16, (1 << 27) + 40, 16
    rng = np.random.default_rng(10)
    at = np.array([0, 1, 511, (1 << 26) - 1, (1 << 26), (1 << 27) - 1, (1 << 27), k - 1])
    x = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
    a = torch.zeros((rank, k), dtype=torch.bfloat16, device="cuda")
    xv, av, bv = (rng.integers(-2, 3, s) / 2.0 for s in ((m, len(at)), (rank, len(at)), (n, rank)))
    cols = torch.from_numpy(at).cuda()
    x[:, cols] = torch.from_numpy(xv).to(torch.bfloat16).cuda()
    a[:, cols] = torch.from_numpy(av).to(torch.bfloat16).cuda()
    b = torch.from_numpy(bv).to(torch.bfloat16).cuda()
    nb = -(-k // 32)
    w = torch.zeros((n, 16 * nb), dtype=torch.uint8, device="cuda")
    ws = torch.full((n, (nb + 15) // 16 * 16), 127, dtype=torch.uint8, device="cuda")
    y = torch.full((m, n), -77.0, device="cuda")
    index = torch.zeros(m, dtype=torch.int32, device="cuda")
    index[5] = -1
    lin = abi.linear_params(1, m, n, k, "bf16", x, x.stride(0), 0, None, 0, 0, w, w.stride(0), 0, ws, ws.stride(0), 0,
                            "f32", y, y.stride(0), 0)
    ad = abi.adapter_params(1, rank, index, None, a, a.stride(0), 0, 0, b, b.stride(0), 0, 0)
    work = torch.full((abi.ar_adapter_work_bytes(lin, ad) // 4,), float("nan"), device="cuda")
    abi.ar_mx4_linear_adapters(lin, ad, work)
    torch.cuda.synchronize()
    want = xv @ av.T @ bv.T
    want[5] = 0.0
    assert np.array_equal(y.double().cpu().numpy(), want)


def test_two_streams_and_a_replayed_graph():
    one, two = Case(8, 4, 16, 500, 640, "mx8", "bf16", 6, 16, _index("each", 16, 6)), Case(9, 1, 90, 200, 300, "mx4", "f32", 3, 40, _index("mixed", 90, 3))
    p1, p2 = one.params(), two.params()
    w1, w2 = one.work(*p1), two.work(*p2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        abi.ar_mx4_linear_adapters(*p1, w1, s1)
        abi.ar_mx4_linear_adapters(*p2, w2, s2)
    torch.cuda.synchronize()
    one.check()
    two.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        abi.ar_mx4_linear_adapters(*p1, w1)
    for seed in range(3):                      # the tokens' adapters are read when the graph runs
        one.index = _index("mixed", 16, 6, seed)
        one.idx.copy_(torch.from_numpy(one.index.astype(np.int32)))
        one.y.fill_(-77.0)
        g.replay()
        torch.cuda.synchronize()
        one.check()
