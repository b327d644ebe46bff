"""Attention over a shared prefix and paged own tokens on the GPU, against the
64-bit form of oracle/cache.py.

The bound on out: a weight is known to e = what its score is off by (dim
products summed in binary32, 2^-23 a step since the matrix cores may truncate,
of at most sum |q||k| scale; the rounding of score * log2(e) - reference, two
of 2^-24 of the largest score; the exponential's own 2^-22), then rounded to 16
bits (u), so sum w v is off by u + 2e of sum w |v|, and by 2^-23 of it for
each addition; the joined row is rounded once more (u of itself).  fp16
weights below 2^-20 of the largest are off by 2^-31 of it instead of u.  (With
8-bit values fp16 weights are two bf16 parts, off by 2^-16.)
"""
import numpy as np
import pytest
import torch

from collective_synchronization_amd import abi, buffers
from oracle import cache as oc
from oracle import layer

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def _round(v, fmt):
    return torch.from_numpy(np.asarray(v, dtype=np.float32)).to(TORCH[fmt]).double().numpy()


class Batch:
    """Inputs of one call: values in binary64 and their device forms."""

    def __init__(self, seed, lengths, queries, heads, kv, dim, page, prefix, fmt="bf16", cache="same", spare=2,
                 sharp=1.0, width=None, head_major=False, pad=0, poison=True, pages=None):
        rng = np.random.default_rng(seed)
        self.lengths, self.queries, self.heads, self.kv, self.dim = list(lengths), queries, heads, kv, dim
        self.fmt, self.prefix, self.page, self.scale = fmt, prefix, page, dim ** -0.5
        n = len(self.lengths)
        need = [-(-max(x, 0) // page) for x in self.lengths]
        width = max(1, max(need, default=0)) if width is None else width
        shared = -(-prefix // page)
        count = shared + sum(min(x, width) for x in need) + spare if pages is None else pages
        order = rng.permutation(count)
        self.prefix_pages = order[:shared].astype(np.int32)
        self.pages = np.full((n, width), -1, dtype=np.int32)
        at = shared
        for i, x in enumerate(need):
            x = min(x, width)
            self.pages[i, :x] = order[at:at + x]
            at += x
        shape = (count, page, kv, dim)
        self.k, self.v = rng.standard_normal(shape), rng.standard_normal(shape)
        self.q = _round(rng.standard_normal((n * queries, heads, dim)) * sharp, fmt)
        used = np.zeros((count, page), dtype=bool)
        p, s, _ = oc.tokens(self.prefix_pages, prefix, page, count)
        used[p, s] = True
        for i, x in enumerate(self.lengths):
            p, s, _ = oc.tokens(self.pages[i], max(x, 0), page, count)
            used[p, s] = True
        scales = {}
        for name in ("k", "v"):
            x = getattr(self, name)
            if cache == "row8":
                rows = x.reshape(-1, dim)
                sc = (np.abs(rows).max(-1) / 448).astype(np.float32)
                codes = layer.signed_codes(rows / sc[:, None].astype(np.float64), layer.E4M3, 128)
                x = layer.dequantize(codes, sc, "row8", dim).reshape(shape)
                codes, sc = codes.reshape(shape), sc.reshape(shape[:3])
                if poison:
                    codes[~used], sc[~used] = 0x7F, np.nan
                setattr(self, name, x)
                dev = torch.from_numpy(codes)
                scales[name] = torch.from_numpy(sc).cuda()
            else:
                x = _round(x, fmt)
                setattr(self, name, x)
                host = x.copy()
                if poison:
                    host[~used] = rng.choice([np.nan, np.inf, -np.inf], size=host[~used].shape)
                dev = torch.from_numpy(host).to(TORCH[fmt])
            if head_major:                       # [pages, heads, page, dim]
                dev = dev.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3)
            else:
                dev = dev.cuda()
            setattr(self, name + "d", dev)
        kd = self.kd
        ks, vs = scales.get("k"), scales.get("v")
        self.cache = abi.cache_params("row8" if cache == "row8" else fmt, count, page, kv, dim, kd, self.vd,
                                      *kd.stride()[:3], ks, vs, *(ks.stride() if ks is not None else ()))
        self.n = n
        rows = n * queries
        self.qd = torch.full((rows, heads, dim + pad), float("nan"), dtype=TORCH[fmt], device="cuda")
        self.qd[..., :dim] = torch.from_numpy(self.q).to(TORCH[fmt])
        self.out = torch.full((rows + 1, heads, dim + pad), -77.0, dtype=TORCH[fmt], device="cuda")
        self.lse = torch.full((rows + 1, heads + pad), -77.0, device="cuda")
        self.dev = [torch.from_numpy(np.ascontiguousarray(x)).cuda() if x.size else None
                    for x in (self.prefix_pages, np.asarray(self.lengths, dtype=np.int32), self.pages)]

    def params(self, lse=True):
        q, o = self.qd, self.out
        pp, ln, pg = self.dev
        return abi.attention_params(self.cache, self.n, self.queries, self.heads, self.scale, self.fmt, q, q.stride(0),
                                    q.stride(1), o, o.stride(0), o.stride(1), self.lse if lse else None,
                                    self.lse.stride(0) if lse else 0, self.prefix, pp, ln, pg, self.pages.shape[1],
                                    self.pages.shape[1])

    def work(self, p):
        # filled with NaN: nothing may be read that was not written
        n = abi.ar_prefix_attention_work_bytes(p)
        return torch.full((max(64, n // 4),), float("nan"), device="cuda")

    def run(self, lse=True):
        p = self.params(lse)
        abi.ar_prefix_attention(p, self.work(p))
        torch.cuda.synchronize()
        self.check(lse)

    def check(self, lse=True):
        rows = self.n * self.queries
        out, dim = self.out.double().cpu().numpy(), self.dim
        got_lse = self.lse.double().cpu().numpy()
        assert (out[rows:] == -77.0).all() and (out[..., dim:] == -77.0).all()
        want, wl, size, top, mass = oc.attention(self.q, self.k, self.v, self.scale, self.prefix, self.prefix_pages,
                                                 self.lengths, self.pages, self.queries)
        absent = np.isnan(wl)
        got, gl = out[:rows, :, :dim], got_lse[:rows, :self.heads]
        assert (got[absent] == -77.0).all()
        keys = self.prefix + max(max(self.lengths, default=0), 0)
        e = dim * 2.0 ** -23 * mass + 2 * 2.0 ** -24 * top * 1.4427 + 2.0 ** -22
        u = U[self.fmt]
        vmax = max(np.abs(self.v).max(), 1.0)
        tol = size * (u + 2 * e[..., None] + keys * 2.0 ** -23) + u * np.abs(want) + 2.0 ** -25
        if self.fmt == "f16":
            tol = tol + keys * 2.0 ** -31 * vmax
        ok = absent[..., None] | (np.abs(got - want) <= tol)
        assert ok.all(), (np.argwhere(~ok)[:5], got[~ok][:5], want[~ok][:5])
        if not lse:
            assert (got_lse == -77.0).all()
            return
        assert (got_lse[rows:] == -77.0).all() and (got_lse[:, self.heads:] == -77.0).all()
        assert (gl[absent] == -77.0).all()
        none = np.isneginf(wl)
        assert (gl[none] == -np.inf).all() and (got[none] == 0).all()
        fine = ~absent & ~none
        # the sum of weights known to e, its logarithm, and two roundings
        tl = e + keys * 2.0 ** -23 + 2.0 ** -21 + 4 * 2.0 ** -24 * np.abs(wl)
        assert (np.abs(gl[fine] - wl[fine]) <= tl[fine]).all()


SHAPES = [
    # lengths, queries, heads, kv, dim, page, prefix
    ((1,), 1, 1, 1, 16, 16, 0), ((1,), 1, 1, 1, 16, 16, 1), ((0,), 1, 2, 1, 32, 16, 5), ((0,), 1, 2, 2, 64, 16, 0),
    ((33,), 1, 8, 2, 64, 16, 0), ((31, 32, 33, 0, 1), 1, 4, 4, 128, 32, 63), ((500,), 1, 32, 8, 128, 16, 1000),
    ((129, 7, 64), 1, 16, 1, 128, 64, 300),                       # 16 rows a sequence, 48 behind the prefix
    ((129, 7, 64), 1, 17, 1, 80, 16, 65),                         # 17: the other form
    ((90, 1, 0, 200), 4, 8, 1, 96, 32, 127),                      # 32 rows a sequence
    ((40, 300), 5, 64, 2, 128, 16, 200),                          # 160 rows: two tiles
    ((70,) * 20, 1, 8, 1, 192, 128, 1), ((70,) * 20, 2, 4, 1, 256, 16, 100), ((3, 2, 1), 4, 6, 2, 112, 16, 40),
    ((700, 0, -1, 333, 16, 15), 1, 10, 2, 128, 64, 129), ((-1, -5), 2, 4, 2, 64, 16, 50),
    ((2000,), 1, 4, 1, 256, 1024, 0), ((40,) * 130, 1, 1, 1, 48, 16, 90), ((0,) * 3, 3, 4, 1, 64, 16, 600),
]


@pytest.mark.parametrize("cache", ["same", "row8"])
@pytest.mark.parametrize("fmt", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
def test_attention(shape, fmt, cache):
    Batch(3, *shape, fmt=fmt, cache=cache).run()


@pytest.mark.parametrize("cache", ["same", "row8"])
@pytest.mark.parametrize("dim", [16, 64, 96, 128, 160, 208, 256])
@pytest.mark.parametrize("queries", [1, 6])
def test_head_sizes_layouts_and_strides(dim, queries, cache):
    Batch(dim, (45, 130, 3), queries, 12, 3, dim, 32, 77, "bf16", cache, head_major=True, pad=16).run()


@pytest.mark.parametrize("queries", [1, 9])
def test_sharp_scores_and_no_lse(queries):
    """Scores of +-60 and more: one key takes all the weight, and references move far."""
    Batch(1, (300, 17), queries, 8, 4, 128, 16, 513, "f16", sharp=20.0).run()
    Batch(1, (300, 17), queries, 8, 4, 128, 16, 513, "bf16", sharp=20.0).run(lse=False)


@pytest.mark.parametrize("cache", ["same", "row8"])
@pytest.mark.parametrize("group", [1, 5, 8])
def test_many_tokens_of_a_step(group, cache):
    """Several tiles of a sequence's rows, whose tokens stop at different keys, or before the first."""
    Batch(8, (150, 149, 20, 0, 400, -1, 290), 150, 2 * group, 2, 64, 16, 33, "bf16", cache).run()
    Batch(9, (150, 1000), 150, 2 * group, 2, 128, 64, 0, "f16", cache).run()


@pytest.mark.parametrize("queries", [1, 3])
def test_rising_scores(queries):
    """Every key scores more than all before it, by steps around the slack of the reference."""
    b = Batch(2, (400, 64), queries, 8, 1, 64, 16, 640, "bf16", poison=False)
    b.q[:] = 1.0
    b.qd.fill_(1.0)
    step = np.zeros((b.k.shape[0], 16))
    for t, p in enumerate(b.prefix_pages):
        step[p] = (16 * t + np.arange(16)) / 8
    for i in range(b.n):
        for t, p in enumerate(b.pages[i]):
            if p >= 0:
                step[p] = 80 + (16 * t + np.arange(16)) / 4
    b.k = _round(np.broadcast_to(step[:, :, None, None] / 8, b.k.shape), "bf16")
    b.kd.copy_(torch.from_numpy(b.k).to(torch.bfloat16))
    b.run()


@pytest.mark.parametrize("queries", [1, 20])
def test_pages_that_are_not_there(queries):
    """Table entries outside the cache, in the prefix's list and in a sequence's: their tokens do not count."""
    b = Batch(5, (200, 90), queries, 4, 2, 64, 16, 100)
    b.pages[0, 3], b.pages[0, 7], b.pages[1, 0] = -1, b.k.shape[0], 2 ** 31 - 1
    b.prefix_pages[2] = -2 ** 31
    b.dev[2].copy_(torch.from_numpy(b.pages))
    b.dev[0].copy_(torch.from_numpy(b.prefix_pages))
    b.run()


def test_lengths_past_the_table():
    """What lies past the table's pages does not count; the tokens keep their places."""
    Batch(6, (200, 33), 2, 4, 2, 64, 16, 20, width=3).run()


@pytest.mark.parametrize("queries", [1, 9])
def test_infinite_and_nan_keys(queries):
    """A key of -inf takes no weight; a NaN among the keys seen is seen by every row of its sequence, and by no other."""
    b = Batch(7, (50, 50), queries, 4, 1, 64, 16, 30, poison=False)
    b.q = np.abs(b.q) + 0.25
    b.qd.copy_(torch.from_numpy(b.q).to(torch.bfloat16))
    b.q = b.qd.double().cpu().numpy()
    p, s = int(b.prefix_pages[0]), 3
    b.kd[p, s] = float("-inf")
    b.k[p, s] = -np.inf
    p2 = int(b.pages[1, 0])
    b.kd[p2, 5] = float("nan")
    prm = b.params()
    abi.ar_prefix_attention(prm, b.work(prm))
    torch.cuda.synchronize()
    out = b.out[:2 * queries].double().cpu().numpy()
    assert np.isnan(out[queries:]).all() and np.isfinite(out[:queries]).all()
    keep = b.k.copy()
    keep[p, s] = -1e4
    want = oc.attention(b.q, keep, b.v, b.scale, b.prefix, b.prefix_pages, b.lengths, b.pages, queries)
    assert (np.abs(out - want[0])[:queries] <= 2.0 ** -6 * want[2][:queries]).all()


@pytest.mark.parametrize("fmt,cache,what", [(f, c, w) for f in ("bf16", "f16") for c, w in
                                            (("same", "nan"), ("same", "inf"), ("row8", "nan"), ("row8", "scale"))])
@pytest.mark.parametrize("queries,heads", [(3, 4), (9, 4), (40, 2), (5, 32)])
def test_odd_values_of_later_tokens_are_not_seen(queries, heads, fmt, cache, what):
    """Infinities and NaNs in the keys and values of the step's last token leave the tokens before it as they are."""
    b = Batch(12, (70, 64 + queries), queries, heads, 2, 64, 16, 20, fmt, cache, poison=False)
    for i in range(2):
        at = b.lengths[i] - 1
        p, s = int(b.pages[i, at // 16]), at % 16
        if what == "scale":
            for sc in b.cache.tensors[2:]:
                sc[p, s] = float("inf") if i else float("nan")
        elif cache == "row8":
            b.kd[p, s] = b.vd[p, s] = 0x7F
        else:
            b.kd[p, s] = b.vd[p, s] = float("nan") if what == "nan" else float("inf")
    prm = b.params()
    abi.ar_prefix_attention(prm, b.work(prm))
    torch.cuda.synchronize()
    last = np.arange(2 * queries) % queries == queries - 1
    got = b.out[:2 * queries, :, :64].double().cpu().numpy()
    if what != "scale":                        # (a key's infinite scale can give it the score -inf)
        assert not np.isfinite(got[last]).any(-1).any()
    # the others: as from tokens that are there
    want, _, size, top, mass = oc.attention(b.q, b.k, b.v, b.scale, b.prefix, b.prefix_pages, b.lengths, b.pages, queries)
    e = 64 * 2.0 ** -23 * mass + 2 * 2.0 ** -24 * top * 1.4427 + 2.0 ** -22
    u = U[fmt]
    tol = size * (u + 2 * e[..., None] + 200 * 2.0 ** -23) + u * np.abs(want) + 200 * 2.0 ** -31 * np.abs(b.v).max() + 2.0 ** -25
    assert (np.abs(got - want)[~last] <= tol[~last]).all()


def test_nothing_to_see():
    """No prefix and no pages at all: zeros, and no work buffer."""
    q = torch.ones((3, 4, 32), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full_like(q, -77.0), torch.full((3, 4), -77.0, device="cuda")
    c = abi.cache_params("bf16", 0, 16, 2, 32, None, None, 1024, 64, 32)
    lengths = torch.tensor([0, 5, -1], dtype=torch.int32, device="cuda")
    p = abi.attention_params(c, 3, 1, 4, 1.0, "bf16", q, 128, 32, out, 128, 32, lse, 4, 0, None, lengths, None, 0, 0)
    assert abi.ar_prefix_attention_work_bytes(p) == 0
    abi.ar_prefix_attention(p, None)
    torch.cuda.synchronize()
    assert (out[:2] == 0).all() and (lse[:2] == float("-inf")).all() and (out[2] == -77.0).all() and (lse[2] == -77.0).all()


def test_far_offsets():
    """A cache of more than 2^32 bytes, its last pages in use."""
    page, kv, dim = 128, 8, 128
    count = (5 << 30) // (page * kv * dim * 2)
    c = buffers.PagedCache(count, page, kv, dim, "bf16")
    b = Batch(8, (200, 150), 1, 16, kv, dim, page, 130, poison=False)
    n = b.k.shape[0]
    c.k[count - n:].copy_(b.kd)
    c.v[count - n:].copy_(b.vd)
    for x in (0, 2):
        b.dev[x] = torch.where(b.dev[x] >= 0, b.dev[x] + (count - n), b.dev[x])
    b.cache = c.params
    b.run()


def test_equal_calls_give_equal_bits():
    outs = []
    for _ in range(3):
        b = Batch(9, (900, 300, 20), 1, 16, 2, 128, 16, 2000)
        b.run()
        outs.append((b.out.view(torch.int16).clone(), b.lse.clone()))
    for o, l in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(l, outs[0][1])


def test_two_streams_and_a_replayed_graph():
    a, b = Batch(10, (100, 5), 1, 8, 2, 128, 16, 400), Batch(11, (64,), 3, 8, 2, 64, 16, 30, "f16")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    pa, pb = a.params(), b.params()
    wa, wb = a.work(pa), b.work(pb)
    torch.cuda.synchronize()
    for _ in range(5):
        abi.ar_prefix_attention(pa, wa, streams[0])
        abi.ar_prefix_attention(pb, wb, streams[1])
    torch.cuda.synchronize()
    a.check()
    b.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        abi.ar_prefix_attention(pa, wa)
    for length in (100, 7, 0):                 # lengths are read when the graph runs
        a.lengths[0] = length
        a.dev[1].copy_(torch.tensor(a.lengths, dtype=torch.int32))
        a.out.fill_(-77.0)
        a.lse.fill_(-77.0)
        g.replay()
        torch.cuda.synchronize()
        a.check()
