"""A step's keys and values into the paged cache on the GPU: copies are equal to
the bit, 8-bit rows to the nearest codes under scales within one rounding."""
import numpy as np
import pytest
import torch

from collective_synchronization_amd import abi, buffers
from oracle import cache as oc
from oracle import layer

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16}


def _inputs(seed, lengths, queries, kv, dim, page, fmt, width=None):
    rng = np.random.default_rng(seed)
    n = len(lengths)
    need = [-(-max(x, 0) // page) for x in lengths]
    width = max(1, max(need)) if width is None else width
    count = sum(min(x, width) for x in need) + 2
    order = rng.permutation(count)
    pages = np.full((n, width), -1, dtype=np.int32)
    at = 0
    for i, x in enumerate(need):
        x = min(x, width)
        pages[i, :x] = order[at:at + x]
        at += x
    k, v = (torch.from_numpy(rng.standard_normal((n * queries, kv, dim)) * np.exp2(rng.integers(-20, 10, (n * queries, kv, 1))))
            .to(TORCH[fmt]).cuda() for _ in range(2))
    return pages, count, k, v


def _fill(c):
    for t in (c.k, c.v):
        t.view(torch.uint8 if t.dtype == torch.uint8 else torch.int16).fill_(0x33)
    if c.k_scales is not None:
        c.k_scales.fill_(-77.0)
        c.v_scales.fill_(-77.0)


def _check(c, k, v, lengths, queries, pages, fmt):
    where = oc.places(lengths, queries, pages, c.page, c.pages)
    for src, dst, sc in ((k, c.k, c.k_scales), (v, c.v, c.v_scales)):
        rows = src.double().cpu().numpy()
        if sc is None:
            want = torch.full_like(dst.view(torch.int16), 0x33)
            for r, p, s in where:
                want[p, s] = src[r].view(torch.int16)
            assert torch.equal(dst.view(torch.int16), want)
            continue
        codes, scales = dst.cpu().numpy().copy(), sc.double().cpu().numpy().copy()
        for r, p, s in where:
            for h in range(rows.shape[1]):
                x, got, g = rows[r, h], codes[p, s, h], scales[p, s, h]
                most = np.abs(x).max()
                if not np.isfinite(most):
                    assert np.isnan(g) and (got == 0x7F).all()
                elif most / 448 < 2.0 ** -126:
                    assert g == 2.0 ** -126
                    assert np.array_equal(got, layer.signed_codes(x / 2.0 ** -126, layer.E4M3, 128))
                else:
                    assert abs(g - most / 448) <= most / 448 * 2.0 ** -24
                    # 448 * x is exact in binary64, and a quotient next to a border is not rounded across it
                    assert np.array_equal(got, layer.signed_codes(448 * x / most, layer.E4M3, 128))
            codes[p, s], scales[p, s] = 0x33, -77.0
        assert (codes == 0x33).all() and (scales == -77.0).all()


@pytest.mark.parametrize("cache", ["same", "row8"])
@pytest.mark.parametrize("fmt", ["bf16", "f16"])
@pytest.mark.parametrize("lengths,queries,kv,dim,page", [
    ((1,), 1, 1, 16, 16), ((16, 17, 0, -3, 1000), 1, 8, 128, 16), ((5, 300, 2), 4, 3, 80, 32),
    ((700, 64), 64, 2, 256, 64), ((33,) * 7, 7, 5, 48, 16), ((129,), 129, 1, 192, 128)])
def test_append(lengths, queries, kv, dim, page, fmt, cache):
    pages, count, k, v = _inputs(1, lengths, queries, kv, dim, page, fmt)
    c = buffers.PagedCache(count, page, kv, dim, fmt if cache == "same" else "row8")
    _fill(c)
    c.append(k, v, torch.tensor(lengths, dtype=torch.int32, device="cuda"), torch.from_numpy(pages).cuda())
    torch.cuda.synchronize()
    _check(c, k, v, lengths, queries, pages, fmt)


@pytest.mark.parametrize("fmt", ["bf16", "f16"])
def test_every_16_bit_pattern_to_8_bits(fmt):
    """Rows over all patterns, NaNs and infinities, subnormal numbers and zeros among them."""
    bits = np.random.default_rng(2).permutation(np.arange(65536, dtype=np.uint16).astype(np.int64)).astype(np.uint16)
    order = np.sort(bits.view(np.int16) & 0x7FFF, kind="stable")          # rows of one size each ...
    for rows in (bits, order.astype(np.uint16)):                          # ... and of any
        t = torch.from_numpy(rows.view(np.int16).reshape(64, 16, 64)).cuda().view(TORCH[fmt])
        c = buffers.PagedCache(5, 16, 16, 64, "row8")
        _fill(c)
        pages = np.array([[3, 0, 2, 4]], dtype=np.int32)
        c.append(t, t.flip(0).contiguous(), torch.tensor([64], dtype=torch.int32, device="cuda"),
                 torch.from_numpy(pages).cuda())
        torch.cuda.synchronize()
        _check(c, t, t.flip(0), [64], 64, pages, fmt)


def test_strides_bad_pages_and_a_short_table():
    lengths, queries = (40, 20, 70), 6
    pages, count, k, v = _inputs(3, lengths, queries, 4, 64, 16, "bf16", width=3)
    pages[0, 2], pages[1, 1] = count, -7
    wide = torch.zeros((18, 4, 3, 64), dtype=torch.bfloat16, device="cuda")
    wide[:, :, 0], wide[:, :, 2] = k, v
    c = buffers.PagedCache(count, 16, 4, 64, "bf16")
    _fill(c)
    c.append(wide[:, :, 0], wide[:, :, 2], torch.tensor(lengths, dtype=torch.int32, device="cuda"),
             torch.from_numpy(pages).cuda())
    torch.cuda.synchronize()
    _check(c, k, v, lengths, queries, pages, "bf16")


def test_far_pages():
    c = buffers.PagedCache((5 << 30) // (128 * 8 * 128 * 2), 128, 8, 128, "bf16")
    k, v = (torch.randn((3, 8, 128), device="cuda").bfloat16() for _ in range(2))
    pages = torch.tensor([[0], [c.pages - 1], [c.pages // 2]], dtype=torch.int32, device="cuda")
    c.append(k, v, torch.tensor([1, 128, 5], dtype=torch.int32, device="cuda"), pages)
    for i, s in enumerate((0, 127, 4)):
        assert torch.equal(c.k[int(pages[i])][s], k[i]) and torch.equal(c.v[int(pages[i])][s], v[i])
    assert int((c.k != 0).any(-1).sum()) == 24
