"""PagedCache.append: which shapes and strides it passes on and which it refuses
(no GPU is touched: the call below it is recorded)."""
import pytest
import torch

from collective_synchronization_amd import abi, buffers


@pytest.fixture
def cache(monkeypatch):
    calls = []
    monkeypatch.setattr(abi, "ar_cache_append", lambda *a: calls.append(a))
    c = buffers.PagedCache.__new__(buffers.PagedCache)
    c.fmt, c.pages, c.page, c.kv_heads, c.dim, c.params = abi.AR_BF16, 8, 16, 2, 32, None
    c.calls = calls
    return c


def _rows(n):
    return torch.zeros((n, 2, 32), dtype=torch.bfloat16)


def _table(n, width=3):
    return torch.zeros((n, width), dtype=torch.int32)


def _lengths(n):
    return torch.ones(n, dtype=torch.int32)


@pytest.mark.parametrize("lengths,pages", [
    (_lengths(1), _table(1)),
    (torch.ones((1, 5), dtype=torch.int32)[:, 2], _table(1)),          # one length of a table of them
    (torch.tensor(7, dtype=torch.int32), _table(1)),
    (_lengths(4), _table(4)),
    (torch.ones((4, 1), dtype=torch.int32), _table(4)),
    (_lengths(4), _table(4, 9)[:, 2:5]),
    (_lengths(4), _table(3, 4).t()[:, :1]),                            # one page each
])
def test_passed_on(cache, lengths, pages):
    n = pages.shape[0]
    cache.append(_rows(2 * n), _rows(2 * n), lengths, pages)
    (params, sequences, queries, *_), = cache.calls
    assert (sequences, queries) == (n, 2)


@pytest.mark.parametrize("k,lengths,pages", [
    (_rows(8), torch.ones(8, dtype=torch.int32)[::2], _table(4)),      # lengths apart
    (_rows(8), _lengths(1).expand(4), _table(4)),                      # the same one again
    (_rows(8), _lengths(3), _table(4)),
    (_rows(8), _lengths(4).long(), _table(4)),
    (_rows(8), _lengths(4), _table(4).long()),
    (_rows(8), _lengths(4), _table(4).flatten()),
    (_rows(8), _lengths(4), _table(3, 4).t()),
    (_rows(7), _lengths(4), _table(4)),
    (_rows(8)[..., :16], _lengths(4), _table(4)),
    (_rows(8).flatten(1), _lengths(4), _table(4)),
    (_rows(8).transpose(1, 2).contiguous().transpose(1, 2), _lengths(4), _table(4)),
    (_rows(8).float(), _lengths(4), _table(4)),
])
def test_refused(cache, k, lengths, pages):
    with pytest.raises(ValueError):
        cache.append(k, k, lengths, pages)
    assert not cache.calls
