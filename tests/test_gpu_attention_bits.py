"""Attention over a shared prefix and paged own tokens on the GPU: equal calls
give equal bits, whatever shared memory held before."""
import pytest
import torch

from collective_synchronization_amd import abi, buffers
from test_gpu_attention import Batch

pytestmark = pytest.mark.gpu


def _leave_in_shared_memory(dim, value):
    """Tiles of keys and values that are all `value` through every CU's shared
    memory: a prefix of 16384 bf16 tokens for 8 heads of the cache and 64 rows of each."""
    cache = buffers.PagedCache(256, 64, 8, dim, "bf16")
    cache.k.fill_(value)
    cache.v.fill_(value)
    q = torch.ones((64, 8, dim), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    pages = torch.arange(256, dtype=torch.int32, device="cuda")
    lengths = torch.zeros(64, dtype=torch.int32, device="cuda")
    p = abi.attention_params(cache.params, 64, 1, 8, 1.0, "bf16", q, 8 * dim, dim, out, 8 * dim, dim, None, 0,
                             16384, pages, lengths, None, 0, 0)
    abi.ar_prefix_attention(p, buffers.device_bytes(abi.ar_prefix_attention_work_bytes(p)))
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", ["bf16", "f16"])
@pytest.mark.parametrize("queries", [2, 9])                # up to 16 rows of a sequence, and more
@pytest.mark.parametrize("dim", [48, 80, 96, 128, 144, 192, 224])
def test_bits_do_not_depend_on_what_shared_memory_held(dim, queries, fmt):
    """8-bit rows of heads that do not fill their places in shared memory: what an earlier kernel left behind them is
    no value.  Every sequence ends inside a tile, where some tokens do not see all keys."""
    lengths = [20 + 13 * i for i in range(24)]
    b = Batch(4, lengths, queries, 8, 2, dim, 16, 70, fmt, "row8", poison=False)
    p = b.params()
    work = b.work(p)
    seen = []
    for value in (0.0, float("inf"), 0.0, float("nan")):
        _leave_in_shared_memory(128 if dim <= 128 else 256, value)
        abi.ar_prefix_attention(p, work)
        torch.cuda.synchronize()
        seen.append((b.out.view(torch.int16).clone(), b.lse.view(torch.int32).clone()))
    for out, lse in seen[1:]:
        assert torch.equal(lse, seen[0][1]) and torch.equal(out, seen[0][0])
    b.check()


@pytest.mark.parametrize("queries", [1, 2, 9])
@pytest.mark.parametrize("dim", [64, 96, 192])
@pytest.mark.parametrize("fmt,cache", [("bf16", "same"), ("f16", "same"), ("bf16", "row8"), ("f16", "row8")])
def test_equal_calls_give_equal_bits_in_every_form(fmt, cache, dim, queries):
    """Several calls, their inputs laid out anew, with other work in between."""
    outs = []
    for i in range(3):
        b = Batch(9, (900, 300, 20, 77), queries, 8, 2, dim, 16, 1000, fmt, cache)
        if i:
            _leave_in_shared_memory(128 if i == 1 else 256, 3.0)
        b.run()
        outs.append((b.out.view(torch.int16).clone(), b.lse.view(torch.int32).clone()))
    for o, l in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(l, outs[0][1])
