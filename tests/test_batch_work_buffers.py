"""The work buffers of the operators for a batch of many requests, on the host: a
buffer for the largest batch does for every smaller one."""
import ctypes
import random

import pytest

from collective_synchronization_amd import abi

A = 1 << 20            # an address aligned to everything


def _linear(rows, ranks=1, outputs=8192, inputs=8192, x_fmt="mx8", shared=False):
    bits = {"bf16": 16, "row8": 8, "mx8": 8, "mx4": 4}[x_fmt]
    xs = inputs if bits > 4 else inputs // 2
    ws = -(-inputs // 128) * 4
    scales = {"bf16": 0, "row8": 1}.get(x_fmt, ws)
    return abi.linear_params(ranks, rows, outputs, inputs, x_fmt, A, xs, 0 if shared else rows * xs, A, scales,
                             0 if shared else rows * scales, A, inputs // 2, outputs * (inputs // 2), A, ws,
                             outputs * ws, "bf16", A, outputs, rows * outputs)


def _adapters(rank, inputs, outputs, adapters=8):
    r8 = -(-rank // 8) * 8
    return abi.adapter_params(adapters, rank, A, None, A, inputs, rank * inputs, 0, A, r8, outputs * r8, 0)


@pytest.mark.parametrize("ranks,outputs,inputs,rank,x_fmt,shared", [
    (1, 8192, 8192, 16, "mx8", False), (4, 8192, 2048, 16, "mx8", False), (8, 4096, 512, 16, "bf16", False),
    (2, 4000, 2080, 24, "mx4", True), (1, 256, 256, 128, "row8", False), (8, 8192, 1024, 64, "bf16", True),
    (1, 131072, 512, 4, "mx8", False)])
def test_fewer_tokens_need_no_larger_buffer(ranks, outputs, inputs, rank, x_fmt, shared):
    last = 0
    for rows in [*range(0, 600), *range(600, 5000, 37), 8192, 20000, 32768, 40000, 100000]:
        lin, ad = _linear(rows, ranks, outputs, inputs, x_fmt, shared), _adapters(rank, inputs, outputs)
        need = abi.ar_adapter_work_bytes(lin, ad)
        assert need >= last and need % 256 == 0, rows
        if rows:
            # t and nothing less, and the refusal is of what the function says
            assert need >= (1 if shared else ranks) * rows * rank * 4
            run = abi.raw().ar_mx4_linear_adapters
            assert run(ctypes.byref(lin), ctypes.byref(ad), A, need - 1, None) == -3
        last = need


def test_a_step_of_single_tokens_needs_little():
    """The promise costs a decode step no more than its own rows."""
    for rows in (1, 16, 32):
        need = abi.ar_adapter_work_bytes(_linear(rows), _adapters(16, 8192, 8192))
        assert need <= rows * (64 + 8192 * 4) + 512


def _attend(**kw):
    d = dict(sequences=2, queries=1, heads=8, scale=0.1, fmt="bf16", q=A, q_stride=1 << 14, q_head_stride=256, out=A,
             out_stride=1 << 14, out_head_stride=256, lse=None, lse_stride=0, prefix=100, prefix_pages=A, lengths=A,
             pages=A, pages_stride=1 << 20, max_pages=5)
    page, kv, dim = kw.pop("page", 64), kw.pop("kv", 4), kw.pop("dim", 128)
    d.update(kw)
    cache = abi.cache_params("bf16", 10, page, kv, dim, A, A, page * kv * dim, kv * dim, dim)
    return abi.attention_params(cache, **d)


def test_smaller_batches_need_no_larger_buffer():
    """Fewer sequences, a shorter prefix or fewer pages, one or all of them, with the other sizes the same."""
    rng = random.Random(3)
    for _ in range(400):
        kv = rng.choice([1, 2, 4, 8])
        fixed = dict(kv=kv, heads=kv * rng.choice([1, 3, 8]), queries=rng.choice([1, 2, 5, 64]),
                     dim=rng.choice([16, 64, 96, 128, 256]), page=rng.choice([16, 64, 1024]))
        big = dict(sequences=int(2 ** rng.uniform(0, 9)), prefix=int(2 ** rng.uniform(0, 18)) - 1,
                   max_pages=int(2 ** rng.uniform(0, 12)) - 1)
        p = _attend(**fixed, **big)
        need = abi.ar_prefix_attention_work_bytes(p)
        rows = big["sequences"] * fixed["queries"] * fixed["heads"]
        parts = (big["prefix"] > 0) + (big["max_pages"] > 0)
        assert need >= parts * rows * (fixed["dim"] + 2) * 4
        if need:
            assert abi.raw().ar_prefix_attention(ctypes.byref(p), A, need - 1, None) == -3
        for _ in range(10):
            small = {k: rng.choice([v, rng.randint(1 if k == "sequences" else 0, v)]) for k, v in big.items()}
            assert abi.ar_prefix_attention_work_bytes(_attend(**fixed, **small)) <= need, (fixed, big, small)
