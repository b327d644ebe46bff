"""The all-reduce with the residual norm, started before its payloads: pieces
of the receive buffers arrive one after the other, in several orders, while
the call polls on another stream.  Every wait has a deadline of its own, so a
piece that did not arrive would end the call with AR_ETIMEOUT."""
import time

import numpy as np
import pytest
import torch

from collective_synchronization_amd import abi, buffers, inputs
from layer_cases import float_rows, out_rows, to_type
from test_gpu_reduce_norm import _check, _h

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def streams():
    """Two streams whose kernels can run beside each other: a pair may share a
    hardware queue, where the second waits for the first to end."""
    ws = buffers.Workspace(2, 512, "ll")
    y = torch.zeros((1, 512), dtype=torch.bfloat16, device="cuda")
    p = abi.norm_params(1, 512, 1e-5, "bf16", None, "bf16", None, 0, None, 0, "bf16", y, 512)
    t = torch.zeros((8, 8), device="cuda")
    waits = torch.cuda.Stream()
    for _ in range(8):
        sends = torch.cuda.Stream()
        torch.cuda.synchronize()
        ws.reduce_norm(p, timeout_ns=200_000_000, stream=waits)      # nobody sends: 0.2 s
        with torch.cuda.stream(sends):
            t[:, :4].add_(1.0)
            done = sends.record_event()
        time.sleep(0.05)
        beside = done.query()
        torch.cuda.synchronize()
        ws.reset_ctrl()
        if beside:
            return waits, sends
    pytest.skip("no two streams here run beside each other")


class Call:
    """A packed copy of the receive buffers, and the call that waits for it."""

    def __init__(self, streams, proto, nranks=4, ncons=1, rows=1, hidden=16384, y_fmt="mx8", seed=0):
        self.rows, self.hidden = rows, hidden
        count = rows * hidden
        rng = np.random.default_rng(seed)
        self.bits = inputs.payload(seed, (nranks, count))
        self.res = to_type(rng.standard_normal((ncons * rows, hidden)), "f32")
        self.y_fmt = y_fmt
        xd, stride = buffers.rows_to_device(self.bits)
        source, self.ws = (buffers.Workspace(nranks, count, proto, ncons) for _ in range(2))
        source.pack(xd, stride)
        slot = abi.ar_desc_slot_bytes(source.desc)
        shape = (ncons, 2, nranks, slot)

        def sent(ws):
            return ws.scratch[:ws.scratch_bytes].view(shape)[:, ws.epoch.parity]
        self.source, self.target = sent(source), sent(self.ws)
        self.rd = float_rows(self.res, "f32")
        self.out, self.y = out_rows(ncons * rows, hidden, "f32"), out_rows(ncons * rows, hidden, y_fmt)
        self.p = abi.norm_params(rows, hidden, 1e-5, "bf16", None, "f32", self.rd.data, self.rd.stride, self.out.data,
                                 self.out.stride, y_fmt, self.y.data, self.y.stride, self.y.scales,
                                 self.y.scale_stride)
        # the kernels are loaded before the clock matters
        warm = buffers.Workspace(nranks, count, proto, ncons)
        warm.pack(xd, stride)
        warm.reduce_norm(self.p, timeout_ns=2_000_000_000)
        self.out.data.fill_(-77.0)
        self.y.data.fill_(0xA5)
        self.y.scales.fill_(0xA5)
        self.waits, self.sends = streams
        with torch.cuda.stream(self.sends):
            scrap = torch.zeros_like(self.target)
            scrap[..., :8].copy_(self.source[..., :8])
        torch.cuda.synchronize()

    def run(self, pieces, pause, timeout_ns):
        """Start the call, then send each piece (an index of the buffers)."""
        self.ws.reduce_norm(self.p, timeout_ns=timeout_ns, stream=self.waits)
        for at in pieces:
            time.sleep(pause)
            with torch.cuda.stream(self.sends):
                self.target[at].copy_(self.source[at])
            self.sends.synchronize()
        torch.cuda.synchronize()
        return self.ws.status()

    def check(self):
        _check(self.out, self.y, _h(self.bits, self.res, self.rows, self.hidden), "f32", None, self.y_fmt)


def _ranks(n, order):
    return [(slice(None), r) for r in order(range(n))]


def _spans(size, step):
    return [(slice(None), slice(None), slice(i, min(i + step, size))) for i in range(0, size, step)]


@pytest.mark.parametrize("proto", ("ll", "ll128", "sentinel"))
@pytest.mark.parametrize("order", ("whole", "ranks", "reverse"))
@pytest.mark.parametrize("ncons,rows,hidden", ((1, 1, 16384), (4, 3, 520), (1, 2, 8192)))
def test_payloads_after_the_call(streams, proto, order, ncons, rows, hidden):
    print(f"[arrival] {proto} {order} C={ncons} {rows}x{hidden}", flush=True)
    c = Call(streams, proto, ncons=ncons, rows=rows, hidden=hidden, seed=hidden + rows)
    if order == "whole":
        pieces = [(slice(None),)]
    else:
        pieces = _ranks(4, list if order == "ranks" else lambda r: list(reversed(r)))
    if proto == "ll128":                                # data of a line before its flag
        lines = c.source.shape[-1] // 128
        c.source = c.source.reshape(*c.source.shape[:-1], lines, 128)
        c.target = c.target.unflatten(-1, (lines, 128))
        pieces = [at + (Ellipsis, part) for at in pieces for part in (slice(0, 120), slice(120, 128))]
    assert c.run(pieces, 0.002, 5_000_000_000) == 0
    c.check()


@pytest.mark.parametrize("proto", ("ll", "sentinel"))
@pytest.mark.parametrize("backwards", (False, True))
def test_spans_of_a_row_one_by_one(streams, proto, backwards):
    """16-byte words of all ranks a few thousand at a time, from either end."""
    c = Call(streams, proto, hidden=16384, seed=5)
    pieces = _spans(c.source.shape[-1], 5 * 512 - 16)
    assert c.run(pieces[::-1] if backwards else pieces, 0.001, 5_000_000_000) == 0
    c.check()


@pytest.mark.parametrize("proto", ("ll", "sentinel"))
def test_one_deadline_for_a_row(streams, proto):
    """A thread has four chunks of this row; they come 0.3 s apart, and 0.4 s is
    the deadline for all four."""
    c = Call(streams, proto, nranks=2, hidden=16384, seed=6)
    pieces = _spans(c.source.shape[-1], c.source.shape[-1] // 4)
    assert c.run(pieces, 0.3, 400_000_000) == abi.AR_ETIMEOUT
    assert bool((c.out.data == -77.0).all()) and bool((c.y.data == 0xA5).all())
