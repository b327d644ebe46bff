"""Refusals of the operators for a batch of many requests, on the host: every bad
argument comes back as its status before anything is enqueued (no GPU is
touched; the addresses are made up), and what the work buffers have to hold."""
import gc
import weakref

import numpy as np
import pytest
import torch

from collective_synchronization_amd import abi, buffers
from oracle import cache as oc

A = 1 << 20            # an address aligned to everything


def _code(fn, *args, **kw):
    try:
        fn(*args, **kw)
    except abi.ArError as e:
        return e.code
    return 0


# ---------------------------------------------------------------- adapters --

def _linear(**kw):
    d = dict(nranks=2, rows=4, outputs=48, inputs=256, x_fmt="mx8", x=A, x_stride=256, x_rank_stride=1024,
             x_scales=A, x_scale_stride=8, x_scale_rank_stride=32, w=A, w_stride=128, w_rank_stride=128 * 48,
             w_scales=A, w_scale_stride=8, w_scale_rank_stride=8 * 48, y_fmt="bf16", y=A, y_stride=48,
             y_rank_stride=192)
    d.update(kw)
    return abi.linear_params(**d)


def _adapters(**kw):
    d = dict(adapters=3, rank=16, index=A, scale=A, a=A, a_stride=256, a_adapter_stride=16 * 256,
             a_rank_stride=3 * 16 * 256, b=A, b_stride=16, b_adapter_stride=48 * 16, b_rank_stride=0)
    d.update(kw)
    return abi.adapter_params(**d)


def _run(lin=None, ad=None, work=A, work_bytes=1 << 20):
    lin, ad = lin or _linear(), ad or _adapters()
    import ctypes
    return abi.raw().ar_mx4_linear_adapters(ctypes.byref(lin), ctypes.byref(ad), work, work_bytes, None)


BAD_ADAPTERS = [
    (dict(adapters=-1), -1), (dict(rank=-1), -1), (dict(index=None), -1), (dict(a=None), -1), (dict(b=None), -1),
    (dict(a_stride=248), -1), (dict(b_stride=8), -1), (dict(a_adapter_stride=-8), -1), (dict(b_adapter_stride=-8), -1),
    (dict(a_rank_stride=-8), -1), (dict(b_rank_stride=-8), -1), (dict(a_stride=0), -1), (dict(b_stride=-16), -1),
    (dict(index=A + 2), -2), (dict(scale=A + 1), -2), (dict(a=A + 8), -2), (dict(b=A + 2), -2), (dict(a_stride=260), -2),
    (dict(b_stride=17), -2), (dict(a_adapter_stride=4100), -2), (dict(b_adapter_stride=770), -2),
    (dict(a_rank_stride=12), -2), (dict(b_rank_stride=4), -2),
    (dict(rank=129), -3), (dict(a_stride=1 << 41), -3), (dict(b_stride=1 << 23), -3), (dict(a_adapter_stride=1 << 41), -3),
    (dict(b_adapter_stride=1 << 41), -3), (dict(a_rank_stride=1 << 41), -3), (dict(b_rank_stride=1 << 41), -3),
    (dict(adapters=2 ** 31 - 1, a_adapter_stride=1 << 39), -3), (dict(adapters=2 ** 31 - 1, b_adapter_stride=1 << 39), -3),
]


@pytest.mark.parametrize("kw,want", BAD_ADAPTERS)
def test_adapter_refusals(kw, want):
    assert _run(ad=_adapters(**kw)) == want


def test_adapters_refuse_what_the_layer_refuses():
    for kw, want in ((dict(nranks=0), -1), (dict(x=None), -1), (dict(y=A + 1), -2), (dict(w_stride=136), -2),
                     (dict(y_stride=1 << 41), -3), (dict(rows=1 << 30, outputs=1 << 30, y_stride=1 << 30), -3)):
        assert _run(lin=_linear(**kw)) == want, kw
        # ... also where no adapter counts
        assert _run(lin=_linear(**kw), ad=_adapters(rank=0)) == want, kw
    p = _adapters()
    p.reserved = 1
    assert _run(ad=p) == -1
    raw = abi.raw().ar_mx4_linear_adapters
    assert raw(None, None, A, 1 << 20, None) == -1


def test_adapters_refuse_a_bad_work_buffer():
    need = abi.ar_adapter_work_bytes(_linear(), _adapters())
    assert need > 0
    assert _run(work=None) == -1 and _run(work=A + 16) == -2 and _run(work_bytes=need - 1) == -3
    assert _run(work_bytes=0) == -3
    # nothing to do is no error, whatever else is missing
    assert _run(lin=_linear(rows=0, x=None, y=None), ad=_adapters(index=None), work=None, work_bytes=0) == 0
    assert _run(lin=_linear(outputs=0, w=None, y=None), ad=_adapters(b=None), work=None, work_bytes=0) == 0


def test_adapter_work_bytes():
    def need(ad=None, **kw):
        return abi.ar_adapter_work_bytes(_linear(**kw), ad or _adapters())

    assert need(ad=_adapters(adapters=0)) == 0 and need(ad=_adapters(rank=0)) == 0
    assert need(rows=0) == 0 and need(inputs=0) == 0
    # t of every rank and token at least, 16 dimensions of binary32
    assert need() >= 2 * 4 * 64 and need() % 256 == 0
    shared = _linear(x_rank_stride=0, x_scale_rank_stride=0)
    assert abi.ar_adapter_work_bytes(shared, _adapters(a_rank_stride=0)) < need()
    assert _code(abi.ar_adapter_work_bytes, _linear(nranks=0), _adapters()) == -1
    assert _code(abi.ar_adapter_work_bytes, _linear(), _adapters(rank=200)) == -3


# ------------------------------------------------------------------- cache --

def _cache(**kw):
    d = dict(fmt="bf16", pages=10, page=16, kv_heads=4, dim=64, k=A, v=A, page_stride=16 * 256, token_stride=256,
             head_stride=64, k_scales=None, v_scales=None, scale_page_stride=0, scale_token_stride=0, scale_head_stride=0)
    d.update(kw)
    return abi.cache_params(**d)


R8 = dict(fmt="row8", k_scales=A, v_scales=A, scale_page_stride=64, scale_token_stride=4, scale_head_stride=1)
BAD_CACHE = [
    (dict(fmt="f32"), -1), (dict(fmt="mx8"), -1), (dict(fmt=9), -1), (dict(pages=-1), -1), (dict(page=0), -1),
    (dict(page=8), -1), (dict(page=48), -1), (dict(page=-16), -1), (dict(kv_heads=0), -1), (dict(dim=0), -1),
    (dict(dim=8), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(page_stride=-4096), -1),
    (dict(token_stride=248), -1), (dict(head_stride=56), -1), (dict(token_stride=64), -1), (dict(page_stride=4088), -1),
    (dict(head_stride=0), -1), (dict(R8, k_scales=None), -1), (dict(R8, v_scales=None), -1),
    (dict(R8, scale_token_stride=3), -1), (dict(R8, scale_head_stride=-1), -1),
    (dict(dim=72), -2), (dict(k=A + 8), -2), (dict(v=A + 4), -2), (dict(page_stride=16 * 256 + 4), -2),
    (dict(token_stride=260, page_stride=1 << 14), -2), (dict(R8, token_stride=264, page_stride=1 << 14), -2),
    (dict(R8, k_scales=A + 2), -2), (dict(R8, v_scales=A + 1), -2),
    (dict(dim=272), -3), (dict(page=1 << 21), -3), (dict(pages=1 << 31), -3), (dict(page_stride=1 << 30), -3),
    (dict(token_stride=1 << 26), -3), (dict(head_stride=1 << 30), -3), (dict(R8, scale_page_stride=1 << 30), -3),
]


def _append(cache=None, sequences=2, queries=3, fmt="bf16", k=A, k_stride=256, k_head_stride=64, v=A, v_stride=256,
            v_head_stride=64, lengths=A, pages=A, pages_stride=5, max_pages=5):
    return _code(abi.ar_cache_append, cache or _cache(), sequences, queries, fmt, k, k_stride, k_head_stride, v,
                 v_stride, v_head_stride, lengths, pages, pages_stride, max_pages, stream=0)


def _attend(cache=None, work=A, work_bytes=1 << 30, **kw):
    d = dict(sequences=2, queries=3, heads=8, scale=0.1, fmt="bf16", q=A, q_stride=512, q_head_stride=64, out=A,
             out_stride=512, out_head_stride=64, lse=A, lse_stride=8, prefix=100, prefix_pages=A, lengths=A, pages=A,
             pages_stride=5, max_pages=5)
    d.update(kw)
    import ctypes
    p = abi.attention_params(cache or _cache(), **d)
    return abi.raw().ar_prefix_attention(ctypes.byref(p), work, work_bytes, None)


@pytest.mark.parametrize("kw,want", BAD_CACHE)
def test_cache_refusals(kw, want):
    assert _append(_cache(**kw)) == want
    assert _attend(_cache(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(sequences=-1), -1), (dict(queries=-1), -1), (dict(max_pages=-1), -1), (dict(fmt="f32"), -1), (dict(fmt="row8"), -1),
    (dict(fmt="f16"), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(lengths=None), -1), (dict(pages=None), -1),
    (dict(pages_stride=4), -1), (dict(k_stride=-8), -1), (dict(v_head_stride=-8), -1),
    (dict(k=A + 8), -2), (dict(v=A + 2), -2), (dict(k_stride=260), -2), (dict(v_stride=4), -2), (dict(k_head_stride=60), -2),
    (dict(v_head_stride=4), -2), (dict(lengths=A + 2), -2), (dict(pages=A + 1), -2),
    (dict(sequences=1 << 30), -3), (dict(sequences=1 << 20, queries=1 << 12), -3), (dict(max_pages=1 << 30, pages_stride=1 << 30), -3),
    (dict(k_stride=1 << 30), -3), (dict(v_head_stride=1 << 30), -3), (dict(pages_stride=1 << 30), -3)])
def test_append_refusals(kw, want):
    assert _append(**kw) == want


def test_append_of_nothing():
    for kw in (dict(sequences=0), dict(queries=0), dict(max_pages=0, pages=None), dict(cache=_cache(pages=0, k=None))):
        assert _append(**dict(dict(k=None), **kw)) == 0
    import ctypes
    assert abi.raw().ar_cache_append(None, bytes(96), None) == -1
    assert abi.raw().ar_cache_append(ctypes.byref(_cache()), None, None) == -1


@pytest.mark.parametrize("kw,want", [
    (dict(sequences=-1), -1), (dict(queries=0), -1), (dict(heads=0), -1), (dict(heads=6), -1), (dict(prefix=-1), -1),
    (dict(max_pages=-1), -1), (dict(fmt="f32"), -1), (dict(fmt="f16"), -1), (dict(scale=0.0), -1), (dict(scale=-1.0), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(q=None), -1), (dict(out=None), -1),
    (dict(lengths=None), -1), (dict(pages=None), -1), (dict(prefix_pages=None), -1), (dict(pages_stride=4), -1),
    (dict(q_stride=-8), -1), (dict(out_head_stride=56), -1), (dict(out_stride=504), -1), (dict(lse_stride=7), -1),
    (dict(work=None), -1),
    (dict(q=A + 8), -2), (dict(out=A + 8), -2), (dict(q_stride=516), -2), (dict(q_head_stride=68), -2),
    (dict(out_stride=516), -2), (dict(out_head_stride=68, out_stride=1024), -2), (dict(lse=A + 2), -2), (dict(lengths=A + 1), -2),
    (dict(pages=A + 2), -2), (dict(prefix_pages=A + 2), -2), (dict(work=A + 64), -2),
    (dict(sequences=(1 << 30) + 1), -3), (dict(prefix=(1 << 30) + 1), -3), (dict(max_pages=1 << 27, pages_stride=1 << 27), -3),
    (dict(sequences=1 << 23), -3), (dict(q_stride=1 << 36), -3), (dict(out_stride=1 << 36), -3), (dict(lse_stride=1 << 36), -3),
    (dict(pages_stride=1 << 30), -3), (dict(work_bytes=100), -3)])
def test_attention_refusals(kw, want):
    assert _attend(**kw) == want


def test_attention_scale_is_finite_in_units_of_log2():
    assert _attend(scale=2.0 ** 127, sequences=0) == 0
    assert _attend(scale=2.4e38, sequences=0) == -1


def test_attention_refuses_null_and_reserved():
    raw = abi.raw()
    assert raw.ar_prefix_attention(None, A, 1 << 30, None) == -1
    assert raw.ar_prefix_attention_work_bytes(None) == -1
    assert _attend(sequences=0, q=None, out=None, lengths=None, work=None, work_bytes=0) == 0


def test_attention_work_bytes():
    def need(**kw):
        d = dict(sequences=2, queries=3, heads=8, scale=0.1, fmt="bf16", q=A, q_stride=512, q_head_stride=64, out=A,
                 out_stride=512, out_head_stride=64, lse=None, lse_stride=0, prefix=100, prefix_pages=A, lengths=A, pages=A,
                 pages_stride=5, max_pages=5)
        d.update(kw)
        return abi.ar_prefix_attention_work_bytes(abi.attention_params(_cache(), **d))

    row = 2 * 3 * 8 * (64 + 2) * 4
    assert need() >= 2 * row and need() % 256 == 0         # a part of the prefix, and one of the own tokens
    assert need(prefix=0) >= row and need(max_pages=0) >= row and need(prefix=0, max_pages=0) == 0
    assert need(sequences=0) == 0
    assert _code(need, queries=0) == -1 and _code(need, sequences=1 << 24) == -3
    # the pieces fill the chip and no more: parts are bounded whatever the lengths
    assert need(prefix=1 << 30, max_pages=1 << 20) < 2048 * row


# ----------------------------------------------------------------- binding --

def test_tensors_not_on_the_gpu_are_refused():
    t = torch.zeros(64, dtype=torch.bfloat16)
    for make in (lambda: _adapters(index=t), lambda: _adapters(scale=t), lambda: _adapters(a=t), lambda: _adapters(b=t),
                 lambda: _cache(k=t), lambda: _cache(v=t), lambda: _cache(**dict(R8, k_scales=t)), lambda: _attend(q=t),
                 lambda: _attend(lse=t), lambda: _attend(prefix_pages=t), lambda: _attend(pages=t)):
        with pytest.raises(abi.ArError) as e:
            make()
        assert e.value.code == abi.AR_EINVAL
    assert _append(k=t) == -1 and _append(pages=t) == -1
    with pytest.raises(abi.ArError):
        abi.ar_mx4_linear_adapters(_linear(), _adapters(), t, stream=0)
    with pytest.raises(abi.ArError):
        buffers.PagedCache(2, 16, 1, 16, "bf16", device="cpu")
    with pytest.raises(ValueError):
        buffers.PagedCache(2, 16, 1, 16, "mx8", device="cpu")


class Held:
    """What the binding asks of a tensor, on a device of its own."""
    device = "cuda:0"

    def get_device(self):
        return 0

    def data_ptr(self):
        return A


def test_parameters_keep_their_tensors(monkeypatch):
    """The memory behind the addresses lives as long as the parameters, the
    cache's as long as those of a call on it."""
    monkeypatch.setattr(abi, "_current_device", lambda: 0)
    t = [Held() for _ in range(14)]
    refs = [weakref.ref(x) for x in t]
    ad = _adapters(index=t[0], scale=t[1], a=t[2], b=t[3])
    cache = _cache(**dict(R8, k=t[4], v=t[5], k_scales=t[6], v_scales=t[7]))
    att = abi.attention_params(cache, 2, 1, 8, 0.1, "bf16", t[8], 512, 64, t[9], 512, 64, t[10], 8, 16, t[11], t[12], t[13], 5, 5)
    del t, cache
    gc.collect()
    assert all(r() is not None for r in refs)
    del ad, att
    gc.collect()
    assert all(r() is None for r in refs)


# ------------------------------------------------ the 64-bit forms' own pins --

def test_attention_form_by_hand():
    """One head, two keys: weights 1/4 and 3/4 at a score difference of log 3."""
    k = np.zeros((2, 16, 1, 1))
    v = np.zeros_like(k)
    k[1, 0, 0, 0], k[0, 0, 0, 0] = 0.0, np.log(3.0)
    v[1, 0, 0, 0], v[0, 0, 0, 0] = 8.0, 4.0
    out, lse, size, top, mass = oc.attention(np.ones((1, 1, 1)), k, v, 1.0, 1, np.array([1]), [1], np.array([[0]]), 1)
    assert np.isclose(out[0, 0, 0], 5.0) and np.isclose(lse[0, 0], np.log(4.0))
    # nothing seen, and a sequence that is not there
    out, lse, *_ = oc.attention(np.ones((2, 1, 1)), k, v, 1.0, 0, np.array([]), [0, -1], np.array([[0], [0]]), 1)
    assert out[0, 0, 0] == 0 and lse[0, 0] == -np.inf and np.isnan(out[1, 0, 0])


def test_places_by_hand():
    pages = np.array([[5, 7], [3, -1], [2, 9]])
    assert oc.places([18, 17, -2], 2, pages, 16, 9) == [(0, 7, 0), (1, 7, 1), (2, 3, 15)]
    assert oc.places([1, 40, 0], 3, pages, 16, 9) == [(2, 5, 0)]
    p, s, t = oc.tokens(np.array([4, -1, 6]), 40, 16, 9)
    assert p.tolist() == [4] * 16 + [6] * 8 and s.tolist() == list(range(16)) + list(range(8)) and t[16] == 32
