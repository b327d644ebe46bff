"""Refusals of the layer operators, on the host: every bad argument comes back
as its status before anything is enqueued (no GPU is touched; the addresses
are made up).  And the 64-bit forms' own tables, against torch's types."""
import ctypes

import numpy as np
import pytest
import torch

from collective_synchronization_amd import abi
from oracle import layer

A = 1 << 20            # an address aligned to everything


def _code(fn, *args):
    try:
        fn(*args, stream=0)
    except abi.ArError as e:
        return e.code
    return 0


def _norm(**kw):
    d = dict(rows=2, hidden=64, eps=1e-5, fmt="bf16", gamma=A, res_fmt="bf16", residual=A,
             residual_stride=64, residual_out=A, residual_out_stride=64, y_fmt="bf16", y=A,
             y_stride=64, scales=None, scale_stride=0)
    d.update(kw)
    return abi.norm_params(**d)


BAD_NORM = [
    (dict(rows=-1), -1), (dict(hidden=-1), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
    (dict(eps=float("inf")), -1), (dict(fmt="mx8"), -1), (dict(fmt=-1), -1), (dict(fmt=6), -1),
    (dict(res_fmt="f16"), -1), (dict(res_fmt="row8"), -1), (dict(y_fmt="f32"), -1), (dict(y_fmt=9), -1),
    (dict(y=None), -1), (dict(y_stride=56), -1), (dict(y_stride=0), -1), (dict(y_stride=-64), -1),
    (dict(residual_stride=8), -1), (dict(residual_out_stride=8), -1),
    (dict(y_fmt="mx8"), -1), (dict(y_fmt="mx8", scales=A, scale_stride=1), -1),
    (dict(y_fmt="row8"), -1), (dict(y_fmt="mx4", scales=A, scale_stride=4, y_stride=16), -1),
    (dict(gamma=A + 8), -2), (dict(y=A + 8), -2), (dict(residual=A + 2), -2), (dict(residual_out=A + 4), -2),
    (dict(y_stride=68), -2), (dict(residual_stride=65), -2),
    (dict(y_fmt="mx8", scales=A, scale_stride=6), -2), (dict(y_fmt="mx8", scales=A + 2, scale_stride=4), -2),
    (dict(y_fmt="row8", scales=A + 2), -2), (dict(y_fmt="row8", scales=A, y_stride=72), -2),
    (dict(hidden=32769, y_stride=1 << 17, residual_stride=1 << 17, residual_out_stride=1 << 17), -3),
    (dict(rows=1 << 31), -3), (dict(y_stride=1 << 41), -3),
]


@pytest.mark.parametrize("kw,want", BAD_NORM)
def test_residual_norm_refusals(kw, want):
    assert _code(abi.ar_residual_norm, _norm(**kw), A, 64) == want


def test_residual_norm_refuses_its_input():
    assert _code(abi.ar_residual_norm, _norm(), None, 64) == -1
    assert _code(abi.ar_residual_norm, _norm(), A, 56) == -1
    assert _code(abi.ar_residual_norm, _norm(), A + 8, 64) == -2
    assert _code(abi.ar_residual_norm, _norm(), A, 66) == -2
    p = _norm()
    p.reserved = 1
    assert _code(abi.ar_residual_norm, p, A, 64) == -1
    assert abi.raw().ar_residual_norm(None, A, 64, None) == -1
    # nothing to do is no error, whatever else is missing
    assert _code(abi.ar_residual_norm, _norm(rows=0, y=None), None, 0) == 0
    assert _code(abi.ar_residual_norm, _norm(hidden=0, y=None), None, 0) == 0


def _reduce(desc=None, params=None, scratch=A, epoch=None, ctrl=A, timeout=0, flags=0):
    d = desc or abi.make_desc(4, 128, "ll")
    try:
        abi.ar_reduce_norm(d, scratch, params or _norm(), epoch or abi.ar_epoch_init(), ctrl, timeout,
                           flags, stream=0)
    except abi.ArError as e:
        return e.code
    return 0


def test_reduce_norm_refusals():
    for kw, want in BAD_NORM:
        if kw.get("rows", 0) < 0 or kw.get("hidden", 0) < 0 or "rows" not in kw and "hidden" not in kw:
            assert _reduce(params=_norm(**kw)) == want, kw
    assert _reduce(desc=abi.make_desc(4, 120, "ll")) == -1            # not rows * hidden
    assert _reduce(desc=abi.make_desc(17, 128, "ll")) == -1
    assert _reduce(desc=abi.make_desc(4, 128, "ll", 4, "twoshot")) == -1
    assert _reduce(desc=abi.make_desc(4, 128, "ll", 4, "allgather")) == -1
    assert _reduce(desc=abi.make_desc(4, 128, "ll"), params=_norm(fmt="f32", res_fmt="f32", y_fmt="f32")) == -1
    assert _reduce(params=_norm(hidden=60), desc=abi.make_desc(4, 120, "ll")) == -2
    assert _reduce(scratch=None) == -1 and _reduce(ctrl=None) == -1
    assert _reduce(scratch=A + 16) == -2 and _reduce(ctrl=A + 16) == -2
    assert _reduce(epoch=abi.ar_epoch(0, 0)) == -1 and _reduce(epoch=abi.ar_epoch(1, 2)) == -1
    assert _reduce(timeout=abi.AR_MAX_TIMEOUT_NS + 1) == -1 and _reduce(flags=2) == -1
    h = abi.AR_REDUCE_NORM_MAX_HIDDEN + 8
    big = _norm(rows=1, hidden=h, y_stride=h, residual_stride=h, residual_out_stride=h)
    assert _reduce(params=big, desc=abi.make_desc(2, h, "ll")) == -3
    assert _reduce(params=_norm(rows=0), desc=abi.make_desc(4, 0, "ll"), scratch=None, ctrl=None) == 0
    assert abi.raw().ar_reduce_norm(None, A, None, abi.ar_epoch_init(), A, 0, 0, None) == -1
    d = abi.make_desc(4, 128, "ll")
    assert abi.raw().ar_reduce_norm(ctypes.byref(d), A, None, abi.ar_epoch_init(), A, 0, 0, None) == -1


@pytest.mark.parametrize("back", (False, True))
def test_mx_refusals(back):
    def go(rows=2, cols=64, f="bf16", p=A, stride=64, q="mx8", codes=A, codes_stride=64, scales=A,
           scale_stride=4):
        if back:
            return _code(abi.ar_dequantize_mx, rows, cols, q, codes, codes_stride, scales, scale_stride, f, p,
                         stride)
        return _code(abi.ar_quantize_mx, rows, cols, f, p, stride, q, codes, codes_stride, scales, scale_stride)

    for kw in (dict(rows=-1), dict(cols=-1), dict(f="mx8"), dict(q="row8"), dict(q="bf16"), dict(p=None),
               dict(codes=None), dict(scales=None), dict(stride=56), dict(codes_stride=48),
               dict(scale_stride=1), dict(codes_stride=-64), dict(cols=65), dict(q=7)):
        assert go(**kw) == -1, kw
    for kw in (dict(p=A + 8), dict(codes=A + 4), dict(scales=A + 1), dict(stride=68), dict(codes_stride=72),
               dict(scale_stride=7)):
        assert go(**kw) == -2, kw
    for kw in (dict(rows=1 << 31), dict(rows=1 << 29), dict(stride=1 << 41)):
        assert go(**kw) == -3, kw
    assert go(rows=0, p=None, codes=None) == 0 and go(cols=0, p=None, scales=None) == 0


def _linear(**kw):
    d = dict(nranks=2, rows=4, outputs=48, inputs=256, x_fmt="mx8", x=A, x_stride=256, x_rank_stride=1024,
             x_scales=A, x_scale_stride=8, x_scale_rank_stride=32, w=A, w_stride=128, w_rank_stride=128 * 48,
             w_scales=A, w_scale_stride=8, w_scale_rank_stride=8 * 48, y_fmt="bf16", y=A, y_stride=48,
             y_rank_stride=192)
    d.update(kw)
    return abi.linear_params(**d)


BAD_LINEAR = [
    (dict(nranks=0), -1), (dict(nranks=17), -1), (dict(rows=-1), -1), (dict(outputs=-1), -1),
    (dict(inputs=-1), -1), (dict(x_fmt="f16"), -1), (dict(x_fmt="f32"), -1), (dict(x_fmt=6), -1),
    (dict(y_fmt="f16"), -1), (dict(y_fmt="mx8"), -1), (dict(x=None), -1), (dict(w=None), -1),
    (dict(w_scales=None), -1), (dict(x_scales=None), -1), (dict(y=None), -1), (dict(y_stride=47), -1),
    (dict(x_stride=240), -1), (dict(w_stride=112), -1), (dict(x_scale_stride=4), -1),
    (dict(w_scale_stride=4), -1), (dict(x_rank_stride=-16), -1), (dict(w_rank_stride=-16), -1),
    (dict(y_rank_stride=-1), -1), (dict(x_scale_rank_stride=-4), -1), (dict(w_scale_rank_stride=-4), -1),
    (dict(x_fmt="bf16", x_stride=248), -1), (dict(inputs=257), -1),
    (dict(x=A + 8), -2), (dict(w=A + 8), -2), (dict(y=A + 1), -2), (dict(y_fmt="f32", y=A + 2), -2),
    (dict(x_scales=A + 2), -2), (dict(w_scales=A + 1), -2), (dict(x_stride=264), -2), (dict(w_stride=136), -2),
    (dict(x_scale_stride=10), -2), (dict(w_scale_stride=9), -2), (dict(x_rank_stride=1032), -2),
    (dict(w_rank_stride=8), -2), (dict(w_scale_rank_stride=386), -2), (dict(x_scale_rank_stride=34), -2),
    (dict(x_fmt="bf16", x_rank_stride=1028), -2),
    (dict(rows=(1 << 30) + 1), -3), (dict(outputs=(1 << 30) + 1), -3), (dict(y_stride=1 << 41), -3),
    (dict(x_rank_stride=1 << 41), -3), (dict(rows=1 << 30, outputs=1 << 30, y_stride=1 << 30), -3),
]


@pytest.mark.parametrize("kw,want", BAD_LINEAR)
def test_linear_refusals(kw, want):
    assert _code(abi.ar_mx4_linear, _linear(**kw)) == want


def test_linear_refuses_null_and_reserved():
    assert abi.raw().ar_mx4_linear(None, None) == -1
    p = _linear()
    p.reserved = 2
    assert _code(abi.ar_mx4_linear, p) == -1
    assert _code(abi.ar_mx4_linear, _linear(rows=0, x=None, y=None)) == 0
    assert _code(abi.ar_mx4_linear, _linear(outputs=0, w=None, y=None)) == 0


def test_tensors_not_on_the_gpu_are_refused():
    """Their addresses would fault it."""
    t = torch.zeros((2, 64), dtype=torch.bfloat16)
    for make in (lambda: _norm(y=t), lambda: _norm(gamma=t), lambda: _norm(residual=t),
                 lambda: _norm(residual_out=t), lambda: _norm(scales=t), lambda: _linear(x=t),
                 lambda: _linear(w_scales=t), lambda: _linear(y=t),
                 lambda: abi.ar_residual_norm(_norm(), t, 64, stream=0),
                 lambda: abi.ar_quantize_mx(2, 64, "bf16", t, 64, "mx8", A, 64, A, 4, stream=0),
                 lambda: abi.ar_dequantize_mx(2, 64, "mx8", A, 64, A, 4, "bf16", t, 64, stream=0),
                 lambda: abi.ar_reduce_norm(abi.make_desc(4, 128, "ll"), t, _norm(), abi.ar_epoch_init(), A,
                                            stream=0)):
        with pytest.raises(abi.ArError) as e:
            make()
        assert e.value.code == abi.AR_EINVAL


# ------------------------------------------------ the 64-bit forms' tables --

def test_e4m3_table_is_torch_s():
    codes = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(codes.view(torch.float8_e4m3fn).double().numpy(), layer.E4M3)


def test_e4m3_rounding_is_torch_s():
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.standard_normal(20000) * 50, layer.E4M3, (layer.E4M3[1:] + layer.E4M3[:-1]) / 2])
    v = np.clip(np.concatenate([v, -v]), -448, 448).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(layer.signed_codes(v, layer.E4M3, 128), want)


def test_scale_codes_and_round_trip():
    assert layer.scale_codes([0.0, 1.0, 1.999, 2.0, 2.0 ** -200, np.inf, 448.0], "mx8").tolist() == \
        [0, 119, 119, 120, 0, 255, 127]
    assert layer.scale_codes([6.0, 4.0, 3.9], "mx4").tolist() == [127, 127, 126]
    for fmt in ("mx8", "mx4"):
        rng = np.random.default_rng(1)
        v = rng.standard_normal((3, 70))
        c, s = layer.quantize(v, fmt)
        d = layer.dequantize(c, s, fmt, 70)
        # in units of the scale a block's top is below 512 (8) and values saturate at 448 (6): off by
        # (512 - 448) / 512 = 2^-3 or (8 - 6) / 8 = 2^-2 of the top; half a step of the top binade is
        # 16 / 256 or 1 / 4 of it
        step = {"mx8": 2.0 ** -3, "mx4": 2.0 ** -2}[fmt]
        top = np.repeat(np.abs(layer.blocks_of(v)).max(-1), 32, axis=1)[:, :70]
        assert (np.abs(d - v) <= top * step).all()
        c2, s2 = layer.quantize(d, fmt)
        assert np.array_equal(layer.dequantize(c2, s2, fmt, 70), d)
    p = np.arange(16, dtype=np.uint8)[None]
    assert np.array_equal(layer.unpack4(layer.pack4(p)), p)
