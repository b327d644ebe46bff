"""The binding of the layer operators, without a GPU."""
import gc
import os
import subprocess
import sys
import weakref

import pytest

from collective_synchronization_amd import abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Held:
    """What the binding asks of a tensor, on a device of its own."""
    device = "cuda:0"

    def get_device(self):
        return 0

    def data_ptr(self):
        return 1 << 20


@pytest.fixture
def device(monkeypatch):
    monkeypatch.setattr(abi, "_current_device", lambda: 0)


def _norm(*t):
    gamma, residual, residual_out, y, scales = t
    return abi.norm_params(2, 64, 1e-5, "bf16", gamma, "bf16", residual, 64, residual_out, 64, "mx8", y, 64,
                           scales, 4)


def _linear(*t):
    x, xs, w, ws, y = t
    return abi.linear_params(1, 2, 48, 64, "mx8", x, 64, 0, xs, 4, 0, w, 32, 0, ws, 4, 0, "bf16", y, 48, 0)


@pytest.mark.parametrize("make", (_norm, _linear))
def test_parameters_keep_their_tensors(make, device):
    """The memory behind the addresses lives as long as the parameters."""
    tensors = [Held() for _ in range(5)]
    refs = [weakref.ref(t) for t in tensors]
    p = make(*tensors)
    del tensors
    gc.collect()
    assert all(r() is not None for r in refs)
    del p
    gc.collect()
    assert all(r() is None for r in refs)


def test_import_without_gpu_names_in_torch():
    """A torch built for the CPU alone: the module is there, a tensor that is
    not on a GPU is refused as always."""
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    delattr(torch._C, name)
from collective_synchronization_amd import abi
assert abi.ar_slot_bytes("ll", 8) > 0
try:
    abi.norm_params(1, 8, 0.0, "f32", None, "f32", None, 0, None, 0, "f32", torch.zeros(1, 8), 8)
except abi.ArError as e:
    assert e.code == abi.AR_EINVAL
else:
    raise SystemExit("not refused")
"""
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True, timeout=120)
