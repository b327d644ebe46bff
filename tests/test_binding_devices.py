"""Parameters made of tensors on one device are refused while another one is
current, whose kernels would read and write that memory (no GPU is touched)."""
import pytest
import torch

from collective_synchronization_amd import abi


class Held:
    """What the binding asks of a tensor, on a device of its own."""

    def __init__(self, device=0):
        self.index = device
        self.device = f"cuda:{device}"

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 1 << 20


class Current:
    def __init__(self, monkeypatch):
        self.index = 0
        monkeypatch.setattr(abi, "_current_device", lambda: self.index)


@pytest.fixture
def current(monkeypatch):
    return Current(monkeypatch)


def _norm():
    t = Held()
    return abi.norm_params(0, 64, 1e-5, "bf16", t, "bf16", t, 64, t, 64, "mx8", t, 64, t, 4)


def _linear():
    t = Held()
    return abi.linear_params(1, 0, 48, 64, "mx8", t, 64, 0, t, 4, 0, t, 32, 0, t, 4, 0, "bf16", t, 48, 0)


def _adapters():
    t = Held()
    return abi.adapter_params(0, 16, t, t, t, 64, 1024, 0, t, 16, 768, 0)


def _cache():
    t = Held()
    return abi.cache_params("bf16", 4, 16, 1, 64, t, t, 1024, 64, 64)


def _attention(cache):
    t = Held(abi._current_device())
    return abi.attention_params(cache, 0, 1, 4, 0.1, "bf16", t, 256, 64, t, 256, 64, None, 0, 16, t, t, t, 4, 4)


def _append(cache):
    t = Held(abi._current_device())
    abi.ar_cache_append(cache, 0, 1, "bf16", t, 64, 64, t, 64, 64, t, t, 4, 4, stream=0)


# nothing in any of these calls (no rows, no sequences): where the device is right, it returns
CALLS = {
    "norm": (_norm, lambda p: abi.ar_residual_norm(p, Held(abi._current_device()), 64, stream=0)),
    "linear": (_linear, lambda p: abi.ar_mx4_linear(p, stream=0)),
    "adapters' layer": (_linear, lambda p: abi.ar_mx4_linear_adapters(p, abi.adapter_params(
        0, 0, None, None, None, 0, 0, 0, None, 0, 0, 0), None, stream=0)),
    "adapters": (_adapters, lambda p: abi.ar_mx4_linear_adapters(abi.linear_params(
        1, 0, 48, 64, "mx8", 1 << 20, 64, 0, 1 << 20, 4, 0, 1 << 20, 32, 0, 1 << 20, 4, 0, "bf16", 1 << 20, 48, 0), p,
        None, stream=0)),
    "append": (_cache, _append),
    "attention": (lambda: _attention(_cache()), lambda p: abi.ar_prefix_attention(p, None, stream=0)),
    "attention's cache": (_cache, _attention),
}


@pytest.mark.parametrize("call", CALLS)
def test_parameters_of_another_device(call, current):
    make, use = CALLS[call]
    p = make()
    use(p)
    current.index = 1
    with pytest.raises(abi.ArError) as e:
        use(p)
    assert e.value.code == abi.AR_EINVAL and "device" in str(e.value)
    current.index = 0
    use(p)


def test_reduce_norm_of_another_device(current):
    p = _norm()
    current.index = 1
    with pytest.raises(abi.ArError) as e:
        abi.ar_reduce_norm(abi.ar_desc(), Held(1), p, 0, Held(1), stream=0)
    assert e.value.code == abi.AR_EINVAL and "device" in str(e.value)


class Buffer(Held):
    """A work buffer, every other element of its memory or all of them."""

    def __init__(self, step):
        super().__init__()
        self.t = torch.empty(4096, dtype=torch.uint8)[::step]
        self.numel, self.element_size, self.is_contiguous = self.t.numel, self.t.element_size, self.t.is_contiguous


def test_a_work_buffer_with_gaps(current):
    """Its bytes would be written one after the other, over what lies in the gaps."""
    calls = (lambda w: abi.ar_prefix_attention(_attention(_cache()), w, stream=0),
             lambda w: abi.ar_mx4_linear_adapters(_linear(), _adapters(), w, stream=0))
    for call in calls:
        call(Buffer(1))
        with pytest.raises(abi.ArError) as e:
            call(Buffer(2))
        assert e.value.code == abi.AR_EINVAL and "contiguous" in str(e.value)


def test_addresses_have_no_device(current):
    p = abi.adapter_params(0, 16, 1 << 20, None, 1 << 20, 64, 1024, 0, 1 << 20, 16, 768, 0)
    current.index = 1
    abi.ar_mx4_linear_adapters(abi.linear_params(
        1, 0, 48, 64, "mx8", 1 << 20, 64, 0, 1 << 20, 4, 0, 1 << 20, 32, 0, 1 << 20, 4, 0, "bf16", 1 << 20, 48, 0), p,
        None, stream=0)
