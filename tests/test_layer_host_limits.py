"""Limits of the layer operators that are checked on the host (no GPU is
touched; the addresses are made up)."""
import pytest

from collective_synchronization_amd import abi

A = 1 << 20            # an address aligned to everything


def _reduce(nranks, rows, hidden, proto="barrier"):
    p = abi.norm_params(rows, hidden, 1e-5, "bf16", None, "bf16", None, 0, None, 0, "bf16", A, hidden)
    with pytest.raises(abi.ArError) as e:
        abi.ar_reduce_norm(abi.make_desc(nranks, rows * hidden, proto), A, p, abi.ar_epoch_init(), A, stream=0)
    return e.value.code


def test_reduce_norm_of_more_rows_than_a_launch():
    """64 threads a row at least: 2^26 rows are 2^32 threads."""
    assert _reduce(1, 1 << 26, 8) == abi.AR_ESIZE
