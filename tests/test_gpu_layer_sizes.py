"""Layer operators on more rows or outputs than one launch has threads for
(2^32): they go out in several launches, and every row is its own."""
import numpy as np
import pytest
import torch

from collective_synchronization_amd import abi

pytestmark = pytest.mark.gpu

GIB = 1 << 30


def _need(gib):
    if torch.cuda.mem_get_info()[0] < (gib + 4) * GIB:
        pytest.skip(f"needs {gib} GiB of device memory")


def _bf16_rows(rows):
    """[rows, 8] bf16 whose row r is r mod 251 of a table, and the table."""
    table = torch.randn((251, 8), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    x = torch.empty((rows, 8), dtype=torch.bfloat16, device="cuda")
    whole = rows // 251 * 251
    x[:whole] = table.to("cuda").repeat(whole // 251, 1)
    x[whole:] = table[:rows - whole].to("cuda")
    return x, table


def _same_as_table(y, want):
    """Row r of y is row r mod 251 of want, bit for bit."""
    rows = y.shape[0]
    whole = rows // 251 * 251
    w = want.to("cuda")
    assert bool((y[:whole].view(-1, 251, 8) == w).all())
    assert bool((y[whole:] == w[:rows - whole]).all())


def _norm_of_table(table):
    """The kernel's own norm of the few rows."""
    t = table.to("cuda")
    y = torch.empty_like(t)
    p = abi.norm_params(251, 8, 1e-5, "bf16", None, "bf16", None, 0, None, 0, "bf16", y, 8)
    abi.ar_residual_norm(p, t, 8)
    torch.cuda.synchronize()
    h = table.double().numpy()
    v = h / np.sqrt((h * h).mean(-1, keepdims=True) + 1e-5)
    assert (np.abs(y.double().cpu().numpy() - v) <= np.abs(v) * 2.0 ** -7).all()
    return y


def test_norm_of_more_rows_than_a_launch():
    """64 threads a row, 2^26 + 300 rows, in place."""
    _need(1)
    x, table = _bf16_rows((1 << 26) + 300)
    want = _norm_of_table(table)
    p = abi.norm_params(x.shape[0], 8, 1e-5, "bf16", None, "bf16", None, 0, None, 0, "bf16", x, 8)
    abi.ar_residual_norm(p, x, 8)
    torch.cuda.synchronize()
    _same_as_table(x, want)


@pytest.mark.parametrize("ranks,m,n", ((2, 1, 1 << 30), (1, (1 << 27) + 40, 16)))
def test_linear_of_more_outputs_than_a_launch(ranks, m, n):
    """Many outputs of one token on shared weights, and many tokens of few
    outputs: tables of 256 weight rows and of 251 tokens, over and over."""
    _need(30)
    k = 32
    rng = np.random.default_rng(4)
    codes = torch.from_numpy(rng.integers(0, 256, (256, 16), dtype=np.uint8))
    lut = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
    c = codes.numpy()
    wv = np.stack((lut[c & 15], lut[c >> 4]), -1).reshape(256, 32)
    w = codes.to("cuda").repeat(max(1, n // 256), 1)[:n].contiguous()
    ws = torch.full((n, 4), 127, dtype=torch.uint8, device="cuda")
    table = torch.from_numpy(rng.integers(-4, 5, (251, 32)) / 2.0).to(torch.bfloat16)
    x = table.to("cuda").repeat(-(-m // 251), 1)[:m].contiguous()
    xv = table.double().numpy()
    y = torch.empty((ranks, m, n), dtype=torch.bfloat16, device="cuda")
    p = abi.linear_params(ranks, m, n, k, "bf16", x, k, 0, None, 0, 0, w, 16, 0, ws, 4, 0, "bf16", y, n, m * n)
    abi.ar_mx4_linear(p)
    torch.cuda.synchronize()
    want = torch.from_numpy(xv @ wv.T).to(torch.bfloat16).to("cuda")        # [251, 256], exact sums
    for r in range(ranks):
        if m == 1:
            assert bool((y[r].view(-1, 256) == want[0]).all())
        else:
            whole = m // 251 * 251
            assert bool((y[r, :whole].view(-1, 251, n) == want[:, :n]).all())
            assert bool((y[r, whole:] == want[:m - whole, :n]).all())
