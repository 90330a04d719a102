"""The norm's row factor is the real one rounded to fp32 once (GPU)."""
import pytest
import torch

import grouped_gemm_persistent_gb300 as tg
from test_residual_norm import BF, F, HF, lib  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]


def rows_of(kind, M, K, g):
    x = torch.randn(M, K, generator=g, device="cuda")
    if kind == "columns":                          # of unequal size, a few much larger
        size = torch.exp(0.5 * torch.randn(K, generator=g, device="cuda"))
        size[torch.rand(K, generator=g, device="cuda") < 0.01] *= 20.0
        x *= size
    elif kind == "dominant":                       # one that is nearly all of a row
        x[:, K // 3] *= 300.0
    return x


@pytest.mark.parametrize("K", [1, 2, 8, 100, 128, 384, 1001, 1544, 4096, 8192, 16384, 16400, 32768])
@pytest.mark.parametrize("kind", ["normal", "columns", "dominant"])
@pytest.mark.parametrize("dt,rt", [(BF, None), (HF, None), (F, None), (BF, BF), (BF, F)])
def test_rows_rounded_once(K, kind, dt, rt):
    """A thread adds 32 squares a sum at most, from a number of twice the largest: an addition leaves out up to 2^-24 of 3 times the sum,
    so what is left out is 96 * 2^-24 of it at most, and adding that up is off by 2^-24 of this each time: 32 * 96 * 2^-48 of the
    sum.  Lanes and warps add 10 times two roundings of it: together less than 2^-35.6, the factor by half of that.  It falls on the
    other side of a border between two fp32 numbers (at least 2^-24 of it apart) in fewer than 2 * 2^-36.6 * 2^24 < 2^-11 of the rows."""
    M = max(64, min(20000, 4_000_000 // K))
    g = torch.Generator(device="cuda").manual_seed(K)
    x = rows_of(kind, M, K, g).to(dt)
    residual = None if rt is None else rows_of(kind, M, K, g).to(rt)
    eps = 1e-6
    n = tg.rmsnorm(x, None, eps, residual=residual)
    h = n.hidden.double()
    want = (1.0 / (h.square().mean(1) + float(torch.tensor(eps, dtype=F).double())).sqrt()).float()
    other = n.row_scale != want
    assert int(other.sum()) <= 1 + M * 2.0 ** -11
    assert bool(((n.row_scale.view(torch.int32) - want.view(torch.int32)).abs() <= 1).all())
