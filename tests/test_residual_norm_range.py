"""The norm over the whole range of its types: squares that pass fp32's range, squares that fall below it, any eps (GPU)."""
import pytest
import torch

import grouped_gemm_persistent_gb300 as tg
from test_residual_norm import BF, E4, F, HF, U, lib  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]


def rows_of(sizes, K, dt, seed=0):
    """A row of +- each size, and one of normal values times it, cut to the type's range."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for s in sizes:
        sign = torch.where(torch.rand(K, generator=g, device="cuda") < 0.5, -1.0, 1.0).double()
        out += [sign * s, torch.randn(K, generator=g, device="cuda").double() * s]
    top = torch.finfo(dt).max
    return torch.stack(out).clamp(-top, top).to(dt)


def check(h, n, gain, eps):
    """row_scale and y of the fp32 rows against 64 bits."""
    x = h.double()
    e = float(torch.tensor(eps, dtype=F).double())
    r = 1.0 / (x.square().mean(1) + e).sqrt()
    # r to 3.1 half steps as elsewhere, or to a step of fp32's subnormal numbers where it is one
    off = 3.1 * U * r + 2.0 ** -149
    assert bool(((n.row_scale.double() - r).abs() <= off).all())
    # y is the fp32 products of that factor: r's own error and two half steps
    g = gain.double()
    want = x * r[:, None] * g
    tol = 2.1 * U * want.abs() + x.abs() * off[:, None] * g.abs() + 2.0 ** -148 * (1 + g.abs())
    assert bool(((n.y.double() - want).abs() <= tol).all())
    q, scale = tg.quantize_fp8(n.y)
    assert torch.equal(n.q.view(torch.uint8), q.view(torch.uint8)) and torch.equal(n.scale, scale)


def norm(x, eps, residual=None):
    g = torch.Generator(device="cuda").manual_seed(9)
    gain = torch.rand(x.shape[1], generator=g, device="cuda") + 0.5
    n = tg.rmsnorm(x, gain, eps, residual=residual, out_dtype=F, fp8_dtype=E4)
    check(n.hidden, n, gain, eps)
    return n


@pytest.mark.parametrize("K", [1, 7, 384, 1001, 8192, 16384, 32768])
@pytest.mark.parametrize("dt", [F, BF])
def test_squares_past_fp32(K, dt):
    x = rows_of((1e15, 1e18, 2e19, 1e20, 1e25, 1e30, 1e36, 3e38), K, dt)
    for eps in (1e-6, 0.0):
        n = norm(x, eps)
        assert bool((n.row_scale > 0).all())
    norm(torch.zeros_like(x), 1e-6, residual=x)
    one = torch.zeros_like(x)
    one[:, K // 2] = x[:, 0]                       # a single value is all of a row
    norm(one, 1e-6)


@pytest.mark.parametrize("K", [1, 384, 1001, 8192, 32768])
@pytest.mark.parametrize("eps", [1e30, 2e33, 2e38, 2.9e38])
def test_an_eps_as_large_as_the_squares(K, eps):
    """Any finite eps counts, beside squares that fp32 holds and beside those that it does not."""
    root = eps ** 0.5
    norm(rows_of((1.0, root * 1e-9, root * 1e-3, root * 0.5, root, root * 1.5, root * 30, 1e25), K, F), eps)


@pytest.mark.parametrize("K", [1, 384, 1001, 8192, 32768])
@pytest.mark.parametrize("dt", [F, BF])
@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-38, 1e-31, 1e-29])
def test_squares_below_fp32(K, dt, eps):
    """Without an eps, or with one of their own size, rows of small numbers have a factor as others have."""
    x = rows_of((1e-12, 1e-15, 1e-17, 1e-19, 1e-20, 1e-22, 3e-23, 1e-25, 1e-30, 1e-35, 1e-37), K, dt)
    if K > 1:                                      # (a single value may happen to be next to nothing)
        norm(x, eps)
        norm(torch.zeros_like(x), eps, residual=x)
    norm(x[::2].contiguous(), eps)


@pytest.mark.parametrize("K", [8, 1001])
def test_factors_past_fp32(K):
    """Without an eps a row below 2^-128 has a factor that fp32 does not hold: infinity, as for a row of zeros."""
    x = torch.full((3, K), 2.0 ** -140, device="cuda")
    x[1] = 0.0
    x[2] = 2.0 ** -127
    n = tg.rmsnorm(x, None, 0.0, out_dtype=F)
    assert bool(n.row_scale[:2].isinf().all()) and float(n.row_scale[2]) == 2.0 ** 127
    assert bool(n.y[0].isinf().all()) and bool(n.y[1].isnan().all()) and bool((n.y[2] == 1.0).all())
