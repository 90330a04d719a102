"""Infinities in the adapters' products: the same in both forms as in 64 bits, infinities and NaN told apart (GPU)."""
import pytest
import torch

import grouped_gemm_persistent_gb300 as tg
from test_lora import BF, F, HF, check, lib, make  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]


def same_kind(got, want):
    """NaN where NaN is wanted, the same infinities, numbers elsewhere."""
    assert torch.equal(got.isnan(), want.isnan())
    for sign in (1.0, -1.0):
        assert torch.equal(got == sign * float("inf"), want == sign * float("inf"))


@pytest.mark.parametrize("T,K,N,G", [(20, 320, 200, 5), (600, 4096, 200, 5), (5000, 320, 200, 5), (5000, 136, 100, 400)])
@pytest.mark.parametrize("r", [1, 8, 24, 40, 100])
@pytest.mark.parametrize("dt", [BF, HF])
def test_an_infinity_in_x_at_ranks_that_are_filled_up(T, K, N, G, r, dt):
    """The few rows' form has no ranks past r; the tiles fill them up, with nothing that an infinity may meet."""
    base, x, a, b, ids, scale = make(50, T, K, N, r, G, dt, F, "rows")
    ids[3] = 1
    x[3, 7] = float("inf")
    # u = +-inf by the sign of A's column 7; even columns of B go with those signs, so that their sums are infinite
    sign = a[1, :, 7].float().sign()
    b[1, ::2] = (b[1, ::2].float().abs() * sign).to(dt)
    b[1, 2::4] = -b[1, 2::4]
    got = tg.lora_add(base, x, a, b, ids, scale)
    u = float(scale[1]) * (x[3].double() * a[1].double()).sum(1)
    want = base[3].double() + (u * b[1].double()).sum(1)
    assert bool(want[::2].isinf().all())
    same_kind(got[3], want)
    others = torch.arange(T, device="cuda") != 3
    assert bool(got[others].isfinite().all())


@pytest.mark.parametrize("T", [20, 5000])
def test_numbers_past_fp16_beside_an_infinity(T):
    """An adapter with an infinite weight of one rank, whose other ranks give numbers that fp16 does not hold."""
    K, N, r = 256, 72, 16
    base, x, a, b, ids, scale = make(51, T, K, N, r, 3, HF, F, "rows")
    x, a = (x.float() * 100).to(HF), (a.float() * 200 * K ** 0.5).to(HF)
    a[1, 2, 7] = float("inf")
    ids[3] = 1
    got = tg.lora_add(base, x, a, b, ids, scale)
    rows = torch.nonzero(ids == 1)[:, 0]
    u = float(scale[1]) * (x[rows].double()[:, None] * a[1].double()[None]).sum(2)
    assert bool((u.abs() > 65504).any(1).all())
    want = base[rows].double() + (u[:, None] * b[1].double()[None]).sum(2)
    assert bool(want.isinf().all())
    same_kind(got[rows], want)


@pytest.mark.parametrize("T", [20, 5000])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("size,weight", [(3.4e38, 1e-3), (1e37, 1e-2), (1e-36, 100.0), (3e-38, 300.0)])
def test_numbers_at_the_ends_of_fp32_between_the_products(T, dt, size, weight):
    """A factor that takes what is between the two products next to fp32's largest or smallest numbers; the result is well inside."""
    base, x, a, b, ids, _ = make(52, T, 8, 72, 16, 3, dt, F, "rows")
    x = torch.zeros_like(x)
    x[:, 0] = 1.0
    a = torch.where(a < 0, -1.0, 1.0).to(dt)
    b, base = (b.float() * weight).to(dt), torch.zeros_like(base)
    scale = torch.full((3,), size, device="cuda")
    check(base, x, a, b, ids, scale, tg.lora_add(base, x, a, b, ids, scale))


@pytest.mark.parametrize("T", [20, 5000])
@pytest.mark.parametrize("size,weight", [(1e-36, 1e38), (3.4e38, 1e-38), (1e-37, 3e37), (1.5e38, 1e-36)])
def test_opposite_ends_of_fp32_in_one_product(T, size, weight):
    """A number at one end of the range times weights at the other: the products are ordinary, in bf16 alone."""
    base, x, a, b, ids, _ = make(53, T, 8, 72, 16, 3, BF, F, "rows")
    x = torch.zeros_like(x)
    x[:, 0] = 1.0
    a = torch.where(a < 0, -1.0, 1.0).to(BF)
    b = (b.float() * weight).to(BF)
    scale = torch.full((3,), size, device="cuda")
    check(base, x, a, b, ids, scale, tg.lora_add(base, x, a, b, ids, scale))
