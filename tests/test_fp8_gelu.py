"""GELU of the 8-bit products with fp32 output: as exact as fp32 holds it, by every way a tile is stored (GPU)."""
import pytest
import torch

import fp8_reference as ref
import grouped_gemm_persistent_gb300 as tg

E4 = torch.float8_e4m3fn
U = 2.0 ** -24      # half a step of fp32

pytestmark = pytest.mark.gpu


def single_terms(M, N, K, G=None):
    """A and B with one k each that is not zero, so that every product is exact, and a bias for each column."""
    g = torch.Generator(device="cuda").manual_seed(31)
    lead = () if G is None else (G,)
    a = torch.zeros(M, K, device="cuda")
    b = torch.zeros(*lead, N, K, device="cuda")
    a[:, 5] = torch.randn(M, generator=g, device="cuda") * 2
    b[..., 5] = torch.randn(*lead, N, generator=g, device="cuda")
    bias = torch.randn(*lead, N, generator=g, device="cuda").bfloat16()
    sa = torch.ones(M, ref.blocks(K), device="cuda")
    sb = torch.ones(*lead, ref.blocks(K), ref.blocks(N), device="cuda")
    return a.to(E4), sa, b.to(E4).transpose(-1, -2), sb, bias


def check(out, a, b, bias):
    """z is one product of two 8-bit values (exact) plus a bias: one rounding, half a step U, times gelu's slope of at
    most 1.13.  With t = z (c0 + c1 z^2) off by at most four half steps (the constants count as one, three operations),
    e^-2u = 2^t is off by 8 |u| of them and the three of the hardware's 2^-22.5; 1 + e by one, its reciprocal by two,
    the product by one: 8 |u| + 7 in all, and 8 |u| + 8 with the second order."""
    z = a.double() @ b.double() + bias.double()
    want = ref.gelu(z)
    u = 0.7978845608028654 * (z + 0.044715 * z ** 3)
    bound = (8 * u.abs() + 8) * U * want.abs() + 1.13 * U * z.abs() + 1e-38
    err = (out.double() - want).abs()
    assert (err <= bound).all(), f"worst {float((err / bound).max()):.3g} of the bound, {float((err / z.abs()).max()):.3g} of z"


@pytest.mark.parametrize("tile", ["1x128", "2x256", None])
@pytest.mark.parametrize("M,N,K", [(1, 520, 1024),        # tiles split over a cluster
                                   (300, 512, 128),       # whole, aligned tiles
                                   (300, 515, 128),       # ragged columns, unaligned rows
                                   (64, 24, 16)])
def test_dense(monkeypatch, tile, M, N, K):
    if tile:
        monkeypatch.setenv("TG_TILE", tile)
    a, sa, b, sb, bias = single_terms(M, N, K)
    out = torch.empty(M, N, device="cuda")                # rows of N elements: not aligned when N is odd
    tg.gemm_fp8(a, sa, b, sb, out, bias=bias, epilogue="bias_gelu")
    tg.device_status()
    check(out, a, b, bias)


def test_dense_column_scales():
    a, sa, b, _, bias = single_terms(300, 512, 128)
    out = tg.gemm_fp8(a, sa, b, torch.ones(1, 512, device="cuda"), bias=bias, epilogue="bias_gelu",
                      out_dtype=torch.float32)
    tg.device_status()
    check(out, a, b, bias)


@pytest.mark.parametrize("tile", ["1x128", "2x256", None])
def test_experts(monkeypatch, tile):
    if tile:
        monkeypatch.setenv("TG_TILE", tile)
    counts = [3, 0, 130, 260]
    a, sa, b, sb, bias = single_terms(sum(counts), 264, 128, len(counts))
    out = tg.moe_gemm_fp8(a, sa, b, sb, torch.tensor(counts, dtype=torch.int32, device="cuda"), bias=bias,
                          epilogue="bias_gelu", out_dtype=torch.float32)
    tg.device_status()
    r = 0
    for i, m in enumerate(counts):
        if m:
            check(out[r:r + m], a[r:r + m], b[i], bias[i])
        r += m


def test_far_values():
    """z far out on both sides, where e^-2u overflows and underflows: z itself and zero."""
    z = torch.tensor([-448.0, -60.0, -20.0, -10.0, -6.0, 6.0, 10.0, 20.0, 60.0, 448.0], device="cuda")
    a = torch.zeros(10, 16, device="cuda")
    a[:, 0] = z
    b = torch.zeros(16, 16, device="cuda")
    b[0] = 1.0
    for scale in (1.0, 2.0 ** 60):
        out = tg.gemm_fp8(a.to(E4), torch.full((10, 1), scale, device="cuda"), b.to(E4), torch.ones(1, 1, device="cuda"),
                          bias=torch.zeros(16, dtype=torch.bfloat16, device="cuda"), epilogue="bias_gelu",
                          out_dtype=torch.float32)
        tg.device_status()
        big = z.abs() * scale >= 20.0                     # gelu is z or below the smallest fp32 there
        want = torch.where(z > 0, z * scale, 0.0)[:, None].expand(10, 16)
        assert torch.equal(out[big], want[big])
        if scale == 1.0:
            check(out, a, b, torch.zeros(16, device="cuda"))
