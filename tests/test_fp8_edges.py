"""Edges of the 8-bit calls: products over an empty K."""
import pytest
import torch

import fp8_reference as ref
import grouped_gemm_persistent_gb300 as tg

E4 = torch.float8_e4m3fn


def empty_k(device, rows, G, N):
    a, sa = torch.zeros(rows, 0, device=device).to(E4), torch.zeros(rows, 0, device=device)
    b, sb = torch.zeros(G, 0, N, device=device).to(E4), torch.zeros(G, 0, ref.blocks(N), device=device)
    return a, sa, b, sb


def test_experts_with_an_empty_k_pass_the_checks():
    """(On the CPU: the first thing wrong with the call is where its tensors are.)"""
    a, sa, b, sb = empty_k("cpu", 5, 2, 32)
    with pytest.raises(ValueError, match="CUDA"):
        tg.moe_gemm_fp8(a, sa, b, sb, torch.tensor([2, 3], dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        tg.gemm_fp8(a, sa, b[0], sb[0])


@pytest.mark.gpu
@pytest.mark.parametrize("tile", ["1x128", "2x256", None])
@pytest.mark.parametrize("epilogue", ["none", "bias", "bias_gelu"])
def test_experts_with_an_empty_k(monkeypatch, tile, epilogue):
    """The empty sum: zeros, the expert's bias, or its GELU."""
    if tile:
        monkeypatch.setenv("TG_TILE", tile)
    counts = [3, 0, 260, 2]
    a, sa, b, sb = empty_k("cuda", sum(counts) + 4, 4, 136)
    bias = torch.randn(4, 136, device="cuda").bfloat16() if epilogue != "none" else None
    out = torch.full((sum(counts) + 4, 136), -5.0, device="cuda")
    tg.moe_gemm_fp8(a, sa, b, sb, torch.tensor(counts, dtype=torch.int32, device="cuda"), out, bias=bias,
                    epilogue=epilogue)
    tg.device_status()
    r = 0
    for i, m in enumerate(counts):
        z = torch.zeros(136, device="cuda", dtype=torch.float64) if bias is None else bias[i].double()
        want = ref.gelu(z) if epilogue == "bias_gelu" else z
        # the bias is exact; its GELU is off by e / (1 + e) (8 |u| + 3) + 5 half steps, e = e^-2u: below 16 of z
        assert ((out[r:r + m].double() - want).abs() <= (0 if epilogue != "bias_gelu" else 16 * 2.0 ** -24) * z.abs()).all()
        r += m
    assert (out[r:] == -5.0).all()
