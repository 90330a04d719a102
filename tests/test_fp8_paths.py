"""The 8-bit calls on the paths that large calls take: quantiser tiles inside the matrix, pair tiles with every layout
and scale form, several tiles a unit, experts with every type, and whole tiles only, against 64 bits (GPU)."""
import pytest
import torch

import fp8_reference as ref
import grouped_gemm_persistent_gb300 as tg
from test_fp8 import E4, E5, LAYOUTS, check_moe, check_product, check_quantize, cuda_gen, make, make_moe, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [E4, E5])
@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("M,K", [(32, 512), (70, 1024), (33, 1100), (65, 1544)])
def test_quantize_rows_in_whole_tiles(M, K, xt, dtype):
    """32 x 512 tiles inside the matrix, past the first tile column and the first tile row, and ragged ends of both."""
    g = cuda_gen(40)
    x = values(g, M, K, xt)
    check_quantize(x, (1, 128), dtype)
    x[M // 2, K - 1] = float("inf")
    x[M - 1, 600 % K] = float("nan")
    check_quantize(x, (1, 128), dtype)
    # rows of Q that are not 8-byte aligned
    buf = torch.zeros(M, K + 3, dtype=torch.uint8, device="cuda")
    check_quantize(x, (1, 128), dtype, q=buf.view(dtype)[:, 1:K + 1])
    assert not buf[:, 0].any() and not buf[:, K + 1:].any()


@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", [(128, 1), (128, 128)])
def test_quantize_blocks_in_whole_tiles(block, xt):
    check_quantize(values(cuda_gen(41), 260, 520, xt), block, E5)


@pytest.mark.parametrize("a_layout,b_layout", LAYOUTS)
@pytest.mark.parametrize("sb", ["square", "column"])
@pytest.mark.parametrize("M,N,K", [(2560, 2560, 300), (3000, 2200, 700)])
def test_gemm_many_tiles_of_every_layout(M, N, K, a_layout, b_layout, sb):
    """Whole pair tiles, one and more a unit, and a last wave in half tiles."""
    g = cuda_gen(42)
    t = make(g, M, N, K, a_layout, b_layout, at=E5 if sb == "column" else E4, sb=sb)
    for out_dtype in (torch.float32, torch.bfloat16):
        out = tg.gemm_fp8(*t, out_dtype=out_dtype)
        tg.device_status()
        check_product(out, *t)


@pytest.mark.parametrize("tile", ["1x128", "2x256"])
def test_gemm_column_scales_over_three_tiles_a_unit(monkeypatch, tile):
    """The ring of scales goes on from tile to tile; 11 k-blocks end inside a group of four."""
    monkeypatch.setenv("TG_TILE", tile)
    g = cuda_gen(43)
    M, N = (3400, 4200) if tile == "2x256" else (2400, 3300)
    for K in (130, 1300):
        t = make(g, M, N, K, "col", "row", at=E5, sb="column")
        out = tg.gemm_fp8(*t, out_dtype=torch.float32)
        tg.device_status()
        check_product(out, *t)


@pytest.mark.parametrize("epilogue", ["none", "bias", "bias_gelu"])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_gemm_many_tiles_column_scales_epilogues(out_dtype, epilogue):
    g = cuda_gen(44)
    a, sa, b, sb = make(g, 2600, 2312, 260, "col", "row", sb="column")
    sa, sb = sa * 2.0 ** -8, sb * 2.0 ** -8
    bias = torch.randn(2312, generator=g, device="cuda").bfloat16() if epilogue != "none" else None
    out = tg.gemm_fp8(a, sa, b, sb, bias=bias, epilogue=epilogue, out_dtype=out_dtype)
    tg.device_status()
    check_product(out, a, sa, b, sb, bias, epilogue)


@pytest.mark.parametrize("mode", ["0", "1"])
@pytest.mark.parametrize("M,N,K", [(1, 1000, 4096), (40, 512, 2000), (2560, 2560, 256), (3000, 2200, 200)])
@pytest.mark.parametrize("sb", ["square", "column"])
def test_gemm_with_whole_tiles_only(monkeypatch, mode, M, N, K, sb):
    """TG_STREAM_K=0: no tile is split over a cluster and none halved; 1 changes nothing here."""
    g = cuda_gen(45)
    t = make(g, M, N, K, sb=sb)
    bias = torch.randn(N, generator=g, device="cuda").bfloat16()
    usual = tg.gemm_fp8(*t, bias=bias, epilogue="bias", out_dtype=torch.float32)
    monkeypatch.setenv("TG_STREAM_K", mode)
    out = tg.gemm_fp8(*t, bias=bias, epilogue="bias", out_dtype=torch.float32)
    tg.device_status()
    check_product(out, *t, bias, "bias")
    if mode == "1":
        assert torch.equal(out, usual)


def test_single_row_repeats_between_other_calls():
    """Tiles split over a cluster: the same bits whatever ran before, on the same and on other operands."""
    g = cuda_gen(46)
    t, other = make(g, 1, 4096, 4096), make(g, 1, 4096, 4096)
    bias = torch.randn(4096, generator=g, device="cuda").bfloat16()
    first = tg.gemm_fp8(*t, bias=bias, epilogue="bias")
    check_product(first, *t, bias, "bias")
    for i in range(200):
        if i % 3 == 0:
            tg.gemm_fp8(*other, bias=bias, epilogue="bias")
        assert torch.equal(first, tg.gemm_fp8(*t, bias=bias, epilogue="bias"))


@pytest.mark.parametrize("tile", ["1x128", "2x256", None])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("at", [E4, E5])
@pytest.mark.parametrize("b_layout", ["col", "row"])
def test_moe_types(monkeypatch, tile, out_dtype, at, b_layout):
    if tile:
        monkeypatch.setenv("TG_TILE", tile)
    g = cuda_gen(47)
    for counts, N, K in (([3, 0, 130, 1, 256, 0, 129, 300], 200, 272), ([700, 0, 1, 520], 264, 640)):
        a, sa, b, sb, c = make_moe(g, counts, N, K, b_layout=b_layout, at=at)
        sa, sb = sa * 2.0 ** -8, sb * 2.0 ** -8                    # sums that fp16 holds
        bias = torch.randn(len(counts), N, generator=g, device="cuda").bfloat16()
        out = tg.moe_gemm_fp8(a, sa, b, sb, c, bias=bias, epilogue="bias", out_dtype=out_dtype)
        tg.device_status()
        check_moe(out, counts, a, sa, b, sb, bias, "bias")


@pytest.mark.parametrize("out_dtype", [torch.float16, torch.bfloat16])
def test_moe_many_tiles_of_other_types(out_dtype):
    """CTA pairs with several tiles a unit, e5m2 rows and N-contiguous experts."""
    g = cuda_gen(48)
    counts = [1000, 0, 257, 1, 640, 129, 2048, 384]
    a, sa, b, sb, c = make_moe(g, counts, 2312, 300, b_layout="row", at=E5)
    sa, sb = sa * 2.0 ** -8, sb * 2.0 ** -8
    out = tg.moe_gemm_fp8(a, sa, b, sb, c, out_dtype=out_dtype)
    tg.device_status()
    check_moe(out, counts, a, sa, b, sb)


def replay_us(f, n=20):
    f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(n):
            f()
    times = []
    for _ in range(9):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        graph.replay()
        end.record()
        torch.cuda.synchronize()
        times.append(begin.elapsed_time(end) * 1e3 / n)
    return sorted(times)[4]


def test_split_tiles_run_in_one_wave():
    """A tile is not cut into more CTAs than fit beside the other tiles': fewer columns never take much longer than more
    (a second wave costs half as much again)."""
    K, tiles = 4096, (15, 16, 19, 20, 36, 37, 38, 39)
    g = cuda_gen(49)
    us = {}
    for n in tiles:
        a, sa, b, sb = make(g, 1, n * 128, K)
        out = torch.empty(1, n * 128, dtype=torch.bfloat16, device="cuda")
        tg.gemm_fp8(a, sa, b, sb, out)
        check_product(out, a, sa, b, sb)
        us[n] = replay_us(lambda: tg.gemm_fp8(a, sa, b, sb, out))
    for n in tiles[:-1]:
        assert us[n] <= 1.25 * min(us[m] for m in tiles if m > n), us
