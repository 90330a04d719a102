"""8-bit products and their quantiser: refusals (CPU) and parity with 64-bit references (GPU).

Bounds are derived in fp8_reference.product_bound from the number of fp32 operations and half a step of the
output type; the quantiser's bytes and scales must be equal."""
import ctypes

import pytest
import torch

import fp8_reference as ref
import grouped_gemm_persistent_gb300 as tg
from grouped_gemm_persistent_gb300 import _binding
from grouped_gemm_persistent_gb300.build import build

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
PTR = 0x10000       # fake aligned device addresses: never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    build()
    return tg.load()


# ------------------------------------------------------------------------------------------ refusals (CPU)


def operand(**kw):
    d = dict(data=PTR, ld=128, scale=2 * PTR, scale_stride=1, scale_k_stride=1, dtype=tg.E4M3, layout=0, block=1)
    d.update(kw)
    return _binding.Fp8Operand(**d)


def call_gemm(lib, A=None, B=None, C=3 * PTR, cd=0, ldc=128, M=64, N=64, K=128, epi=0, bias=None):
    A = operand() if A is None else A
    B = operand(layout=1) if B is None else B
    return lib.tg_gemm_scaled(ctypes.byref(A), ctypes.byref(B), C, cd, ldc, M, N, K, epi, bias, None)


def call_moe(lib, A=None, B=None, C=3 * PTR, cd=0, ldc=128, T=64, N=64, K=128, G=2, es=64 * 128, ss=1, counts=4 * PTR,
             epi=0, bias=None):
    A = operand() if A is None else A
    B = operand(layout=1, block=128) if B is None else B
    return lib.tg_moe_gemm_scaled(ctypes.byref(A), T, K, ctypes.byref(B), es, ss, G, N, C, cd, ldc, counts, epi, bias, None)


@pytest.mark.parametrize("kw,code", [
    (dict(A=operand(dtype=0)), tg.TG_ERR_INVALID_ARG),               # bf16 operand
    (dict(A=operand(dtype=5)), tg.TG_ERR_INVALID_ARG),
    (dict(B=operand(layout=2)), tg.TG_ERR_INVALID_ARG),
    (dict(A=operand(block=64)), tg.TG_ERR_INVALID_ARG),
    (dict(A=operand(data=None)), tg.TG_ERR_INVALID_ARG),
    (dict(B=operand(layout=1, scale=None)), tg.TG_ERR_INVALID_ARG),
    (dict(A=operand(ld=112)), tg.TG_ERR_INVALID_ARG),                # ld < K
    (dict(A=operand(layout=1, ld=48)), tg.TG_ERR_INVALID_ARG),       # column-major A: ld < M
    (dict(B=operand(layout=0, ld=48)), tg.TG_ERR_INVALID_ARG),       # row-major B: ld < N
    (dict(A=operand(scale_stride=-1)), tg.TG_ERR_INVALID_ARG),
    (dict(A=operand(scale=2 * PTR + 2)), tg.TG_ERR_INVALID_ARG),
    (dict(A=operand(data=PTR + 8)), tg.TG_ERR_UNSUPPORTED),
    (dict(A=operand(ld=136)), tg.TG_ERR_UNSUPPORTED),
    (dict(cd=3), tg.TG_ERR_INVALID_ARG),
    (dict(cd=7), tg.TG_ERR_INVALID_ARG),
    (dict(epi=3), tg.TG_ERR_INVALID_ARG),
    (dict(epi=1), tg.TG_ERR_INVALID_ARG),                            # no bias
    (dict(epi=1, bias=PTR + 1), tg.TG_ERR_INVALID_ARG),
    (dict(C=None), tg.TG_ERR_INVALID_ARG),
    (dict(C=3 * PTR + 1), tg.TG_ERR_INVALID_ARG),
    (dict(ldc=63), tg.TG_ERR_INVALID_ARG),
    (dict(M=-1), tg.TG_ERR_INVALID_ARG),
    (dict(K=-128), tg.TG_ERR_INVALID_ARG),
    (dict(N=1 << 31, ldc=1 << 31), tg.TG_ERR_UNSUPPORTED),
])
def test_gemm_refusals(lib, kw, code):
    assert call_gemm(lib, **kw) == code
    assert lib.tg_last_error_message()


def test_gemm_null_operands_and_empty_sizes(lib):
    b = operand(layout=1)
    assert lib.tg_gemm_scaled(None, ctypes.byref(b), PTR, 0, 64, 64, 64, 128, 0, None, None) == tg.TG_ERR_INVALID_ARG
    assert lib.tg_gemm_scaled(ctypes.byref(b), None, PTR, 0, 64, 64, 64, 128, 0, None, None) == tg.TG_ERR_INVALID_ARG
    assert call_gemm(lib, M=0, A=operand(data=None, scale=None), C=None) == tg.TG_OK
    assert call_gemm(lib, N=0, C=None) == tg.TG_OK
    assert call_moe(lib, T=0, A=operand(data=None), C=None) == tg.TG_OK
    assert call_moe(lib, G=0, B=operand(layout=1, block=128, data=None), counts=None) == tg.TG_OK


@pytest.mark.parametrize("kw,code", [
    (dict(A=operand(layout=1)), tg.TG_ERR_INVALID_ARG),
    (dict(A=operand(block=128)), tg.TG_ERR_INVALID_ARG),
    (dict(B=operand(layout=1, block=1)), tg.TG_ERR_INVALID_ARG),
    (dict(counts=None), tg.TG_ERR_INVALID_ARG),
    (dict(counts=PTR + 2), tg.TG_ERR_INVALID_ARG),
    (dict(G=-1), tg.TG_ERR_INVALID_ARG),
    (dict(G=191), tg.TG_ERR_UNSUPPORTED),
    (dict(es=63 * 128), tg.TG_ERR_INVALID_ARG),
    (dict(es=64 * 128 + 8), tg.TG_ERR_UNSUPPORTED),
    (dict(ss=-1), tg.TG_ERR_INVALID_ARG),
    (dict(T=-1), tg.TG_ERR_INVALID_ARG),
])
def test_moe_refusals(lib, kw, code):
    assert call_moe(lib, **kw) == code
    assert lib.tg_last_error_message()


@pytest.mark.parametrize("kw,code", [
    (dict(x_dtype=3), tg.TG_ERR_INVALID_ARG),
    (dict(q_dtype=0), tg.TG_ERR_INVALID_ARG),
    (dict(br=64), tg.TG_ERR_INVALID_ARG),
    (dict(br=1, bc=1), tg.TG_ERR_INVALID_ARG),
    (dict(M=-1), tg.TG_ERR_INVALID_ARG),
    (dict(M=1 << 31), tg.TG_ERR_UNSUPPORTED),
    (dict(X=None), tg.TG_ERR_INVALID_ARG),
    (dict(Q=None), tg.TG_ERR_INVALID_ARG),
    (dict(scale=None), tg.TG_ERR_INVALID_ARG),
    (dict(scale=PTR + 1), tg.TG_ERR_INVALID_ARG),
    (dict(X=PTR + 1), tg.TG_ERR_INVALID_ARG),
    (dict(ldx=255), tg.TG_ERR_INVALID_ARG),
    (dict(ldq=255), tg.TG_ERR_INVALID_ARG),
    (dict(sld=9), tg.TG_ERR_INVALID_ARG),                     # 1 x 128: scale_ld < M
    (dict(br=128, bc=1, sld=255), tg.TG_ERR_INVALID_ARG),     # 128 x 1: scale_ld < K
    (dict(br=128, bc=128, sld=1), tg.TG_ERR_INVALID_ARG),     # 128 x 128: scale_ld < blocks
])
def test_quantize_refusals(lib, kw, code):
    a = dict(X=PTR, x_dtype=0, ldx=256, M=10, K=256, br=1, bc=128, Q=2 * PTR, q_dtype=3, ldq=256, scale=3 * PTR, sld=10)
    a.update(kw)
    assert lib.tg_quantize_blocks(a["X"], a["x_dtype"], a["ldx"], a["M"], a["K"], a["br"], a["bc"], a["Q"], a["q_dtype"],
                               a["ldq"], a["scale"], a["sld"], None) == code
    assert lib.tg_last_error_message()


def test_quantize_empty(lib):
    assert lib.tg_quantize_blocks(None, 0, 0, 0, 128, 1, 128, None, 3, 0, None, 0, None) == tg.TG_OK
    assert lib.tg_quantize_blocks(None, 0, 0, 5, 0, 1, 128, None, 3, 0, None, 0, None) == tg.TG_OK


def test_binding_refusals():
    a, s = torch.zeros(4, 256).to(E4), torch.ones(4, 2)
    b, sb = torch.zeros(64, 256).to(E4).t(), torch.ones(2, 1)
    with pytest.raises(TypeError):
        tg.gemm_fp8(a.float(), s, b, sb)
    with pytest.raises(ValueError):
        tg.gemm_fp8(a, s, b[:128], sb[:1])                       # inner dimensions
    with pytest.raises(ValueError):
        tg.gemm_fp8(a, s[:, :1], b, sb)                          # blocks of K
    with pytest.raises(ValueError):
        tg.gemm_fp8(a, s[:3], b, sb)                             # rows
    with pytest.raises(ValueError):
        tg.gemm_fp8(a, s.half(), b, sb)
    with pytest.raises(ValueError):
        tg.gemm_fp8(a, s, b, sb, epilogue="bias")
    with pytest.raises(ValueError):
        tg.gemm_fp8(a, s, b, sb, out=torch.zeros(4, 63))
    with pytest.raises(ValueError):
        tg.gemm_fp8(a[:, ::2], s[:, :1], b[::2], sb[:1])         # neither rows nor columns contiguous
    with pytest.raises(TypeError):
        tg.gemm_fp8(a, s, b, sb, out_dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        tg.gemm_fp8(a, s, b, sb)                                 # all well, but on the CPU
    with pytest.raises(ValueError):
        tg.quantize_fp8(a.float(), (64, 128))
    with pytest.raises(TypeError):
        tg.quantize_fp8(a.float(), dtype=torch.int8)
    with pytest.raises(TypeError):
        tg.quantize_fp8(a.double())
    with pytest.raises(ValueError):
        tg.quantize_fp8(a.float().t())
    with pytest.raises(ValueError):
        tg.quantize_fp8(a.float(), scale=torch.zeros(4, 2))      # a block column's scales are not side by side
    counts = torch.tensor([4], dtype=torch.int32)
    with pytest.raises(TypeError):
        tg.moe_gemm_fp8(a, s, b[None], sb[None], counts.long())
    with pytest.raises(ValueError):
        tg.moe_gemm_fp8(a, s, b[None], sb, counts)
    with pytest.raises(ValueError):
        tg.moe_gemm_fp8(a, s[:1], b[None], sb[None], counts)


def test_struct_layout():
    assert ctypes.sizeof(_binding.Fp8Operand) == 56
    assert _binding.Fp8Operand.dtype.offset == 40 and _binding.Fp8Operand.block.offset == 48


@pytest.mark.parametrize("view,want", [
    (lambda t: t, (0, 64)), (lambda t: t.t(), (1, 64)), (lambda t: t[:1], (0, 48)), (lambda t: t.t()[:, :1], (1, 48)),
    (lambda t: t[:, :1], (0, 64)), (lambda t: t.t()[:1], (1, 64)), (lambda t: t[:1, :1], (0, 16)),
])
def test_leading_dimensions(view, want):
    assert _binding._fp8_matrix(view(torch.zeros(7, 64).to(E4)[:, :40]), "t") == want


def test_reference_scale_is_the_smallest_power_of_two():
    x = torch.tensor([[448.0, 1.0], [449.0, -2.0], [224.0, 0.0], [0.0, 0.0], [1e-44, 0.0], [3e38, 1.0]])
    _, s = ref.quantize(x, (1, 128), E4)
    assert s.flatten().tolist() == [1.0, 2.0, 0.5, 1.0, 2.0 ** -126, 2.0 ** 120]


# ------------------------------------------------------------------------------------------ quantiser (GPU)


def cuda_gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def values(g, rows, cols, dtype):
    x = torch.randn(rows, cols, generator=g, device="cuda") * torch.exp(3 * torch.randn(rows, 1, generator=g, device="cuda"))
    x[torch.rand(rows, cols, generator=g, device="cuda") < 0.02] = 0.0
    return x.to(dtype)


def check_quantize(x, block, dtype, **kw):
    q, s = tg.quantize_fp8(x, block, dtype=dtype, **kw)
    tg.device_status()
    wq, ws = ref.quantize(x.cpu(), block, dtype)
    assert torch.equal(s.cpu().nan_to_num(-1.0), ws.nan_to_num(-1.0))
    assert torch.equal(q.cpu().float(), wq.float())
    return q, s


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [E4, E5])
@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("block", [(1, 128), (128, 1), (128, 128)])
def test_quantize(block, xt, dtype):
    g = cuda_gen(1)
    for M, K in ((1, 1), (1, 128), (3, 130), (129, 257), (260, 384), (200, 7)):
        check_quantize(values(g, M, K, xt), block, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("block", [(1, 128), (128, 1), (128, 128)])
def test_quantize_edges(block):
    x = torch.zeros(300, 300)
    x[0, 0], x[1, 1], x[2, 2] = 448.0, 449.0, 1e-44             # at and above the top, below the smallest scale
    x[140, 3], x[141, 140] = float("inf"), float("nan")
    x[5, 290], x[270, 270] = 3.4e38, -1.2e-38
    x[6] = torch.linspace(-500, 500, 300)                          # ties of the rounding among them
    check_quantize(x.cuda(), block, E4)
    check_quantize(x.cuda(), block, E5)
    check_quantize(x.bfloat16().cuda(), block, E4)
    check_quantize(x.half().cuda(), block, E4)                     # 3.4e38 becomes an infinity


@pytest.mark.gpu
@pytest.mark.parametrize("block", [(1, 128), (128, 1), (128, 128)])
def test_quantize_views_and_given_outputs(block):
    g = cuda_gen(2)
    full = values(g, 150, 403, torch.bfloat16)
    for x in (full[:, 1:302], full[3:140, 8:308], full[::2, :300]):  # odd base, aligned base, wide rows
        M, K = x.shape
        buf = torch.zeros(M, K + 5, dtype=torch.uint8, device="cuda")
        q = buf.view(E4)[:, 1:K + 1]                                 # unaligned rows
        shape = {(1, 128): (ref.blocks(K), M + 3), (128, 1): (ref.blocks(M), K + 2),
                 (128, 128): (ref.blocks(M), ref.blocks(K) + 1)}[block]
        s = torch.full(shape, -7.0, device="cuda")
        view = s[:, :M].t() if block == (1, 128) else s[:, :K] if block == (128, 1) else s[:, :ref.blocks(K)]
        check_quantize(x, block, E4, q=q, scale=view)
        pad = s[:, M:] if block == (1, 128) else s[:, view.shape[1]:]
        assert (pad == -7.0).all()
        assert not buf[:, 0].any() and not buf[:, K + 1:].any()


# ------------------------------------------------------------------------------------------ products (GPU)


def fp8(g, rows, cols, dtype, scale=1.0):
    """Random 8-bit values of the type's whole range of exponents, in rows of a multiple of 16."""
    x = torch.randn(rows, cols, generator=g, device="cuda") * 16.0 * scale
    full = torch.zeros(rows, -(-cols // 16) * 16, device="cuda").to(dtype)
    full[:, :cols] = x.to(dtype)
    return full[:, :cols]


def scales(g, *shape):
    """Any fp32 values, not powers of two alone."""
    return torch.exp(torch.randn(*shape, generator=g, device="cuda"))


def make(g, M, N, K, a_layout="row", b_layout="col", at=E4, bt=E4, sa="row", sb="square"):
    a = fp8(g, M, K, at) if a_layout == "row" else fp8(g, K, M, at).t()
    b = fp8(g, K, N, bt) if b_layout == "row" else fp8(g, N, K, bt).t()
    kb = ref.blocks(K)
    s_a = scales(g, kb, M).t() if sa == "row" else scales(g, ref.blocks(M), kb)
    s_b = scales(g, kb, N) if sb == "column" else scales(g, kb, ref.blocks(N))
    return a, s_a, b, s_b


def check_product(out, a, sa, b, sb, bias=None, epilogue="none"):
    want, size, z = ref.product(a, sa, b, sb, bias, epilogue)
    bound = ref.product_bound(want, size, z, a.shape[1], epilogue, out.dtype)
    err = (out.double() - want).abs()
    # fp16 cannot hold everything: there an infinity of the right sign is the rounded value
    big = want.abs() > torch.finfo(out.dtype).max
    err = torch.where(big & (out.double() == torch.sign(want) * float("inf")), torch.zeros_like(err), err)
    bad = ~(err <= bound)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outside the bound, first at "
                           f"{torch.nonzero(bad)[0].tolist()}, worst {float((err / bound).max()):.3g} of it")


LAYOUTS = [("row", "col"), ("row", "row"), ("col", "col"), ("col", "row")]


@pytest.mark.gpu
@pytest.mark.parametrize("tile", ["1x128", "2x256", None])
@pytest.mark.parametrize("a_layout,b_layout", LAYOUTS)
@pytest.mark.parametrize("sb", ["square", "column"])
def test_gemm_layouts(monkeypatch, tile, a_layout, b_layout, sb):
    if tile:
        monkeypatch.setenv("TG_TILE", tile)
    g = cuda_gen(3)
    for M, N, K in ((128, 128, 128), (1, 16, 128), (257, 130, 300), (300, 520, 1000), (17, 1000, 129), (513, 257, 16)):
        t = make(g, M, N, K, a_layout, b_layout, sb=sb)
        out = tg.gemm_fp8(*t, out_dtype=torch.float32)
        tg.device_status()
        check_product(out, *t)


@pytest.mark.gpu
@pytest.mark.parametrize("tile", ["1x128", "2x256", None])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("epilogue", ["none", "bias", "bias_gelu"])
def test_gemm_epilogues(monkeypatch, tile, out_dtype, epilogue):
    if tile:
        monkeypatch.setenv("TG_TILE", tile)
    g = cuda_gen(4)
    for M, N, K in ((200, 264, 384), (5, 77, 256), (300, 515, 0), (33, 1, 200)):
        a, sa, b, sb = make(g, M, N, K, sb="square")
        sa, sb = sa * 2.0 ** -8, sb * 2.0 ** -8
        bias = torch.randn(N, generator=g, device="cuda").bfloat16() if epilogue != "none" else None
        out = tg.gemm_fp8(a, sa, b, sb, bias=bias, epilogue=epilogue, out_dtype=out_dtype)
        tg.device_status()
        check_product(out, a, sa, b, sb, bias, epilogue)


@pytest.mark.gpu
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("epilogue", ["none", "bias", "bias_gelu"])
def test_gemm_many_tiles(out_dtype, epilogue):
    """More tiles than CTA pairs, whole and ragged, with a last wave in half tiles."""
    g = cuda_gen(20)
    for M, N, K in ((2560, 2560, 256), (3000, 2200, 200), (2049, 5121, 384)):
        a, sa, b, sb = make(g, M, N, K, sb="square")
        sa, sb = sa * 2.0 ** -8, sb * 2.0 ** -8
        bias = torch.randn(N, generator=g, device="cuda").bfloat16() if epilogue != "none" else None
        out = tg.gemm_fp8(a, sa, b, sb, bias=bias, epilogue=epilogue, out_dtype=out_dtype)
        tg.device_status()
        check_product(out, a, sa, b, sb, bias, epilogue)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    g = cuda_gen(21)
    M, N, K = 66000, 128, 128
    a, sa, b, sb = make(g, M, N, K)
    wide = torch.empty(M, 33000, dtype=torch.bfloat16, device="cuda")      # rows of C 33000 elements apart
    out = wide[:, 32800:32800 + N]
    tg.gemm_fp8(a, sa, b, sb, out)
    tg.device_status()
    check_product(out, a, sa, b, sb)
    x = wide[:, :256]
    x.copy_(torch.randn(M, 256, generator=g, device="cuda"))
    for block in ((1, 128), (128, 1), (128, 128)):
        q, s = tg.quantize_fp8(x, block)
        tail = x[-80:]                                                       # 66000 = 515 * 128 + 80
        wq, ws = ref.quantize(tail.cpu(), block, E4)
        assert torch.equal(q[-80:].cpu().float(), wq.float())
        assert torch.equal((s[-80:] if block == (1, 128) else s[-1:]).cpu(), ws)


@pytest.mark.gpu
@pytest.mark.parametrize("at,bt", [(E4, E5), (E5, E4), (E5, E5)])
@pytest.mark.parametrize("M", [3, 300])
def test_gemm_types(at, bt, M):
    g = cuda_gen(5)
    t = make(g, M, 200, 520, at=at, bt=bt)
    out = tg.gemm_fp8(*t, out_dtype=torch.float32)
    check_product(out, *t)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129])
def test_gemm_few_rows(M):
    g = cuda_gen(6)
    for N, K in ((384, 1024), (1000, 2176), (8, 128), (4096, 256)):
        for sb in ("square", "column"):
            t = make(g, M, N, K, sb=sb)
            bias = torch.randn(N, generator=g, device="cuda").bfloat16()
            out = tg.gemm_fp8(*t, bias=bias, epilogue="bias")
            tg.device_status()
            check_product(out, *t, bias, "bias")


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 40, 300])
def test_gemm_strided_scales_and_outputs(M):
    g = cuda_gen(7)
    N, K = 261, 700
    a, sa, b, sb = make(g, M, N, K, sa="square")                 # a scale per 128 x 128 block of A, too
    check_product(tg.gemm_fp8(a, sa, b, sb), a, sa, b, sb)
    sa = scales(g, M, 2 * ref.blocks(K))[:, ::2]                 # rows of scales with a step
    sb = scales(g, N, ref.blocks(K)).t()
    check_product(tg.gemm_fp8(a, sa, b, sb), a, sa, b, sb)
    one = torch.full((), 0.5, device="cuda")
    sa, sb = one.expand(M, ref.blocks(K)), one.expand(ref.blocks(K), ref.blocks(N))
    check_product(tg.gemm_fp8(a, sa, b, sb), a, sa, b, sb)       # one scale for all: strides of zero
    for dt in (torch.bfloat16, torch.float32):
        full = torch.full((M + 2, N + 6), -3.0, dtype=dt, device="cuda")
        out = full[1:M + 1, 1:N + 1]                             # rows and columns around it stay
        tg.gemm_fp8(a, sa, b, sb, out)
        check_product(out, a, sa, b, sb)
        full[1:M + 1, 1:N + 1] = -3.0
        assert (full == -3.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("tile", ["1x128", "2x256", None])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("start,step,line", [(0, 1, 1024), (0, 1, 1023), (1, 1, 1024), (2, 1, 1020), (0, 2, 2048), (0, 1, 0)])
def test_gemm_column_scales_of_any_stride(monkeypatch, tile, out_dtype, start, step, line):
    # lines of scales in 16-byte words or not, ending inside a word, one line for all k-blocks
    if tile:
        monkeypatch.setenv("TG_TILE", tile)
    g = cuda_gen(15)
    for M, N, K in ((1, 3, 700), (126, 259, 700), (515, 642, 1300)):
        a, _, b, _ = make(g, M, N, K, "col", "row")
        kb = ref.blocks(K)
        sa, sb = (scales(g, kb * 2048 + 4).as_strided((kb, n), (line, step), start) for n in (M, N))
        out = tg.gemm_fp8(a, sa.t(), b, sb, out_dtype=out_dtype)
        tg.device_status()
        check_product(out, a, sa.t(), b, sb)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [2, 150, 600])
def test_gemm_special_values(M):
    g = cuda_gen(8)
    a, sa, b, sb = make(g, M, 300, 400)
    clean = tg.gemm_fp8(a, sa, b, sb, out_dtype=torch.float32)
    bad_sa = sa.clone()
    bad_sa[1, 2] = float("nan")                                  # one row of A not finite
    out = tg.gemm_fp8(a, bad_sa, b, sb, out_dtype=torch.float32)
    assert torch.isnan(out[1]).all()
    keep = torch.arange(M, device="cuda") != 1
    assert torch.equal(out[keep], clean[keep])
    bad_sb = sb.clone()
    bad_sb[0, 1] = float("nan")                                  # columns 128..255 of B
    out = tg.gemm_fp8(a, sa, b, bad_sb, out_dtype=torch.float32)
    assert torch.isnan(out[:, 128:256]).all() and torch.equal(out[:, :128], clean[:, :128])
    bits = a.view(torch.uint8).clone()
    bits[0, 399] = 0x7F                                          # NaN in the last, short block
    full = torch.zeros(M, 400, dtype=torch.uint8, device="cuda")
    full.copy_(bits)
    out = tg.gemm_fp8(full.view(E4), sa, b, sb, out_dtype=torch.float32)
    assert torch.isnan(out[0]).all() and torch.equal(out[1:], clean[1:])


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 512, 4096), (64, 512, 4096), (200, 384, 2048), (512, 640, 1536)])
def test_gemm_repeats_bit_for_bit(M, N, K):
    t = make(cuda_gen(9), M, N, K)
    first = tg.gemm_fp8(*t, out_dtype=torch.float32)
    for _ in range(5):
        assert torch.equal(first, tg.gemm_fp8(*t, out_dtype=torch.float32))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 300])
def test_gemm_on_another_stream_and_in_a_graph(M):
    t = make(cuda_gen(10), M, 384, 1024)
    want = tg.gemm_fp8(*t)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = tg.gemm_fp8(*t, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    x = torch.randn(M, 1024, device="cuda").bfloat16()
    tg.quantize_fp8(x)                                           # kernels loaded before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, s = tg.quantize_fp8(x)
        y = tg.gemm_fp8(q, s, t[2], t[3])
    x.copy_(torch.randn(M, 1024, device="cuda"))
    graph.replay()
    q2, s2 = tg.quantize_fp8(x)
    assert torch.equal(y, tg.gemm_fp8(q2, s2, t[2], t[3]))


@pytest.mark.gpu
def test_quantised_linear_layer_forward_and_backward():
    """The three products of a linear layer on quantised operands, against the same products in 64 bits."""
    g = cuda_gen(11)
    T, I, O = 300, 384, 520
    x = torch.randn(T, I, generator=g, device="cuda").bfloat16()
    w = torch.randn(I, O, generator=g, device="cuda").bfloat16()
    dy = torch.randn(T, O, generator=g, device="cuda").bfloat16()
    xq, xs = tg.quantize_fp8(x)
    wq, ws = tg.quantize_fp8(w, (128, 128))
    gq, gs = tg.quantize_fp8(dy, dtype=E5)
    y = tg.gemm_fp8(xq, xs, wq, ws, out_dtype=torch.float32)
    check_product(y, xq, xs, wq, ws)
    dx = tg.gemm_fp8(gq, gs, wq.t(), ws.t(), out_dtype=torch.float32)
    check_product(dx, gq, gs, wq.t(), ws.t())
    xq, xs = tg.quantize_fp8(x, (128, 1))
    gq, gs = tg.quantize_fp8(dy, (128, 1), dtype=E5)
    dw = tg.gemm_fp8(xq.t(), xs.t(), gq, gs, out_dtype=torch.float32)
    check_product(dw, xq.t(), xs.t(), gq, gs)
    # and the layer's own products, as far as 3 (e4m3) and 2 (e5m2) mantissa bits go: relative errors of at most
    # 2^-4 and 2^-3 a factor, in the 2-norm of each result
    for got, want, rel in ((y, x.double() @ w.double(), 2 * 2.0 ** -4), (dx, dy.double() @ w.double().t(), 2.0 ** -4 + 2.0 ** -3),
                           (dw, x.double().t() @ dy.double(), 2.0 ** -4 + 2.0 ** -3)):
        assert (got.double() - want).norm() <= rel * want.norm()


# ------------------------------------------------------------------------------------------ experts (GPU)


def make_moe(g, counts, N, K, T=None, b_layout="col", at=E4):
    T = sum(counts) if T is None else T
    a, sa = fp8(g, T, K, at), scales(g, ref.blocks(K), T).t()
    G = len(counts)
    if b_layout == "col":
        b = torch.stack([fp8(g, N, -(-K // 16) * 16, E4) for _ in range(G)])[:, :, :K].transpose(1, 2)
        sb = scales(g, G, ref.blocks(N), ref.blocks(K)).transpose(1, 2)
    else:
        b = torch.stack([fp8(g, K, -(-N // 16) * 16, E4) for _ in range(G)])[:, :, :N]
        sb = scales(g, G, ref.blocks(K), ref.blocks(N))
    return a, sa, b, sb, torch.tensor(counts, dtype=torch.int32, device="cuda")


def check_moe(out, counts, a, sa, b, sb, bias=None, epilogue="none"):
    r = 0
    for i, m in enumerate(counts):
        if m:
            check_product(out[r:r + m], a[r:r + m], sa[r:r + m], b[i], sb[i], None if bias is None else bias[i], epilogue)
        r += m


@pytest.mark.gpu
@pytest.mark.parametrize("tile", ["1x128", "2x256", None])
@pytest.mark.parametrize("b_layout", ["col", "row"])
@pytest.mark.parametrize("epilogue", ["none", "bias", "bias_gelu"])
def test_moe(monkeypatch, tile, b_layout, epilogue):
    if tile:
        monkeypatch.setenv("TG_TILE", tile)
    g = cuda_gen(12)
    for counts, N, K in (([3, 0, 130, 1, 256, 0, 129, 300], 200, 272), ([0, 0, 5], 515, 640), ([1] * 40, 136, 256),
                         ([400], 256, 128), ([64, 64, 200], 384, 96)):
        t = make_moe(g, counts, N, K, b_layout=b_layout)
        t = t[:1] + (t[1] * 2.0 ** -8,) + t[2:3] + (t[3] * 2.0 ** -8,) + t[4:]
        bias = torch.randn(len(counts), N, generator=g, device="cuda").bfloat16() if epilogue != "none" else None
        out = tg.moe_gemm_fp8(*t, bias=bias, epilogue=epilogue, out_dtype=torch.float32)
        tg.device_status()
        check_moe(out, counts, *t[:4], bias, epilogue)


@pytest.mark.gpu
@pytest.mark.parametrize("tile", ["1x128", "2x256", None])
def test_moe_rows_past_the_counts_stay(monkeypatch, tile):
    if tile:
        monkeypatch.setenv("TG_TILE", tile)
    g = cuda_gen(13)
    counts = [7, 0, 140, 2]
    for T in (150, 149, 400):
        t = make_moe(g, counts, 136, 256, T=T)
        out = torch.full((T, 136), -5.0, dtype=torch.bfloat16, device="cuda")
        tg.moe_gemm_fp8(*t, out)
        tg.device_status()
        check_moe(out, counts, *t[:4])
        assert (out[sum(counts):] == -5.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("tile", ["1x128", "2x256", None])
@pytest.mark.parametrize("counts", [[60, 41], [50, -1], [2147483647, 2147483647]])
def test_moe_bad_counts_compute_nothing(monkeypatch, tile, counts):
    if tile:
        monkeypatch.setenv("TG_TILE", tile)
    t = make_moe(cuda_gen(14), [50, 50], 128, 256)
    out = torch.full((100, 128), -5.0, dtype=torch.bfloat16, device="cuda")
    tg.device_status()
    tg.moe_gemm_fp8(*t[:4], torch.tensor(counts, dtype=torch.int32, device="cuda"), out)
    with pytest.raises(tg.TGError) as e:
        tg.device_status()
    assert e.value.status == tg.TG_ERR_INVALID_ARG
    assert (out == -5.0).all()
    tg.moe_gemm_fp8(*t, out)                                     # the next call is untouched by it
    tg.device_status()
    check_moe(out, [50, 50], *t[:4])


@pytest.mark.gpu
def test_moe_equals_the_dense_product_and_repeats():
    g = cuda_gen(15)
    counts = [200, 0, 57, 300]
    t = make_moe(g, counts, 264, 512)
    out = tg.moe_gemm_fp8(*t, out_dtype=torch.float32)
    for _ in range(3):
        assert torch.equal(out, tg.moe_gemm_fp8(*t, out_dtype=torch.float32))
    check_moe(out, counts, *t[:4])


@pytest.mark.gpu
@pytest.mark.parametrize("epilogue", ["none", "bias_gelu"])
def test_moe_many_tiles(epilogue):
    """Enough rows an expert for CTA pairs, ragged and empty experts among them."""
    g = cuda_gen(22)
    counts = [1000, 0, 257, 1, 640, 129, 2048, 384]
    a, sa, b, sb, c = make_moe(g, counts, 1160, 256)
    sa, sb = sa * 2.0 ** -8, sb * 2.0 ** -8
    bias = torch.randn(len(counts), 1160, generator=g, device="cuda").bfloat16() if epilogue != "none" else None
    for dt in (torch.bfloat16, torch.float32):
        out = tg.moe_gemm_fp8(a, sa, b, sb, c, bias=bias, epilogue=epilogue, out_dtype=dt)
        tg.device_status()
        check_moe(out, counts, a, sa, b, sb, bias, epilogue)


@pytest.mark.gpu
@pytest.mark.parametrize("block", [0, 1])
def test_withheld_stage_times_out_and_the_next_call_works(block):
    t = make(cuda_gen(16), 2048, 2560, 1024)
    want = tg.gemm_fp8(*t)
    tg.device_status()
    tg.set_wait_budget_ms(50)
    try:
        tg.debug_withhold_stage(3, block)
        tg.gemm_fp8(*t)
        with pytest.raises(tg.TGError) as e:
            tg.device_status()
        assert e.value.status == tg.TG_ERR_TIMEOUT
    finally:
        tg.set_wait_budget_ms(0)
    assert torch.equal(tg.gemm_fp8(*t), want)
    tg.device_status()
