"""RMS norm with the residual's addition and an 8-bit copy, and its gradients: refusals and the reference itself (CPU),
parity with 64 bits (GPU)."""
import subprocess

import pytest
import torch

import grouped_gemm_persistent_gb300 as tg
from grouped_gemm_persistent_gb300 import _binding
from grouped_gemm_persistent_gb300.build import INCLUDE, build

BF, HF, F = torch.bfloat16, torch.float16, torch.float32
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
EPS = 1e-6
U = 2.0 ** -24      # half a step of fp32
PTR = 0x10000


@pytest.fixture(scope="module")
def lib():
    build()
    return tg.load()


# ------------------------------------------------------------------------------------------ refusals (CPU)

FORWARD = dict(M=4, K=64, x=PTR, ldx=64, residual=2 * PTR, ldr=64, gain=3 * PTR, hidden=4 * PTR, ldh=64, y=5 * PTR, ldy=64,
               q=6 * PTR, ldq=64, scale=7 * PTR, scale_ld=4, row_scale=8 * PTR, eps=EPS, xt=0, rt=0, gt=1, yt=0, qt=3)
BACKWARD = dict(M=4, K=64, dy=PTR, lddy=64, hidden=2 * PTR, ldh=64, row_scale=3 * PTR, gain=4 * PTR, d_hidden=5 * PTR, lddh=64,
                dx=6 * PTR, lddx=64, d_gain=7 * PTR, dt=0, ht=0, gt=1)


def forward(lib, **kw):
    return lib.tg_rmsnorm(_binding._RMSNORM.pack(*{**FORWARD, **kw}.values()), None)


def backward(lib, **kw):
    return lib.tg_rmsnorm_backward(_binding._RMSNORM_BACKWARD.pack(*{**BACKWARD, **kw}.values()), None)


BAD, NO = tg.TG_ERR_INVALID_ARG, tg.TG_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), BAD), (dict(K=-1), BAD), (dict(M=1 << 31), NO), (dict(K=32769, ldx=1 << 16), NO), (dict(x=0), BAD),
    (dict(ldx=63), BAD), (dict(ldx=1 << 31), NO), (dict(x=PTR + 1), BAD), (dict(xt=3), BAD), (dict(xt=-1), BAD),
    (dict(rt=2), BAD), (dict(rt=9), BAD), (dict(ldr=63), BAD), (dict(residual=PTR + 1), BAD), (dict(hidden=0), BAD),
    (dict(ldh=63), BAD), (dict(gt=3), BAD), (dict(gain=PTR + 2), BAD), (dict(yt=4), BAD), (dict(ldy=63), BAD),
    (dict(y=PTR + 1), BAD), (dict(y=0, q=0), BAD), (dict(qt=0), BAD), (dict(ldq=63), BAD), (dict(scale=0), BAD),
    (dict(scale=PTR + 2), BAD), (dict(scale_ld=3), BAD), (dict(row_scale=0), BAD), (dict(row_scale=PTR + 2), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD),
])
def test_forward_refusals(lib, kw, code):
    assert forward(lib, **kw) == code
    assert lib.tg_last_error_message()


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), BAD), (dict(K=-1), BAD), (dict(K=32769), NO), (dict(dy=0), BAD), (dict(lddy=63), BAD), (dict(dt=3), BAD),
    (dict(ht=4), BAD), (dict(hidden=0), BAD), (dict(ldh=63), BAD), (dict(row_scale=0), BAD), (dict(gt=7), BAD),
    (dict(gain=PTR + 2), BAD), (dict(lddh=63), BAD), (dict(d_hidden=PTR + 1), BAD), (dict(dx=0), BAD), (dict(lddx=63), BAD),
    (dict(d_gain=PTR + 2), BAD),
])
def test_backward_refusals(lib, kw, code):
    assert backward(lib, **kw) == code
    assert lib.tg_last_error_message()


def test_null_record_and_no_rows(lib):
    assert lib.tg_rmsnorm(None, None) == BAD
    assert lib.tg_rmsnorm_backward(None, None) == BAD
    assert forward(lib, M=0, x=0, y=0, q=0, row_scale=0) == tg.TG_OK
    assert forward(lib, K=0) == tg.TG_OK
    assert backward(lib, M=0, d_gain=0, dy=0, dx=0) == tg.TG_OK


def test_records_match_the_header(tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "tg.h"\nint main(void) {\n'
                   'printf("%zu %zu %zu %zu\\n", sizeof(tg_rmsnorm_args), offsetof(tg_rmsnorm_args, eps),'
                   ' sizeof(tg_rmsnorm_backward_args), offsetof(tg_rmsnorm_backward_args, dy_dtype)); return 0; }\n')
    subprocess.run(["gcc", "-I", INCLUDE, str(src), "-o", str(tmp_path / "sizes")], check=True)
    out = subprocess.run([str(tmp_path / "sizes")], capture_output=True, text=True, check=True).stdout.split()
    f, b = _binding._RMSNORM.size, _binding._RMSNORM_BACKWARD.size
    assert [int(v) for v in out] == [f, f - 24, b, b - 16]


def test_binding_refusals():
    x = torch.zeros(4, 8, dtype=BF)
    n = tg.Normed(None, None, None, x, torch.zeros(4))
    with pytest.raises(TypeError):
        tg.rmsnorm(x.double())
    with pytest.raises(ValueError):
        tg.rmsnorm(x[0])
    with pytest.raises(ValueError):
        tg.rmsnorm(torch.zeros(8, 4, dtype=BF).t())
    with pytest.raises(TypeError):
        tg.rmsnorm(x, residual=x.half())
    with pytest.raises(ValueError):
        tg.rmsnorm(x, residual=x[:2])
    with pytest.raises(ValueError):
        tg.rmsnorm(x, hidden=x)
    with pytest.raises(TypeError):
        tg.rmsnorm(x, residual=x, hidden=x.float())
    with pytest.raises(ValueError):
        tg.rmsnorm(x, torch.ones(7))
    with pytest.raises(ValueError):
        tg.rmsnorm(x, torch.ones(16)[::2])
    with pytest.raises(TypeError):
        tg.rmsnorm(x, torch.ones(8).double())
    with pytest.raises(ValueError):
        tg.rmsnorm(x, out_dtype=None)
    with pytest.raises(TypeError):
        tg.rmsnorm(x, out_dtype=E4)
    with pytest.raises(TypeError):
        tg.rmsnorm(x, fp8_dtype=BF)
    with pytest.raises(ValueError, match="CUDA"):
        tg.rmsnorm(x)
    with pytest.raises(TypeError):
        tg.rmsnorm_backward(n, x.double())
    with pytest.raises(ValueError):
        tg.rmsnorm_backward(n, x[:2])
    with pytest.raises(TypeError):
        tg.rmsnorm_backward(n, x, None, x.float())
    with pytest.raises(TypeError):
        tg.rmsnorm_backward(n, x, out=x.float())
    with pytest.raises(ValueError):
        tg.rmsnorm_backward(n._replace(row_scale=torch.zeros(5)), x)
    with pytest.raises(ValueError, match="CUDA"):
        tg.rmsnorm_backward(n, x)


# ------------------------------------------------------------------------------------------ the reference


def reference(h, gain, eps=EPS):
    """(y, r) of the stream's rows in 64 bits."""
    h = h.double()
    r = 1.0 / (h.square().mean(1, keepdim=True) + eps).sqrt()
    return h * r * (1.0 if gain is None else gain.double()), r[:, 0]


def reference_gradient(h, gain, dy, d_hidden, eps=EPS):
    """(dx, d_gain, sum |d h| of each row, sum |dy h r| of each column) in 64 bits."""
    h, dy = h.double(), dy.double()
    _, r = reference(h, None, eps)
    r = r[:, None]
    d = dy if gain is None else dy * gain.double()
    dx = d * r - h * (d * h).sum(1, keepdim=True) * r ** 3 / h.shape[1]
    if d_hidden is not None:
        dx = dx + d_hidden.double()
    return dx, (dy * h * r).sum(0), (d * h).abs().sum(1, keepdim=True), (dy * h * r).abs().sum(0)


def test_reference_gradient_against_differences():
    g = torch.Generator().manual_seed(0)
    h, dy, dh = (torch.randn(3, 7, generator=g, dtype=torch.float64) for _ in range(3))
    gain = torch.rand(7, generator=g, dtype=torch.float64) + 0.5
    dx, d_gain, *_ = reference_gradient(h, gain, dy, dh)

    def value(h, gain):
        return float((reference(h, gain)[0] * dy).sum() + (h * dh).sum())

    step = 1e-6
    for t in range(3):
        for i in range(7):
            up, down = h.clone(), h.clone()
            up[t, i] += step
            down[t, i] -= step
            assert abs((value(up, gain) - value(down, gain)) / (2 * step) - float(dx[t, i])) < 1e-7
    for i in range(7):
        up, down = gain.clone(), gain.clone()
        up[i] += step
        down[i] -= step
        assert abs((value(h, up) - value(h, down)) / (2 * step) - float(d_gain[i])) < 1e-7


# ------------------------------------------------------------------------------------------ parity (GPU)


def smallest(t):
    """The spacing of a type's subnormal numbers."""
    i = torch.finfo(t)
    return i.tiny * i.eps


def make(seed, M, K, xt, rt=None, gt=None, offset=0):
    """x, residual, gain; with `offset` the rows start that many elements past an aligned address."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def mat(t):
        ld = (K + 15) // 8 * 8
        buf = torch.empty(M * ld + offset, dtype=t, device="cuda")
        m = buf[offset:].view(M, ld)[:, :K]
        return m.copy_(torch.randn(M, K, generator=g, device="cuda") * torch.exp(torch.randn(K, generator=g, device="cuda")))

    return mat(xt), None if rt is None else mat(rt), None if gt is None else (torch.randn(K, generator=g, device="cuda") + 1.0).to(gt)


def check_forward(x, residual, gain, n, eps=EPS):
    h = x if residual is None else (x.float() + residual.float()).to(residual.dtype)
    assert torch.equal(n.hidden, h)
    y, r = reference(h, gain, eps)
    # eight squares: a product's, a fused and two additions' roundings, halved by the root, and r's own
    assert bool(((n.row_scale.double() - r).abs() <= 3.1 * U * r).all())
    if n.y is not None:
        # r's error, two products, the type's rounding
        tol = y.abs() * (torch.finfo(n.y.dtype).eps / 2 * (1 + 6 * U) + 5.2 * U) + smallest(n.y.dtype) / 2 + smallest(F)
        assert bool(((n.y.double() - y).abs() <= tol).all())


def check_backward(n, gain, dy, dh, dx, d_gain, chain=64):
    want, want_gain, sums, columns = reference_gradient(n.hidden, gain, dy, dh)
    h, r = n.hidden.double(), n.row_scale.double()[:, None]
    d = dy.double().abs() * (1.0 if gain is None else gain.double().abs())
    # r three times 3.1 half steps; the row's sum: a chain of 8 + 8 additions in a thread, 5 in a warp, 16 warps, and the
    # product in front; a few products and additions behind
    one = d * r + (0 if dh is None else dh.double().abs())
    tol = torch.finfo(dx.dtype).eps / 2 * want.abs() * (1 + 64 * U) + U * (10 * one + 60 * h.abs() * sums * r ** 3 / h.shape[1]) + smallest(dx.dtype)
    assert bool(((dx.double() - want).abs() <= tol).all())
    if gain is None:
        assert d_gain is None
    else:
        assert bool(((d_gain.double() - want_gain).abs() <= chain * U * columns + smallest(F)).all())


SIZES = [(1, 1), (3, 7), (5, 8), (64, 128), (9, 129), (305, 1000), (2, 1024), (7, 1025), (700, 1544), (64, 4096), (311, 5000),
         (4, 8192), (306, 8200), (3, 16384), (5, 16400), (310, 32768)]
TYPES = [(BF, BF, BF), (BF, F, F), (HF, HF, F), (HF, F, HF), (F, F, F), (BF, None, None), (HF, None, HF), (F, None, BF)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,K", SIZES)
def test_sizes(M, K):
    for i, (xt, rt, gt) in enumerate(TYPES[:3] if M * K > 10 ** 6 else TYPES):
        x, residual, gain = make(i, M, K, xt, rt, gt)
        n = tg.rmsnorm(x, gain, EPS, residual=residual, out_dtype=(BF, HF, F)[i % 3], fp8_dtype=(E4, E5)[i % 2])
        check_forward(x, residual, gain, n)
        # the 8-bit copy is the quantiser's of the same fp32 rows
        y = tg.rmsnorm(x, gain, EPS, residual=residual, out_dtype=F).y
        q, scale = tg.quantize_fp8(y, (1, 128), dtype=n.q.dtype)
        assert torch.equal(n.q.view(torch.uint8), q.view(torch.uint8)) and torch.equal(n.scale, scale)
        only = tg.rmsnorm(x, gain, EPS, residual=residual, out_dtype=None, fp8_dtype=n.q.dtype)
        assert only.y is None and torch.equal(only.q.view(torch.uint8), q.view(torch.uint8))
        dy, dh, _ = make(100 + i, M, K, (BF, F, HF)[i % 3], n.hidden.dtype)
        for past in (dh, None):
            dx, d_gain = tg.rmsnorm_backward(n, dy, gain, past)
            check_backward(n, gain, dy, past, dx, d_gain)
    tg.device_status()


@pytest.mark.gpu
@pytest.mark.parametrize("M,K", [(2000, 1024), (5000, 4096), (20000, 200)])
def test_more_rows_than_one_pass(M, K):
    x, residual, gain = make(3, M, K, BF, BF, F)
    n = tg.rmsnorm(x, gain, EPS, residual=residual)
    check_forward(x, residual, gain, n)
    dy, dh, _ = make(4, M, K, BF, BF)
    dx, d_gain = tg.rmsnorm_backward(n, dy, gain, dh)
    check_backward(n, gain, dy, dh, dx, d_gain)
    again = tg.rmsnorm_backward(n, dy, gain, dh)
    assert torch.equal(again[0], dx) and torch.equal(again[1], d_gain)


@pytest.mark.gpu
@pytest.mark.parametrize("K", [100, 1544, 4104])
@pytest.mark.parametrize("xt,rt", [(BF, BF), (HF, F), (F, F)])
def test_rows_off_the_16_byte_boundaries(K, xt, rt):
    x, residual, _ = make(5, 33, K, xt, rt, None, offset=1)
    gain = torch.rand(K + 1, device="cuda").to(xt)[1:]
    n = tg.rmsnorm(x, gain, EPS, residual=residual, out_dtype=F, fp8_dtype=E4)
    check_forward(x, residual, gain, n)
    q, scale = tg.quantize_fp8(n.y, (1, 128))
    assert torch.equal(n.q.view(torch.uint8), q.view(torch.uint8)) and torch.equal(n.scale, scale)
    dy, dh, _ = make(6, 33, K, xt, rt, None, offset=3)
    dx, d_gain = tg.rmsnorm_backward(n, dy, gain, dh)
    check_backward(n, gain, dy, dh, dx, d_gain)


@pytest.mark.gpu
@pytest.mark.parametrize("K", [1, 7, 15, 17, 127, 129, 255, 257, 1001, 2049, 4095, 8193, 16383, 16391, 32767])
@pytest.mark.parametrize("xt,rt,gt", [(BF, BF, F), (HF, F, HF), (F, F, F)])
def test_rows_without_padding(K, xt, rt, gt):
    """Rows one behind the other, of odd length: each starts elsewhere, the last ends where the memory does."""
    M = 35

    def dense(seed, t):
        return make(seed, M, K, t)[0].contiguous()

    x, residual, dy, dh = dense(20, xt), dense(21, rt), dense(22, xt), dense(23, rt)
    gain = make(24, 1, K, F, None, gt)[2]
    rows = {name: torch.full((M * K + 64,), 7.0, dtype=rt, device="cuda") for name in ("hidden", "dx")}
    view = {name: t[32:32 + M * K].view(M, K) for name, t in rows.items()}
    n = tg.rmsnorm(x, gain, EPS, residual=residual, hidden=view["hidden"], out_dtype=F, fp8_dtype=E4)
    check_forward(x, residual, gain, n)
    q, scale = tg.quantize_fp8(n.y, (1, 128))
    assert torch.equal(n.q.view(torch.uint8), q.view(torch.uint8)) and torch.equal(n.scale, scale)
    half = tg.rmsnorm(x, gain, EPS, residual=residual, out_dtype=BF)
    check_forward(x, residual, gain, half)
    for past in (dh, None):
        dx, d_gain = tg.rmsnorm_backward(n, dy, gain, past, view["dx"])
        check_backward(n, gain, dy, past, dx, d_gain)
    for t in rows.values():
        assert bool((t[:32] == 7.0).all()) and bool((t[32 + M * K:] == 7.0).all())
    tg.device_status()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [5, 400])
@pytest.mark.parametrize("K", [200, 4096])
def test_in_place_and_nothing_beside_the_rows(M, K):
    """The stream written over the residual or x, the gradient over d_hidden; columns and rows beside them stay."""
    x, residual, gain = make(7, M, K, BF, BF, BF)
    want = tg.rmsnorm(x, gain, EPS, residual=residual)
    buf = torch.full((M + 2, K + 24), 7.0, dtype=BF, device="cuda")
    mine = buf[1:M + 1, 8:K + 8]
    mine.copy_(residual)
    n = tg.rmsnorm(x, gain, EPS, residual=mine, hidden=mine)
    assert n.hidden.data_ptr() == mine.data_ptr()
    assert torch.equal(mine, want.hidden) and torch.equal(n.y, want.y)
    over = x.clone()
    m = tg.rmsnorm(over, gain, EPS, residual=residual, hidden=over)
    assert torch.equal(over, want.hidden) and torch.equal(m.y, want.y)
    dy, dh, _ = make(8, M, K, BF, BF)
    dx, d_gain = tg.rmsnorm_backward(want, dy, gain, dh)
    grad = torch.full((M + 2, K + 24), 7.0, dtype=BF, device="cuda")
    past = grad[1:M + 1, 8:K + 8]
    past.copy_(dh)
    into, d_gain2 = tg.rmsnorm_backward(want, dy, gain, past, past)
    assert torch.equal(into, dx) and torch.equal(d_gain, d_gain2)
    over = dy.clone()
    assert torch.equal(tg.rmsnorm_backward(want, over, gain, dh, over)[0], dx)
    for b in (buf, grad):
        b[1:M + 1, 8:K + 8] = 7.0
        assert bool((b == 7.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("K", [8192, 10240, 12096, 12160, 12161, 12200, 12264, 12280, 12287, 12288, 12289, 12296])
@pytest.mark.parametrize("M", [3, 400])
def test_a_gain_that_just_fits(M, K):
    """The gain takes about as much shared memory as a kernel has without asking (48 KB, of which the row's sums take some)."""
    x, residual, gain = make(33, M, K, BF, BF, F)
    n = tg.rmsnorm(x, gain, EPS, residual=residual)
    check_forward(x, residual, gain, n)
    dx, d_gain = tg.rmsnorm_backward(n, x, gain, residual)
    check_backward(n, gain, x, residual, dx, d_gain)


@pytest.mark.gpu
@pytest.mark.parametrize("offset", [0, 1])
def test_long_and_longer_rows_in_turn(offset):
    """The same kernels with more, less and again more shared memory."""
    for K in (32768, 16400, 32768, 24000, 16640, 32768):
        x, residual, gain = make(32, 3, K, BF, BF, F, offset=offset)
        n = tg.rmsnorm(x, gain, EPS, residual=residual)
        check_forward(x, residual, gain, n)
        dx, d_gain = tg.rmsnorm_backward(n, x, gain, residual)
        check_backward(n, gain, x, residual, dx, d_gain)


@pytest.mark.gpu
@pytest.mark.parametrize("K", [4097, 12000, 16391, 16400, 32768])
@pytest.mark.parametrize("dt", [BF, F])
def test_long_gradients_in_place(K, dt):
    """The gradient written over d_hidden or over dy: what a row still reads of them is not lost."""
    for pad in (0, 3):                               # rows on 16-byte boundaries, and off them
        x, residual, gain = make(30, 9, K, dt, dt, F, offset=pad)
        dy, dh, _ = make(31, 9, K, dt, dt, None, offset=pad)
        n = tg.rmsnorm(x, gain, EPS, residual=residual)
        dx, d_gain = tg.rmsnorm_backward(n, dy, gain, dh)
        check_backward(n, gain, dy, dh, dx, d_gain)
        for which in (dh, dy):
            a, b = make(31, 9, K, dt, dt, None, offset=pad)[:2]
            over = a if which is dy else b
            got, got_gain = tg.rmsnorm_backward(n, a, gain, b, over)
            assert got is over or got.data_ptr() == over.data_ptr()
            assert torch.equal(over, dx) and torch.equal(got_gain, d_gain)


@pytest.mark.gpu
@pytest.mark.parametrize("K", [384, 2048])
def test_special_rows(K):
    x, residual, gain = make(9, 6, K, F, F, F)
    x[0] = 0.0
    residual[0] = 0.0
    x[1, 5] = float("inf")
    x[2, 200] = float("nan")
    x[3] = 1e18                       # squares that sum past 2^127 are refused by the definition; these do not
    residual[3] = 0.0
    x[4] = 1e-20                      # squares below fp32's numbers: eps is all there is
    residual[4] = 0.0
    n = tg.rmsnorm(x, gain, EPS, residual=residual, out_dtype=F, fp8_dtype=E4)
    assert bool((n.y[0] == 0).all()) and bool((n.scale[0] == 1).all()) and bool((n.q[0].float() == 0).all())
    assert float(n.row_scale[1]) == 0.0 and bool(n.y[1, 5].isnan()) and float(n.y[1, 6]) == 0.0
    assert bool(n.scale[1, 0].isnan()) and bool((n.q[1].float() == 0).all()) and bool((n.scale[1, 1:] == 1).all())
    assert bool(n.row_scale[2].isnan()) and bool(n.y[2].isnan().all()) and bool(n.scale[2].isnan().all())
    rest = torch.tensor([3, 4, 5], device="cuda")
    part = tg.Normed(n.y[rest], None, None, n.hidden[rest], n.row_scale[rest])
    check_forward(x[rest], residual[rest], gain, part)


@pytest.mark.gpu
def test_zero_rows_without_eps():
    """A zero row without eps is 0 / 0; the others are not touched by it."""
    x = torch.randn(3, 256, device="cuda")
    x[1] = 0.0
    n = tg.rmsnorm(x, None, 0.0, out_dtype=F)
    assert bool(n.row_scale[1].isinf()) and bool(n.y[1].isnan().all())
    keep = torch.tensor([0, 2], device="cuda")
    check_forward(x[keep], None, None, tg.Normed(n.y[keep], None, None, x[keep], n.row_scale[keep]), 0.0)


@pytest.mark.gpu
def test_empty():
    for M, K in ((0, 64), (4, 0), (0, 0)):
        x = torch.zeros(M, K, dtype=BF, device="cuda")
        gain = torch.ones(K, device="cuda")
        n = tg.rmsnorm(x, gain, residual=x, fp8_dtype=E4)
        assert n.y.shape == n.q.shape == n.hidden.shape == (M, K)
        dx, d_gain = tg.rmsnorm_backward(n, x, gain, x)
        assert dx.shape == (M, K) and bool((d_gain == 0).all())


@pytest.mark.gpu
def test_other_stream_and_graph():
    x, residual, gain = make(10, 300, 1544, BF, F, BF)
    dy, dh, _ = make(11, 300, 1544, BF, F)
    want = tg.rmsnorm(x, gain, EPS, residual=residual, fp8_dtype=E4)
    want_dx, want_gain = tg.rmsnorm_backward(want, dy, gain, dh)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    n = tg.rmsnorm(x, gain, EPS, residual=residual, fp8_dtype=E4, stream=side)
    dx, d_gain = tg.rmsnorm_backward(n, dy, gain, dh, stream=side)
    side.synchronize()
    assert torch.equal(n.y, want.y) and torch.equal(dx, want_dx) and torch.equal(d_gain, want_gain)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n = tg.rmsnorm(x, gain, EPS, residual=residual, fp8_dtype=E4)
        dx, d_gain = tg.rmsnorm_backward(n, dy, gain, dh)
    for _ in range(2):
        for t in (n.y, n.hidden, dx, d_gain):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(n.y, want.y) and torch.equal(n.q.view(torch.uint8), want.q.view(torch.uint8))
        assert torch.equal(dx, want_dx) and torch.equal(d_gain, want_gain)
