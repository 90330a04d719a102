"""Low-rank adapters of many requests: refusals (CPU), parity with 64 bits (GPU)."""
import subprocess

import pytest
import torch

import grouped_gemm_persistent_gb300 as tg
from grouped_gemm_persistent_gb300 import _binding
from grouped_gemm_persistent_gb300.build import INCLUDE, build

PTR = 0x10000
BF, HF, F = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24      # half a step of fp32
BAD, NO = tg.TG_ERR_INVALID_ARG, tg.TG_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build()
    return tg.load()


# ------------------------------------------------------------------------------------------ refusals (CPU)

ARGS = dict(T=4, K=64, N=32, r=16, G=3, x=PTR, ldx=64, a=2 * PTR, lda=64, sa=1024, b=3 * PTR, ldb=16, sb=512, adapters=4 * PTR,
            scale=5 * PTR, base=6 * PTR, ldbase=32, out=7 * PTR, ldo=32, dt=0, bt=0)


def call(lib, **kw):
    return lib.tg_lora_add(_binding._LORA.pack(*{**ARGS, **kw}.values()), None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), BAD), (dict(K=-1), BAD), (dict(N=-1), BAD), (dict(r=-1), BAD), (dict(G=-1), BAD), (dict(T=1 << 31), NO),
    (dict(K=(1 << 31) - 1), NO), (dict(N=(1 << 31) - 1), NO), (dict(r=129, ldb=129), NO), (dict(dt=1), BAD), (dict(dt=3), BAD),
    (dict(bt=3), BAD), (dict(x=0), BAD), (dict(a=0), BAD), (dict(b=0), BAD), (dict(base=0), BAD), (dict(out=0), BAD),
    (dict(adapters=0), BAD), (dict(adapters=PTR + 2), BAD), (dict(scale=PTR + 1), BAD), (dict(ldx=63), BAD), (dict(lda=63), BAD),
    (dict(ldb=15), BAD), (dict(ldbase=31), BAD), (dict(ldo=31), BAD), (dict(x=PTR + 1), BAD), (dict(bt=1, out=PTR + 2), BAD),
    (dict(sa=-1), BAD), (dict(sb=-1), BAD), (dict(ldx=1 << 31), NO)])
def test_refusals(lib, kw, code):
    assert call(lib, **kw) == code
    assert lib.tg_last_error_message()


def test_null_record_and_nothing_to_do(lib):
    assert lib.tg_lora_add(None, None) == BAD
    assert call(lib, T=0, x=0, base=0, out=0) == tg.TG_OK
    assert call(lib, N=0, base=0, out=0) == tg.TG_OK


def test_record_matches_the_header(tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "tg.h"\nint main(void) {\n'
                   'printf("%zu %zu\\n", sizeof(tg_lora_args), offsetof(tg_lora_args, dtype)); return 0; }\n')
    subprocess.run(["gcc", "-I", INCLUDE, str(src), "-o", str(tmp_path / "sizes")], check=True)
    out = subprocess.run([str(tmp_path / "sizes")], capture_output=True, text=True, check=True).stdout.split()
    n = _binding._LORA.size
    assert [int(v) for v in out] == [n, n - 8]


def test_binding_refusals():
    base, x, a, b = torch.zeros(4, 6, dtype=BF), torch.zeros(4, 8, dtype=BF), torch.zeros(3, 2, 8, dtype=BF), torch.zeros(3, 6, 2, dtype=BF)
    ids = torch.zeros(4, dtype=torch.int32)

    def bad(error, match=None, **kw):
        args = dict(base=base, x=x, a=a, b=b, adapters=ids) | kw
        with pytest.raises(error, match=match):
            tg.lora_add(**args)

    bad(TypeError, x=x.float())
    bad(TypeError, a=a.half())
    bad(TypeError, base=base.double())
    bad(ValueError, x=x[:3])
    bad(ValueError, a=a[:, :, :7])
    bad(ValueError, b=b[:2])
    bad(ValueError, a=torch.zeros(3, 8, 2, dtype=BF).transpose(1, 2))
    bad(ValueError, adapters=ids.long())
    bad(ValueError, adapters=ids[:3])
    bad(ValueError, scale=torch.zeros(2))
    bad(ValueError, scale=torch.zeros(3, dtype=BF))
    bad(ValueError, x=torch.zeros(8, 4, dtype=BF).t())
    bad(ValueError, out=base.float())
    bad(ValueError, "CUDA")


# ------------------------------------------------------------------------------------------ parity (GPU)


def reference(base, x, a, b, ids, scale):
    """(out, error bound before its rounding) in 64 bits."""
    want, tol = base.double().clone(), torch.zeros(base.shape, dtype=torch.float64, device=base.device)
    K, G, r = x.shape[1], a.shape[0], a.shape[1]
    # what a sum along K is off by, of its magnitudes: an instruction's sum of 17 numbers to four half steps, K / 128 + 1 of
    # them a warp, then 8 warps and the factor (the other form: 16 + 5 additions, one a cut of 512, the factor)
    first = (4 * (K / 128 + 1) + 32) * U
    for g in range(G):
        rows = torch.nonzero(ids == g)[:, 0]
        if not rows.numel():
            continue
        s = 1.0 if scale is None else float(scale[g])
        xr, ag, bg = x[rows].double(), a[g].double(), b[g].double()
        u, mag = s * (xr @ ag.t()), abs(s) * (xr.abs() @ ag.abs().t())
        want[rows] += u @ bg.t()
        # hi + lo: 2^-17 of a value, or with fp16 2^-21 of its row's largest; its instructions along r as along K
        cut = 2.0 ** -17 * u.abs() if x.dtype == BF else 2.0 ** -21 * u.abs().amax(1, keepdim=True).expand_as(u)
        tol[rows] = (first * mag + cut + (8 * (r / 16 + 1) + 4) * U * u.abs()) @ bg.abs().t()
    return want, tol


def check(base, x, a, b, ids, scale, out):
    want, tol = reference(base, x, a, b, ids, scale)
    t = out.dtype
    tol = tol + (torch.finfo(t).eps / 2 * (1 + 4 * U) + 2 * U) * (want.abs() + tol) + torch.finfo(t).tiny * torch.finfo(t).eps
    assert bool(((out.double() - want).abs() <= tol).all())
    none = (ids < 0) | (ids >= a.shape[0])
    assert torch.equal(out[none], base[none])


def adapters_of(g, T, G, kind):
    if kind == "rows":                                             # every row its own, some none, some out of range
        ids = torch.randint(-1, G + 2, (T,), generator=g, device="cuda")
        ids[ids == G + 1] = -7
    elif kind == "requests":
        cuts = torch.sort(torch.randint(0, T + 1, (6,), generator=g, device="cuda")).values
        which = torch.randint(-1, G, (7,), generator=g, device="cuda")
        ids = which[(torch.arange(T, device="cuda")[:, None] >= cuts).sum(1)]
    elif kind == "none":
        ids = torch.full((T,), -1, device="cuda")
    else:
        ids = torch.full((T,), G - 1, device="cuda")
    return ids.int()


def make(seed, T, K, N, r, G, dt, bt, kind, scaled=True, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def mat(rows, cols, t, size=1.0):
        m = torch.empty(rows, cols + pad, dtype=t, device="cuda")[:, pad // 2:pad // 2 + cols]
        return m.copy_(torch.randn(rows, cols, generator=g, device="cuda") * size)

    a = mat(G * r, K, dt, max(K, 1) ** -0.5)
    b = mat(G * N, r, dt, 0.5)
    a, b = a.as_strided((G, r, K), (r * a.stride(0), a.stride(0), 1)), b.as_strided((G, N, r), (N * b.stride(0), b.stride(0), 1))
    scale = torch.randn(G, generator=g, device="cuda") + 1.0 if scaled else None
    return mat(T, N, bt), mat(T, K, dt), a, b, adapters_of(g, T, G, kind), scale


SIZES = [  # T, K, N, r, G
    (1, 4096, 4096, 16, 8), (1, 100, 33, 1, 1), (3, 257, 72, 4, 2), (17, 1544, 520, 8, 5), (64, 512, 1024, 64, 4), (60, 1000, 256, 17, 7),
    (31, 640, 96, 128, 3), (65, 256, 40, 64, 3), (100, 96, 1544, 128, 5), (300, 1544, 136, 16, 6), (129, 31, 7, 40, 2),
    (1000, 257, 300, 32, 20), (700, 2000, 64, 100, 4), (513, 64, 64, 8, 1), (4870, 520, 72, 16, 9), (4900, 136, 264, 33, 5),
    (5000, 264, 130, 64, 30), (4900, 72, 100, 30, 3), (70, 0, 64, 64, 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,r,G", SIZES)
@pytest.mark.parametrize("dt", [BF, HF])
def test_sizes(T, K, N, r, G, dt):
    for i, (bt, kind) in enumerate(((dt, "requests"), (F, "rows"), (HF if dt == BF else BF, "one"), (dt, "rows"), (F, "none"))):
        base, x, a, b, ids, scale = make(i, T, K, N, r, G, dt, bt, kind, scaled=i != 3)
        check(base, x, a, b, ids, scale, tg.lora_add(base, x, a, b, ids, scale))
    tg.device_status()


TILES = [  # more rows, or more work a row: 64-, 32- and 16-row tiles of every width of ranks, clusters, adapters that share a bucket
    (4200, 259, 70, 12, 3), (4200, 64, 72, 31, 5), (4200, 200, 136, 60, 4), (4200, 257, 33, 128, 2), (4500, 257, 33, 9, 200),
    (4500, 96, 200, 24, 200), (4300, 130, 64, 50, 300), (4500, 64, 129, 100, 150), (4200, 72, 40, 8, 700), (5000, 40, 72, 40, 2000),
    (600, 4096, 2000, 64, 2), (600, 4100, 500, 16, 100), (520, 4104, 1500, 32, 3), (700, 2056, 1000, 128, 1), (300, 5000, 4096, 20, 40)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,r,G", TILES)
@pytest.mark.parametrize("dt", [BF, HF])
def test_tiles(T, K, N, r, G, dt):
    for i, (bt, kind) in enumerate(((dt, "rows"), (F, "requests"), (dt, "one"))):
        base, x, a, b, ids, scale = make(i, T, K, N, r, G, dt, bt, kind)
        check(base, x, a, b, ids, scale, tg.lora_add(base, x, a, b, ids, scale))
    tg.device_status()


@pytest.mark.gpu
@pytest.mark.parametrize("G", [255, 256, 350, 370, 375, 379, 380, 381, 382, 383, 384, 385, 511, 512, 513, 700])
def test_numbers_of_adapters(G):
    """The order of the rows counts by adapter in shared memory: about as much as a kernel has without asking, and more."""
    base, x, a, b, ids, scale = make(40, 5000, 64, 40, 8, G, BF, BF, "rows")
    check(base, x, a, b, ids, scale, tg.lora_add(base, x, a, b, ids, scale))


@pytest.mark.gpu
@pytest.mark.parametrize("T,r", [(20, 16), (90, 64), (300, 100), (5000, 32)])
@pytest.mark.parametrize("pad", [2, 8, 6])
def test_strides_and_in_place(T, r, pad):
    """Rows off the 16-byte boundaries and wider than they need be; out over base; what lies beside the rows stays."""
    for bt in (BF, F):
        base, x, a, b, ids, scale = make(40, T, 264, 136, r, 6, BF, bt, "rows", pad=pad)
        want = tg.lora_add(base, x, a, b, ids, scale)
        check(base, x, a, b, ids, scale, want)
        buf = torch.full((T + 2, 136 + 16), 7.0, dtype=bt, device="cuda")
        for at in (0, 3, 8):
            buf.fill_(7.0)
            mine = buf[1:T + 1, at:at + 136]
            mine.copy_(base)
            assert tg.lora_add(mine, x, a, b, ids, scale, mine) is mine
            assert torch.equal(mine, want)
            mine.fill_(7.0)
            assert bool((buf == 7.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [16, 200, 5000])
@pytest.mark.parametrize("dt", [BF, HF])
def test_a_fault_stays_in_its_rows(T, dt):
    """NaN and infinity in an adapter, in a row of x, and in an adapter's factor."""
    base, x, a, b, ids, scale = make(41, T, 320, 200, 64, 5, dt, dt, "rows")
    ids[3], ids[5] = 1, 2
    want = tg.lora_add(base, x, a, b, ids, scale)
    a, b, x, scale = a.clone(), b.clone(), x.clone(), scale.clone()
    a[0, 3, 7] = float("nan")
    b[2, 9, 5] = float("inf")
    scale[4] = float("nan")
    x[3] = float("inf")
    got = tg.lora_add(base, x, a, b, ids, scale)
    touched = (ids == 0) | (ids == 2) | (ids == 4)
    touched[3] = True
    assert torch.equal(got[~touched], want[~touched])
    assert bool(got[ids == 0].isnan().all()) and bool(got[ids == 4].isnan().all())
    assert not bool(got[3].isfinite().any())
    two = torch.nonzero(ids == 2)[:, 0]
    assert not bool(got[two, 9].isfinite().any())
    rest = torch.tensor([n for n in range(200) if n != 9], device="cuda")
    assert torch.equal(got[two][:, rest], want[two][:, rest])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [20, 200])
def test_fp16_values_far_from_one(T):
    """Products beyond fp16's range, and far below it, between the two products."""
    base, x, a, b, ids, scale = make(42, T, 256, 64, 32, 3, HF, F, "rows")
    for size in (200.0, 1e-3):
        y, c = x * size, a * size
        small = (b * (1e-4 if size > 1 else 100.0)).to(HF)
        check(base, y, c, small, ids, scale, tg.lora_add(base, y, c, small, ids, scale))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 100])
def test_without_adapters(T):
    base, x = torch.randn(T, 40, device="cuda"), torch.randn(T, 16, device="cuda").to(BF)
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    for G, r in ((0, 8), (3, 0)):
        a, b = torch.zeros(G, r, 16, dtype=BF, device="cuda"), torch.zeros(G, 40, r, dtype=BF, device="cuda")
        assert torch.equal(tg.lora_add(base, x, a, b, ids), base)
    a, b = torch.zeros(3, 8, 16, dtype=BF, device="cuda"), torch.zeros(3, 40, 8, dtype=BF, device="cuda")
    assert tg.lora_add(base[:0], x[:0], a, b, ids[:0]).shape == (0, 40)
    assert tg.lora_add(base[:, :0], x, a, b[:, :0], ids).shape == (T, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [20, 200])
def test_adapters_past_32_bits(T):
    """The last of 2100 adapters of a million values each."""
    G, r, K, N = 2100, 64, 16384, 96
    a, b = torch.empty(G, r, K, dtype=BF, device="cuda"), torch.empty(G, N, r, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(43)
    a[-1] = torch.randn(r, K, generator=g, device="cuda") / 128
    b[-1] = torch.randn(N, r, generator=g, device="cuda") / 8
    x, base = torch.randn(T, K, generator=g, device="cuda").to(BF), torch.randn(T, N, generator=g, device="cuda").to(BF)
    out = tg.lora_add(base, x, a, b, torch.full((T,), G - 1, dtype=torch.int32, device="cuda"))
    check(base, x, a[-1:], b[-1:], torch.zeros(T, dtype=torch.int32, device="cuda"), None, out)


@pytest.mark.gpu
def test_rows_past_32_bits():
    T, K, N, r = 140000, 16384, 40, 16
    x, base = torch.empty(T, K, dtype=BF, device="cuda"), torch.zeros(T, N, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(44)
    x[-50:] = torch.randn(50, K, generator=g, device="cuda")
    a, b = torch.randn(1, r, K, generator=g, device="cuda").to(BF) / 128, torch.randn(1, N, r, generator=g, device="cuda").to(BF)
    ids = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    ids[-50:] = 0
    out = tg.lora_add(base, x, a, b, ids)
    check(base[-50:], x[-50:], a, b, ids[-50:], None, out[-50:])
    assert bool((out[:-50] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [20, 500])
def test_streams_graphs_and_repeats(T):
    base, x, a, b, ids, scale = make(45, T, 520, 136, 16, 6, BF, BF, "requests")
    want = tg.lora_add(base, x, a, b, ids, scale)
    assert torch.equal(tg.lora_add(base, x, a, b, ids, scale), want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = tg.lora_add(base, x, a, b, ids, scale, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graphs = []
    for _ in range(2):                                              # two graphs with workspaces of their own
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = tg.lora_add(base, x, a, b, ids, scale)
        graphs.append((graph, out))
    for graph, out in graphs * 2:
        out.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for _, out in graphs)
