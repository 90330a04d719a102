"""The gate of a mixture-of-experts layer: refusals and the reference itself (CPU), parity with 64 bits (GPU)."""
import pytest
import torch

import fp8_reference as ref
import grouped_gemm_persistent_gb300 as tg
from grouped_gemm_persistent_gb300.build import build

PTR = 0x10000
INF = float("inf")


@pytest.fixture(scope="module")
def lib():
    build()
    return tg.load()


# ------------------------------------------------------------------------------------------ refusals (CPU)


def forward(lib, logits=PTR, dt=1, ld=64, T=4, G=64, k=2, e=PTR, w=PTR, c=PTR, loss=PTR, slope=PTR):
    return lib.tg_moe_router(logits, dt, ld, T, G, k, 0, e, w, c, loss, slope, None)


def backward(lib, logits=PTR, dt=1, ld=64, T=4, G=64, k=2, e=PTR, w=PTR, slope=PTR, dw=PTR, dl=PTR, out=2 * PTR, ldd=64):
    return lib.tg_moe_router_backward(logits, dt, ld, T, G, k, 0, e, w, slope, dw, dl, out, ldd, None)


SHARED = [
    (dict(dt=3), tg.TG_ERR_INVALID_ARG), (dict(dt=-1), tg.TG_ERR_INVALID_ARG), (dict(T=-1), tg.TG_ERR_INVALID_ARG),
    (dict(G=0, k=0), tg.TG_ERR_INVALID_ARG), (dict(k=0), tg.TG_ERR_INVALID_ARG), (dict(k=65), tg.TG_ERR_INVALID_ARG),
    (dict(G=1025, ld=1025), tg.TG_ERR_UNSUPPORTED), (dict(k=33), tg.TG_ERR_UNSUPPORTED),
    (dict(T=1 << 30, k=2), tg.TG_ERR_UNSUPPORTED), (dict(logits=None), tg.TG_ERR_INVALID_ARG),
    (dict(ld=63), tg.TG_ERR_INVALID_ARG), (dict(logits=PTR + 2), tg.TG_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(e=None), tg.TG_ERR_INVALID_ARG), (dict(w=None), tg.TG_ERR_INVALID_ARG), (dict(c=None), tg.TG_ERR_INVALID_ARG),
    (dict(loss=None), tg.TG_ERR_INVALID_ARG), (dict(slope=None), tg.TG_ERR_INVALID_ARG),
    (dict(w=PTR + 2), tg.TG_ERR_INVALID_ARG),
])
def test_forward_refusals(lib, kw, code):
    assert forward(lib, **kw) == code
    assert lib.tg_last_error_message()


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(e=None), tg.TG_ERR_INVALID_ARG), (dict(w=None), tg.TG_ERR_INVALID_ARG), (dict(slope=None), tg.TG_ERR_INVALID_ARG),
    (dict(out=None), tg.TG_ERR_INVALID_ARG), (dict(ldd=63), tg.TG_ERR_INVALID_ARG), (dict(out=PTR + 2), tg.TG_ERR_INVALID_ARG),
    (dict(dl=PTR + 1), tg.TG_ERR_INVALID_ARG),
])
def test_backward_refusals(lib, kw, code):
    assert backward(lib, **kw) == code
    assert lib.tg_last_error_message()


def test_backward_of_no_rows(lib):
    assert backward(lib, T=0, logits=None, out=None) == tg.TG_OK


def test_binding_refusals():
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        tg.moe_router(x.double(), 2)
    with pytest.raises(ValueError):
        tg.moe_router(x.t(), 2)
    with pytest.raises(ValueError):
        tg.moe_router(x, 0)
    with pytest.raises(ValueError, match="CUDA"):
        tg.moe_router(x, 2)
    r = tg.Routing(torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), torch.zeros(8, dtype=torch.int32),
                   torch.zeros(()), torch.zeros(8), False)
    with pytest.raises(ValueError):
        tg.moe_router_backward(x, r, torch.zeros(4, 3))
    with pytest.raises(ValueError):
        tg.moe_router_backward(x, r, torch.zeros(4, 2), torch.zeros(2))
    with pytest.raises(ValueError):
        tg.moe_router_backward(x, r, out=torch.zeros(4, 8).half())
    with pytest.raises(ValueError):
        tg.moe_router_backward(x, r._replace(slope=torch.zeros(9)))
    with pytest.raises(ValueError, match="CUDA"):
        tg.moe_router_backward(x, r, torch.zeros(4, 2))


@pytest.mark.parametrize("renorm", [False, True])
def test_reference_gradient_against_differences(renorm):
    g = torch.Generator().manual_seed(0)
    T, G, k = 5, 9, 3
    x = torch.randn(T, G, generator=g, dtype=torch.float64) * 2
    x[1, 4] = -INF
    x[2] = -INF
    dw, dl = torch.randn(T, k, generator=g, dtype=torch.float64), 0.7
    experts, _, counts, *_ = ref.route(x, k, renorm)
    d = ref.route_gradient(x, experts, counts, k, renorm, dw, dl)

    def value(y):
        e, w, c, loss, *_ = ref.route(y, k, renorm)
        assert torch.equal(e, experts)                            # the step does not change the choice
        return float((w * dw).sum() + dl * loss)

    h = 1e-6
    for t in range(T):
        for i in range(G):
            if x[t, i] == -INF:
                assert d[t, i] == 0
                continue
            up, down = x.clone(), x.clone()
            up[t, i] += h
            down[t, i] -= h
            assert abs((value(up) - value(down)) / (2 * h) - float(d[t, i])) < 1e-8


# ------------------------------------------------------------------------------------------ parity (GPU)

U = 2.0 ** -24      # half a step of fp32


def check_forward(x, k, renorm, r):
    experts, w, counts, loss, p, rows, chosen = ref.route(x, k, renorm)
    assert torch.equal(r.experts, experts)
    assert torch.equal(r.counts, counts)
    G = x.shape[1]
    # exp of a difference d: |d| half steps from the argument's rounding and 4 for the function; the sum adds G / 32 + 5
    # of them, the reciprocal, the product and the division of the renormalised form a few more
    span = (x.double().masked_fill(x == -INF, INF).amin() - x.double().masked_fill(x == INF, -INF).amax()).abs()
    span = min(float(span), 110.0) if torch.isfinite(span) else 110.0
    rel = (2 * span + G / 32 + 32) * U
    assert (~((r.weights.double() - w).abs() > rel * w + 1e-44)).all() and torch.equal(torch.isnan(r.weights), torch.isnan(w))
    n = max(rows, 1)
    # the loss adds up to n rows in fp32 (a warp's share), warps and blocks
    if torch.isnan(loss):
        assert torch.isnan(r.loss)
    else:
        assert abs(float(r.loss) - float(loss)) <= (rel + (n + 16) * U) * float(loss)
        assert ((r.slope.double() - G * counts.double() / (n * k) / n).abs() <= 2 * U * r.slope.double()).all()
    return experts, counts, p


def check_backward(x, k, r, dw, dl, renorm):
    out = tg.moe_router_backward(x, r, dw, dl)
    tg.device_status()
    want = ref.route_gradient(x, r.experts, r.counts, k, renorm, dw, dl)
    _, w, _, _, p, _, chosen = ref.route(x, k, renorm)
    G = x.shape[1]
    # size of the terms that are added: p u, p sum(p u), w w', p sum(w w')
    u = (r.slope.double() * (float(dl) if dl is not None else 0.0)).abs()
    term = p * u + p * (p * u).sum(1, keepdim=True)
    if dw is not None:
        a = torch.where(chosen, (w * dw.double()).abs(), torch.zeros_like(w))
        tot = a.sum(1, keepdim=True)
        term = term + p * tot
        extra = torch.zeros_like(p)
        extra.scatter_add_(1, r.experts.clamp(min=0).long(), a + w * tot)
        term = term + extra
    live = x.double().masked_fill(x == -INF, INF)
    span = min(float((live.amin() - x.double().amax()).abs()), 110.0)
    rel = (4 * span + G / 16 + 64) * U
    eps = torch.finfo(x.dtype).eps / 2                             # one rounding: half a step
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 1e-38
    bad = ~((out.double() - want).abs() <= rel * term + eps * 1.01 * want.abs() + tiny)
    assert not bad.any(), f"{int(bad.sum())} outside, first {torch.nonzero(bad)[0].tolist()}"
    assert (out[x == -INF] == 0).all()
    return out


def logits(seed, T, G, dtype, banned=0.0, padded=0.0, ties=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, G, generator=g, device="cuda") * 2
    if ties:
        x = torch.round(x)                                         # many equal logits, 0 and -0 among them
    x[torch.rand(T, G, generator=g, device="cuda") < banned] = -INF
    x[torch.rand(T, generator=g, device="cuda") < padded] = -INF
    return x.to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,G,k", [(1, 1, 1), (1, 8, 2), (7, 31, 5), (64, 64, 8), (300, 190, 6), (33, 256, 1), (50, 257, 32),
                                   (40, 600, 9), (9, 1024, 32), (1500, 60, 4)])
def test_router(T, G, k, renorm, dtype):
    for seed, kw in ((1, {}), (2, dict(banned=0.3, padded=0.2)), (3, dict(ties=True)), (4, dict(banned=0.97))):
        x = logits(seed, T, G, dtype, **kw)
        r = tg.moe_router(x, k, renormalize=renorm)
        tg.device_status()
        check_forward(x, k, renorm, r)
        g = torch.Generator(device="cuda").manual_seed(seed)
        dw = torch.randn(T, k, generator=g, device="cuda")
        dl = torch.randn((), generator=g, device="cuda") * T
        for a, b in ((dw, dl), (dw, None), (None, dl)):
            check_backward(x, k, r, a, b, renorm)
    none = tg.moe_router_backward(x, r)
    assert (none == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("G,k", [(60, 4), (256, 8), (256, 32), (300, 5), (1000, 7)])
def test_router_logits_that_differ_in_their_last_bits(G, k):
    """fp32 logits a few steps apart: the choice goes by value to the last bit, at the last place too."""
    g = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randn(64, G, generator=g, device="cuda")
    for t in range(64):
        n = min(G, (1, 2, k, k + 1, k + 2, G)[t % 6])              # so many near the top
        steps = torch.randperm(4 * n, generator=g, device="cuda")[:n]
        where = torch.randperm(G, generator=g, device="cuda")[:n]
        x[t, where] = (torch.full((n,), 8.0 if t % 2 else -0.001, device="cuda").view(torch.int32) + steps.int()).view(torch.float32)
        if t % 2 == 0:
            x[t] = torch.where(x[t] > -0.002, x[t], x[t] - 10.0)   # the near ones lead there, too
    x[5] = torch.where(torch.arange(G, device="cuda") % 2 == 0, 1.0, 1.0 + 2.0 ** -23)
    r = tg.moe_router(x, k, renormalize=True)
    tg.device_status()
    check_forward(x, k, True, r)


@pytest.mark.gpu
def test_router_no_rows_and_no_live_rows():
    for x in (torch.zeros(0, 16, device="cuda"), torch.full((5, 16), -INF, device="cuda")):
        r = tg.moe_router(x, 3, renormalize=True)
        tg.device_status()
        assert not r.counts.any() and float(r.loss) == 0 and not r.slope.any()
        assert (r.experts == -1).all() and (r.weights == 0).all()
        d = tg.moe_router_backward(x, r, torch.ones(x.shape[0], 3, device="cuda"), torch.ones((), device="cuda"))
        assert d.shape == x.shape and (d == 0).all()


@pytest.mark.gpu
def test_router_masks_of_the_lowest_value_and_far_logits():
    x = logits(5, 40, 50, torch.float32)
    x[0] = torch.finfo(torch.float32).min                          # finite: an even choice of the first k
    x[1, 3:] = torch.finfo(torch.float32).min
    x[2] = 1e30
    x[3] = torch.arange(50, device="cuda") * 100.0                 # probabilities that underflow
    x[4] += 30000.0
    r = tg.moe_router(x, 4)
    check_forward(x, 4, False, r)
    assert r.experts[0].tolist() == [0, 1, 2, 3]
    check_backward(x, 4, r, torch.randn(40, 4, device="cuda"), torch.ones((), device="cuda"), False)


@pytest.mark.gpu
def test_router_not_finite():
    x = logits(6, 30, 40, torch.float32)
    x[3, 7] = float("nan")
    x[4, 9] = INF
    r = tg.moe_router(x, 3, renormalize=False)
    tg.device_status()
    check_forward(x, 3, False, r)
    assert r.experts[3, 0] == 7 and r.experts[4, 0] == 9
    assert torch.isnan(r.weights[3:5]).all() and not torch.isnan(r.weights[5:]).any()
    d = tg.moe_router_backward(x, r, torch.ones(30, 3, device="cuda"))
    assert torch.isnan(d[3:5]).all() and not torch.isnan(d[5:]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_router_views_streams_and_repeats(dtype):
    full = logits(7, 5000, 100, dtype)
    for x in (full[:, 1:65], full[::3, 8:72], full[:, :64]):
        r = tg.moe_router(x, 4, renormalize=True)
        check_forward(x, 4, True, r)
        dw, dl = torch.randn(x.shape[0], 4, device="cuda"), torch.full((1,), 3.0, device="cuda")
        wide = torch.full((x.shape[0], 70), -9.0, dtype=dtype, device="cuda")
        d = tg.moe_router_backward(x, r, dw, dl, wide[:, 3:67])
        assert torch.equal(d, check_backward(x, 4, r, dw, dl, True))
        assert (wide[:, :3] == -9).all() and (wide[:, 67:] == -9).all()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        again = tg.moe_router(x, 4, renormalize=True, stream=side)
        side.synchronize()
        for a, b in zip(r[:5], again[:5]):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_router_in_a_graph_and_into_the_products():
    x = logits(8, 256, 16, torch.float32)
    tg.moe_router(x, 2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = tg.moe_router(x, 2)
        d = tg.moe_router_backward(x, r, None, r.loss)
    x.copy_(logits(9, 256, 16, torch.float32))
    graph.replay()
    want = tg.moe_router(x, 2)
    for a, b in zip(r[:5], want[:5]):
        assert torch.equal(a, b)
    assert torch.equal(d, tg.moe_router_backward(x, want, None, want.loss))
    graph.replay()                                                 # the counts start from zero every time
    torch.cuda.synchronize()
    assert torch.equal(r.counts, want.counts)
