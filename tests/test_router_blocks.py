"""The gate over many blocks and over several rows a slot: the join of the blocks' sums, the loops over the rows and
the wide forms, against 64 bits (GPU); the join's order of barrier and remote store (CPU)."""
import os
import re

import pytest
import torch

import grouped_gemm_persistent_gb300 as tg
from grouped_gemm_persistent_gb300.build import CSRC

INF = float("inf")
U = 2.0 ** -24      # half a step of fp32


def kernel_body(path: str, name: str) -> str:
    """Source of a kernel from its name to the brace that closes it, without comments."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, path)).read())
    at = text.index("{", text.index(name + "("))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i]
    raise AssertionError(f"{name}: no end")


def test_join_waits_for_its_cluster_before_the_remote_store():
    """Another block's shared memory may be used once that block has started, which a cluster barrier establishes."""
    body = kernel_body("tg_router.cu", "router_join_kernel")
    barriers = [m.start() for m in re.finditer(r"cluster_sync\(\)", body)]
    store = body.index("st.shared::cluster")
    assert any(b < store for b in barriers), "no cluster barrier before the first remote store"
    assert any(b > store for b in barriers), "no cluster barrier between the remote stores and their reader"


# ------------------------------------------------------------------------------------------ reference and bounds


def route(logits, k, renormalize):
    """(experts, weights, counts, loss, slope, p) in 64 bits, without a loop over the rows; no NaN in the logits."""
    x = logits.double()
    T, G = x.shape
    live = x.amax(1) > -INF
    p = torch.softmax(x.masked_fill(~live[:, None], 0.0), 1) * live[:, None]
    top = torch.sort(x, dim=1, descending=True, stable=True)
    taken = top.values[:, :k] > -INF
    idx = top.indices[:, :k]
    w = torch.where(taken, p.gather(1, idx), 0.0)
    if renormalize:
        w = torch.where(taken, w / w.sum(1, keepdim=True), 0.0)
    counts = torch.bincount(idx[taken], minlength=G)
    n = max(1, int(live.sum()))
    slope = G * counts.double() / (n * k) / n
    return torch.where(taken, idx, -1).int(), w, counts.int(), (slope * p.sum(0)).sum(), slope, p


def gradient(p, experts, w, slope, renormalize, dw, dl):
    """p (u - sum p u) and the chosen experts' terms, by the chain rule in 64 bits, and the sizes of what is added."""
    taken = experts >= 0
    d = torch.where(taken, dw.double(), 0.0) * w
    cw = d.sum(1, keepdim=True)
    extra = d - w * cw if renormalize else d
    u = slope * float(dl)
    c = (p * u).sum(1, keepdim=True) + (0.0 if renormalize else cw)
    at = experts.clamp(min=0).long()
    out = (p * (u - c)).scatter_add(1, at, torch.where(taken, extra, 0.0))
    tot = d.abs().sum(1, keepdim=True)
    size = (p * (u.abs() + (p * u.abs()).sum(1, keepdim=True) + tot)).scatter_add(1, at, d.abs() + w * tot)
    return out, size


def logits(seed, T, G, dtype=torch.float32, banned=0.1, padded=0.1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, G, generator=g, device="cuda") * 2
    x[torch.rand(T, G, generator=g, device="cuda") < banned] = -INF
    x[torch.rand(T, generator=g, device="cuda") < padded] = -INF
    return x.to(dtype)


def check_forward(x, k, renormalize, r):
    """Exact choices and counts; weights and loss within the fp32 operations that make them: an exponential of a
    difference d (2 |d| half steps for its argument and 4 for the function), the sum of G of them in G / 32 + 5 steps, and
    for the loss the sums over the rows, at most n in a row."""
    experts, w, counts, loss, slope, p = route(x, k, renormalize)
    assert torch.equal(r.experts, experts) and torch.equal(r.counts, counts)
    finite = x.double()[x > -INF]
    rel = (2 * float(finite.max() - finite.min()) + x.shape[1] / 32 + 32) * U
    assert ((r.weights.double() - w).abs() <= rel * w + 1e-44).all()
    assert abs(float(r.loss) - float(loss)) <= (rel + (x.shape[0] + 16) * U) * float(loss)
    assert ((r.slope.double() - slope).abs() <= 2 * U * slope).all()
    return experts, w, slope, p


# ------------------------------------------------------------------------------------------ the join (GPU)


@pytest.mark.gpu
@pytest.mark.parametrize("T,G,k", [(300, 8, 2), (5000, 16, 4), (20000, 32, 3), (700, 24, 24), (9000, 33, 2)])
def test_join_with_few_experts(T, G, k):
    """Up to 32 experts: one block of the join has work, and the others go straight to the loss."""
    x = logits(1, T, G)
    first = tg.moe_router(x, k)
    tg.device_status()
    check_forward(x, k, False, first)
    for _ in range(50):
        again = tg.moe_router(x, k)
        for a, b in zip(first[:5], again[:5]):
            assert torch.equal(a, b)


# ------------------------------------------------------------------------------------------ many rows, wide forms (GPU)


def check_backward(x, k, renormalize, r, w, slope, p, dw, dl):
    """Each term of the gradient is off by what its probability is (as in check_forward, the sums over the experts twice
    as many operations), and the result is rounded once to the logits' type."""
    out = tg.moe_router_backward(x, r, dw, dl)
    tg.device_status()
    want, size = gradient(p, r.experts, w, slope, renormalize, torch.zeros_like(w) if dw is None else dw,
                          0.0 if dl is None else dl)
    finite = x.double()[x > -INF]
    rel = (4 * float(finite.max() - finite.min()) + x.shape[1] / 16 + 64) * U
    eps = torch.finfo(x.dtype).eps / 2
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 1e-38       # half a step of fp16's subnormals
    bad = ~((out.double() - want).abs() <= rel * size + eps * 1.01 * want.abs() + tiny)
    assert not bad.any(), f"{int(bad.sum())} outside, first {torch.nonzero(bad)[0].tolist()}"
    assert (out[x == -INF] == 0).all()


# rows of one pass of the grid: 304 blocks of 16 warps, a row a warp above 128 experts, 2 above 64, 4 below
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,G,k", [(12001, 256, 8), (9729, 190, 6), (21000, 100, 5), (45001, 60, 4), (6000, 400, 9),
                                   (6001, 1000, 7), (300, 600, 3), (200, 1024, 32)])
def test_several_rows_a_slot_and_wide_gates(T, G, k, renorm, dtype):
    x = logits(T, T, G, dtype)
    r = tg.moe_router(x, k, renormalize=renorm)
    tg.device_status()
    experts, w, slope, p = check_forward(x, k, renorm, r)
    g = torch.Generator(device="cuda").manual_seed(2)
    dw = torch.randn(T, k, generator=g, device="cuda")
    dl = torch.randn((), generator=g, device="cuda") * T
    for a, b in ((dw, dl), (dw, None), (None, dl)):
        check_backward(x, k, renorm, r, w, slope, p, a, b)


@pytest.mark.gpu
def test_gradient_against_differences():
    """The kernel's own weights, a step of the logits either way: the derivative of sum(weights * dw), row by row."""
    T, G, k = 6000, 200, 4                             # more rows than one pass of the grid
    x = logits(5, T, G, banned=0.0, padded=0.0)
    r = tg.moe_router(x, k, renormalize=True)
    g = torch.Generator(device="cuda").manual_seed(3)
    dw = torch.randn(T, k, generator=g, device="cuda")
    d = tg.moe_router_backward(x, r, dw).double()
    tg.device_status()
    v = torch.randn(T, G, generator=g, device="cuda").double()
    h = 2.0 ** -10

    def value(y):
        s = tg.moe_router(y.float(), k, renormalize=True)
        return (s.weights.double() * dw.double()).sum(1), (s.experts == r.experts).all(1)

    up, same_up = value(x.double() + h * v)
    down, same_down = value(x.double() - h * v)
    ok = same_up & same_down                           # rows whose choice the step changes say nothing
    assert int(ok.sum()) > T // 2
    # the weights, which add up to 1, are off by `rel` of themselves (as in check_forward) and by the logits' rounding
    # to fp32; the third derivative is a fourth cumulant of dw and v, v, v: at most 64 |dw| |v|^3
    size, far = float(dw.abs().max()), float(x.abs().max()) + 1
    rel = (2 * 2 * far + G / 32 + 32 + 2 * far) * U
    bound = (rel / h + h * h * 64 / 6 * float(v.abs().max()) ** 3) * size
    err = ((d * v).sum(1) - (up - down) / (2 * h)).abs()[ok]
    assert float(err.max()) <= bound, float(err.max()) / bound


@pytest.mark.gpu
@pytest.mark.parametrize("T,G,k", [(5000, 16, 2), (12000, 256, 8)])
def test_gate_of_several_blocks_in_a_graph_into_the_experts(T, G, k):
    """Capture of the gate's workspace and its second kernel, and of the expert product that reads its counts."""
    import fp8_reference as ref
    D, N = 256, 136
    g = torch.Generator(device="cuda").manual_seed(4)
    x = logits(6, T, G, banned=0.0, padded=0.0)
    a = torch.randn(T, D, generator=g, device="cuda").bfloat16()
    wq = torch.randn(min(G, 190), N, D, generator=g, device="cuda").to(torch.float8_e4m3fn).transpose(1, 2)
    ws = torch.ones(wq.shape[0], D // 128, ref.blocks(N), device="cuda")
    x[:, wq.shape[0]:] = -INF                          # the expert product takes 190 experts
    dw = torch.randn(T, k, generator=g, device="cuda")

    def step():
        r = tg.moe_router(x, k, renormalize=True)
        rows = a[torch.argsort(r.experts.flatten(), stable=True) // k]
        q, s = tg.quantize_fp8(rows)
        counts = r.counts[:wq.shape[0]].contiguous()
        return (*r[:5], q.view(torch.uint8), s, tg.moe_gemm_fp8(q, s, wq, ws, counts), tg.moe_router_backward(x, r, dw, r.loss))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                         # kernels loaded before the capture
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (7, 8):
        x.copy_(logits(seed, T, G, banned=0.0, padded=0.0))
        x[:, wq.shape[0]:] = -INF
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = step()
        tg.device_status()
        check_forward(x, k, True, tg.moe_router(x, k, renormalize=True))
        for u, v in zip(got, want):
            assert torch.equal(u, v)
