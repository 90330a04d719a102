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
