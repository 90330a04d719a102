"""The operators one after the other, as a served and as a trained block uses them (GPU).

* Serving: the norm's two outputs into the 8-bit projection and, beside it, the requests' adapters.
* Training: the norm's 8-bit copy into the experts, chosen by a gate with sigmoid scores, a bias and groups, forward and
  backward through ``MoELayer.block``.
"""
import pytest
import torch

import fp8_reference as ref
import grouped_gemm_persistent_gb300 as tg
from grouped_gemm_persistent_gb300 import moe_layer
from grouped_gemm_persistent_gb300.build import build

pytestmark = pytest.mark.gpu

E4 = torch.float8_e4m3fn


def wide(q, s):
    return q.float().double() * ref.expand(s, q.shape)


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


def randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()


def serve(x, residual, gain, w, sw, a, b, ids, scale):
    """One decoding step or prompt of a projection with adapters: (result, stream)."""
    n = tg.rmsnorm(x, gain, residual=residual, fp8_dtype=E4)
    base = tg.gemm_fp8(n.q, n.scale, w.t(), sw.t())
    return tg.lora_add(base, n.y, a, b, ids, scale), n.hidden


@pytest.mark.parametrize("T", [1, 37, 700])
def test_projection_with_adapters(T):
    g = torch.Generator(device="cuda").manual_seed(21)
    K, N, r, G = 512, 768, 16, 5
    x, residual, gain = randn(g, T, K), randn(g, T, K), randn(g, K) + 1
    w, sw = tg.quantize_fp8(randn(g, N, K, scale=K ** -0.5), (128, 128))
    a, b = randn(g, G, r, K, scale=K ** -0.5), randn(g, G, N, r, scale=0.3)
    ids = (torch.arange(T, device="cuda") * G // T - 1).int()
    scale = torch.rand(G, device="cuda") + 0.5
    out, stream = serve(x, residual, gain, w, sw, a, b, ids, scale)
    # 64 bits on the same 8-bit and bf16 operands
    h = (x.float() + residual.float()).bfloat16()
    assert torch.equal(stream, h)
    n = h.double() / (h.double().square().mean(1, keepdim=True) + 1e-6).sqrt() * gain.double()
    q, s = tg.quantize_fp8(tg.rmsnorm(x, gain, residual=residual, out_dtype=torch.float32).y)
    base = wide(q, s) @ wide(w, sw).t()
    size = wide(q, s).abs() @ wide(w, sw).abs().t()
    y = n.bfloat16().double()
    add, add_size = torch.zeros_like(base), torch.zeros_like(base)
    for i in range(G):
        rows = ids == i
        f = float(scale[i])
        add[rows] = f * (y[rows] @ a[i].double().t()) @ b[i].double().t()
        add_size[rows] = f * (y[rows].abs() @ a[i].double().abs().t()) @ b[i].double().abs().t()
    # base is rounded to bf16 (2^-8 at most) and so is the sum; y may have fallen on the other side of a border (2^-8 of itself in a
    # few places); the products' fp32 sums
    tol = 2.0 ** -8 * (base.abs() + (base + add).abs() + add_size) + 2.0 ** -14 * size
    assert bool(((out.double() - base - add).abs() <= tol).all())
    # the same captured and replayed, as a serving loop runs it
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        again, stream2 = serve(x, residual, gain, w, sw, a, b, ids, scale)
    again.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, out) and torch.equal(stream2, stream)
    tg.device_status()


@pytest.mark.parametrize("T,G,k,groups", [(200, 16, 2, 4), (513, 32, 4, 8)])
def test_block_of_experts(T, G, k, groups):
    g = torch.Generator(device="cuda").manual_seed(22)
    D, H = 256, 384
    x, residual, gain = randn(g, T, D), randn(g, T, D), randn(g, D, scale=0.2) + 1
    gate, w1, b1, w2 = randn(g, G, D, scale=D ** -0.5), randn(g, G, H, D, scale=D ** -0.5), randn(g, G, H, scale=0.1), randn(g, G, D, H, scale=H ** -0.5)
    bias = torch.randn(G, generator=g, device="cuda") * 0.1
    routing = dict(score="sigmoid", bias=bias, groups=groups, top_groups=groups // 2, group_top=2, weight_scale=2.5)
    layer = moe_layer.MoELayer(gate, w1, b1, w2, k, norm=gain, **routing)
    y, stream, loss, saved = layer.block(x, residual, training=True)
    n, inner = saved
    plain = moe_layer.MoELayer(gate, w1, b1, w2, k, **routing)
    # the norm's 8-bit rows are the quantiser's of fp32 rows, the layer's own of bf16 ones: one rounding more, 2^-8 at most, before
    # the 8 bits' 2^-4; both sides' rows then differ by their own rounding, which the two products carry
    y2, loss2, _ = plain.forward(n.y, training=True)
    assert torch.equal(loss, loss2)
    assert (y.double() - y2.double()).norm() <= (2.0 ** -3 + 2.0 ** -8) * y2.double().norm()
    want = moe_layer.reference(gate, w1, b1, w2, k, n.y, **routing)
    bound = 1.13 * 2.0 ** -3 + 2.0 ** -3 + 2.0 ** -8
    assert (y.double() - want).norm() <= bound * want.norm()
    r = inner[2]
    assert int(r.counts.sum()) == T * k
    # gradients: the layer's own, and behind them the norm's formula in 64 bits
    dy, d_stream, d_loss = randn(g, T, D), randn(g, T, D), torch.full((1,), 3.0, device="cuda")
    dx, d_norm, *d_weights = layer.backward_block(saved, dy, d_stream, d_loss)
    d_normed, *same = layer.backward(inner, dy, d_loss)
    assert all(torch.equal(p, q) for p, q in zip(d_weights, same))
    h = stream.double()
    f = 1.0 / (h.square().mean(1, keepdim=True) + 1e-6).sqrt()
    d = d_normed.double() * gain.double()
    want = f * (d - h * f * (d * h * f).mean(1, keepdim=True)) + d_stream.double()
    assert bool(((dx.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -16 * (d.abs() * f + d_stream.double().abs()).amax(1, keepdim=True)).all())
    want = (d_normed.double() * h * f).sum(0)
    assert bool(((d_norm.double() - want).abs() <= 2.0 ** -16 * (d_normed.double() * h * f).abs().sum(0)).all())


def test_gradient_of_the_gate_in_the_layer():
    """d loss / d logits of the layer's own chain (gate, sigmoid, groups, factor) by autograd in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(23)
    T, G, k, D, H = 150, 16, 3, 128, 256
    x, gate = randn(g, T, D), randn(g, G, D, scale=D ** -0.5)
    routing = dict(score="sigmoid", groups=4, top_groups=2, group_top=2, weight_scale=1.5)
    layer = moe_layer.MoELayer(gate, randn(g, G, H, D, scale=D ** -0.5), randn(g, G, H, scale=0.1), randn(g, G, D, H, scale=H ** -0.5), k, **routing)
    dy = randn(g, T, D)
    _, loss, saved = layer.forward(x, training=True)
    _, logits, r, *_, per_choice = saved[:8]
    d_weights = (per_choice.float() * dy.float()[:, None]).sum(-1)
    d_logits = tg.moe_router_backward(logits, r, d_weights.contiguous(), torch.full((1,), 2.0, device="cuda"))
    z = logits.double().requires_grad_(True)
    s = torch.sigmoid(z)
    w = s.gather(1, r.experts.long())
    w = 1.5 * w / w.sum(1, keepdim=True)
    p = s / s.sum(1, keepdim=True)
    total = (w * d_weights.double()).sum() + 2.0 * G * (r.counts.double() / (T * k) * p.mean(0)).sum()
    (want,) = torch.autograd.grad(total, z)
    # fp32 throughout: a row's sums of 16 numbers and a few factors, of the row's largest part
    size = (d_weights.double().abs().sum(1, keepdim=True) * 1.5 + 2.0 * G / (T * k)).expand_as(want)
    assert bool(((d_logits.double() - want).abs() <= 100 * 2.0 ** -24 * size).all())
