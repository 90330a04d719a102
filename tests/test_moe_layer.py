"""The example layer: forward and backward through the 8-bit products, against the same layer in 64 bits (GPU)."""
import pytest
import torch
import torch.nn.functional as F

from grouped_gemm_persistent_gb300 import moe_layer
from grouped_gemm_persistent_gb300.build import build

pytestmark = pytest.mark.gpu


def make(T, G, k, D, H):
    g = torch.Generator(device="cuda").manual_seed(3)

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()

    return (randn(T, D), randn(G, D, scale=D ** -0.5), randn(G, H, D, scale=D ** -0.5), randn(G, H, scale=0.1),
            randn(G, D, H, scale=H ** -0.5), randn(T, D))


@pytest.mark.parametrize("T,G,k,D,H", [(200, 8, 2, 256, 384), (1, 4, 2, 128, 256), (513, 16, 4, 144, 272)])
def test_layer(T, G, k, D, H):
    build()
    x, gate, w1, b1, w2, dy = make(T, G, k, D, H)
    layer = moe_layer.MoELayer(gate, w1, b1, w2, k)
    y, loss, _ = layer.forward(x)
    want = moe_layer.reference(gate, w1, b1, w2, k, x)
    # Two products in a row with operands rounded to 3 mantissa bits: an element is off by at most 2^-4 of itself, so
    # a product of rounded factors by 2^-3, independently of its neighbours, which leaves the sums' 2-norm within it;
    # the hidden rows carry theirs (times gelu's slope of at most 1.13) into the second product.
    bound = 1.13 * 2.0 ** -3 + 2.0 ** -3
    assert (y.double() - want).norm() <= bound * want.norm()
    yt, loss_t, saved = layer.forward(x, training=True)
    assert torch.equal(loss, loss_t) and (yt.double() - want).norm() <= bound * want.norm()

    # gradients of <y, dy> + loss by autograd in 64 bits, the choice and the counts held fixed
    xd, gd, w1d, b1d, w2d = (t.double().requires_grad_(True) for t in (x, gate, w1, b1, w2))
    r = saved[2]
    p = torch.softmax(xd @ gd.t(), 1)
    w = p.gather(1, r.experts.long())
    w = w / w.sum(1, keepdim=True)
    total = G * (r.counts.double() / (T * k) * p.mean(0)).sum()
    for e in range(G):
        t, j = torch.nonzero(r.experts == e, as_tuple=True)
        hidden = F.gelu(xd[t] @ w1d[e].t() + b1d[e], approximate="tanh")
        total = total + (((hidden @ w2d[e].t()) * w[t, j, None]) * dy[t].double()).sum()
    wants = torch.autograd.grad(total, (xd, gd, w1d, b1d, w2d))
    gots = layer.backward(saved, dy, torch.ones(1, device="cuda"))
    # backward rounds gradients to 2 mantissa bits (2^-3 each) on top, up to twice in a row, and the gate's logits
    # see the products' errors through d_weights
    for name, got, want in zip(("x", "gate", "w1", "b1", "w2"), gots, wants):
        rel = float((got.double() - want).norm() / want.norm())
        assert rel <= bound + 2 * (2.0 ** -3 + 2.0 ** -4), f"{name}: {rel}"


def test_rows_without_an_expert(monkeypatch):
    build()
    x, gate, w1, b1, w2, dy = make(64, 8, 2, 128, 256)
    layer = moe_layer.MoELayer(gate, w1, b1, w2, 2)
    whole, _, _ = layer.forward(x)
    plain = moe_layer.gemm

    def padded(a, b, **kw):
        out = plain(a, b, **kw)
        if out.shape == (64, 8):
            out[::3] = float("-inf")             # padding rows choose nothing
        return out

    monkeypatch.setattr(moe_layer, "gemm", padded)
    y, loss, saved = layer.forward(x, training=True)
    assert (y[::3] == 0).all() and int(saved[2].counts.sum()) == 2 * (64 - 22)
    keep = torch.arange(64, device="cuda") % 3 != 0
    rel = float((y[keep].double() - whole[keep].double()).norm() / whole[keep].double().norm())
    assert rel <= 2.0 ** -8 + 2.0 ** -4          # the same rows; one path rounds before the gelu, the other after
    monkeypatch.setattr(moe_layer, "gemm", plain)
    dx = layer.backward(saved, dy, torch.ones(1, device="cuda"))[0]
    assert torch.isfinite(dx.float()).all() and (dx[::3] == 0).all()
