"""The example layer's backward pass against the same layer in 64 bits on the same 8-bit operands (GPU).

What the 8 bits themselves cost is left out, so that the bound is that of the 16-bit roundings alone and a term with a
wrong factor does not fit under it."""
import math

import pytest
import torch

import fp8_reference as ref
import grouped_gemm_persistent_gb300 as tg
from grouped_gemm_persistent_gb300 import moe_layer

pytestmark = pytest.mark.gpu

E5 = torch.float8_e5m2


def wide(q, s):
    return q.float().double() * ref.expand(s, q.shape)


def in_8_bits(x, block=(1, 128), dtype=torch.float8_e4m3fn):
    """x as its 8-bit copy holds it (the quantiser itself is tested against its definition elsewhere)."""
    return wide(*tg.quantize_fp8(x, block, dtype=dtype))


def gelu_slope(z):
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


@pytest.mark.parametrize("dy_scale,d_loss", [(1.0, 1.0), (1.0, 3000.0), (0.0, 1.0)])
@pytest.mark.parametrize("T,G,k,D,H", [(200, 8, 2, 256, 384), (513, 16, 4, 144, 272)])
def test_backward(T, G, k, D, H, dy_scale, d_loss):
    g = torch.Generator(device="cuda").manual_seed(17)

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()

    x, gate = randn(T, D), randn(G, D, scale=D ** -0.5)
    layer = moe_layer.MoELayer(gate, randn(G, H, D, scale=D ** -0.5), randn(G, H, scale=0.1),
                               randn(G, D, H, scale=H ** -0.5), k)
    dy = (randn(T, D).float() * dy_scale).bfloat16()
    y, loss, saved = layer.forward(x, training=True)
    _, logits, r, order, rows, z, h, per_choice = saved[:8]
    dx, d_gate, d_w1, d_b1, d_w2 = layer.backward(saved, dy, torch.full((1,), d_loss, device="cuda"))

    # 64 bits from here on; what the layer holds in bf16 (d_o, d_h, d_z) is rounded to it, and quantised from there
    w1 = torch.stack([wide(layer.w1[e], layer.s1[e]) for e in range(G)])
    w2 = torch.stack([wide(layer.w2[e], layer.s2[e]) for e in range(G)])
    weights = r.weights.double().flatten()[order]
    expert = r.experts.flatten()[order].long()
    token = order // k
    d_o = (dy.double()[token] * weights[:, None]).bfloat16()
    ends = torch.cumsum(r.counts, 0).tolist()
    parts = [slice(e - c, e) for e, c in zip(ends, r.counts.tolist())]

    def through(rows8, w):
        return torch.cat([rows8[p] @ w[e] for e, p in enumerate(parts)])

    d_h = through(in_8_bits(d_o, dtype=E5), w2).bfloat16()
    d_z = (d_h.double() * gelu_slope(z.double())).bfloat16()
    d_rows = through(in_8_bits(d_z, dtype=E5), w1)
    want_x = torch.zeros(T, D, dtype=torch.float64, device="cuda").index_add_(0, token, d_rows)
    p = torch.softmax(logits.double(), 1)
    w = p.gather(1, r.experts.long())
    d_weights = (per_choice.double() * dy.double()[:, None]).sum(-1)
    total = w.sum(1, keepdim=True)
    d_chosen = (d_weights - (d_weights * w).sum(1, keepdim=True) / total) / total
    d_p = (d_loss * G * r.counts.double() / (T * k) / T).expand(T, G).scatter_add(1, r.experts.long(), d_chosen)
    d_logits = p * (d_p - (p * d_p).sum(1, keepdim=True))
    want_x += d_logits @ gate.double()
    want = {"x": want_x, "gate": d_logits.t() @ x.double(), "w1": [], "b1": [], "w2": []}
    for e, part in enumerate(parts):
        if part.start == part.stop:
            for name, shape in (("w1", (H, D)), ("b1", (H,)), ("w2", (D, H))):
                want[name].append(torch.zeros(shape, dtype=torch.float64, device="cuda"))
            continue
        want["w2"].append(in_8_bits(d_o[part], (128, 1), E5).t() @ in_8_bits(h[part], (128, 1)))
        want["w1"].append(in_8_bits(d_z[part], (128, 1), E5).t() @ in_8_bits(rows[part], (128, 1)))
        want["b1"].append(d_z[part].double().sum(0))
    for name, got in (("x", dx), ("gate", d_gate), ("w1", d_w1), ("b1", d_b1), ("w2", d_w2)):
        value = want[name] if isinstance(want[name], torch.Tensor) else torch.stack(want[name])
        if dy_scale == 0.0 and name in ("w1", "b1", "w2"):
            assert not got.any()
            continue
        # dx rounds its logits' part and itself to bf16, 2^-9 each in the 2-norm (half a step is at most 2^-8 of a
        # value, its root mean square at most half of that).  bf16 values that fall the other way for an fp32 sum's last
        # bits (one in 2^12) move by 2^-8, and to another of the 8-bit values one in 2^6 of those, by a quarter: 2^-11.
        rel = float((got.double() - value).norm() / value.norm())
        assert rel <= (2 * 2.0 ** -9 if name == "x" else 0.0) + 2.0 ** -10, f"{name}: {rel}"
    live = r.experts >= 0
    assert bool(live.all())
