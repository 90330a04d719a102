"""A mixture-of-experts feed-forward layer on the 8-bit products: the gate, the experts and their gradients.

    python -m grouped_gemm_persistent_gb300.moe_layer [--tokens T] [--experts G] [--top-k K] [--dim D] [--hidden H]
        [--score sigmoid] [--groups N --top-groups N] [--block]

``MoELayer`` shows how the entry points go together.  Forward: the gate's logits (``gemm``), choice, weights, counts
and balance loss (``moe_router``), the chosen rows grouped by expert and quantised (``quantize_fp8``), and two expert
products (``moe_gemm_fp8``) that read the counts where the router left them.  Backward: the rows' gradients through the
same 8-bit weights, the weights' gradients in blocks along the tokens (``gemm_fp8``), and the gate's logits
(``moe_router_backward``).  Rows are moved by torch indexing.  ``MoELayer.block`` puts a residual stream's norm in front
(``rmsnorm``, whose 8-bit copy is what the experts read).  The command runs one step and prints its times and how far the
8-bit layer is from the same layer in 64 bits.
"""
from __future__ import annotations

import argparse

import torch
import torch.nn.functional as F

from ._binding import (gemm, gemm_fp8, moe_gemm_fp8, moe_router, moe_router_backward, quantize_fp8, rmsnorm,
                       rmsnorm_backward)

GRAD = torch.float8_e5m2      # gradients have the wider range


def quantize_experts(w: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """(q [G, N, K], scale [G, ceil(N / 128), ceil(K / 128)]) of the experts' weights [G, N, K]; K a multiple of 16."""
    parts = [quantize_fp8(e, (128, 128)) for e in w]
    return torch.stack([q for q, _ in parts]), torch.stack([s for _, s in parts])


class MoELayer:
    """y[t] = sum_j weights[t, j] * W2[e] gelu(W1[e] x[t] + b1[e]), e = experts[t, j].

    ``w1`` [G, hidden, dim] and ``w2`` [G, dim, hidden] are quantised once; ``gate`` is [G, dim], ``b1`` [G, hidden],
    all bf16.  dim and hidden are multiples of 16.  ``norm`` (bf16 or fp32 [dim]) is the gain of the norm that ``block``
    puts in front; ``routing`` are moe_router's score, bias, groups, top_groups, group_top and weight_scale.
    """

    def __init__(self, gate: torch.Tensor, w1: torch.Tensor, b1: torch.Tensor, w2: torch.Tensor, top_k: int, *,
                 norm: torch.Tensor | None = None, eps: float = 1e-6, **routing):
        self.gate, self.b1, self.top_k = gate, b1, top_k
        self.norm, self.eps, self.routing = norm, eps, routing
        self.w1, self.s1 = quantize_experts(w1)
        self.w2, self.s2 = quantize_experts(w2)

    def _experts(self, rows, counts, w, s, transposed, **kw):
        """rows (quantised here, or a pair of 8-bit rows and scales) times each expert's w[g]^T, or w[g] when ``transposed``."""
        to = kw.pop("to", torch.float8_e4m3fn)
        q, sq = rows if isinstance(rows, tuple) else quantize_fp8(rows, dtype=to)
        b, sb = (w, s) if transposed else (w.transpose(1, 2), s.transpose(1, 2))
        return moe_gemm_fp8(q, sq, b, sb, counts, **kw)

    def forward(self, x: torch.Tensor, training: bool = False):
        """(y [T, dim] bf16, balance loss, what backward needs or None) for x [T, dim] bf16."""
        return self._forward(x, None, training)

    def block(self, x: torch.Tensor, residual: torch.Tensor, training: bool = False):
        """(y, stream, balance loss, what backward_block needs or None): the layer behind the norm of stream = x + residual.

        y is not added to the stream: the next block's norm does that, with y as its x and the stream as its residual.
        """
        n = rmsnorm(x, self.norm, self.eps, residual=residual, fp8_dtype=torch.float8_e4m3fn)
        y, loss, saved = self._forward(n.y, (n.q, n.scale), training)
        return y, n.hidden, loss, (n, saved) if training else None

    def backward_block(self, saved, dy: torch.Tensor, d_stream: torch.Tensor, d_loss: torch.Tensor):
        """Gradients (x and residual alike, norm, gate, w1, b1, w2) from y's ``dy``, the stream's and the loss's."""
        n, inner = saved
        d_normed, *d_weights = self.backward(inner, dy, d_loss)
        dx, d_norm = rmsnorm_backward(n, d_normed, self.norm, d_stream)
        return dx, d_norm, *d_weights

    def _forward(self, x, in_8_bits, training):
        T, G, k = x.shape[0], self.gate.shape[0], self.top_k
        logits = gemm(x, self.gate.t(), out_dtype=torch.float32)
        r = moe_router(logits, k, renormalize=True, **self.routing)
        # rows in expert order; a choice of no expert (-1) goes last, past the counts
        key = torch.where(r.experts < 0, G, r.experts).flatten()
        order = torch.argsort(key, stable=True)
        rows = x[order // k]
        first = rows
        if in_8_bits is not None:                      # a row's 8-bit copy does not depend on its place
            q, scale = (t[order // k] for t in in_8_bits)
            first = (q, scale)
        if training:
            z = self._experts(first, r.counts, self.w1, self.s1, False, bias=self.b1, epilogue="bias")
            h = F.gelu(z, approximate="tanh")
        else:
            z = None
            h = self._experts(first, r.counts, self.w1, self.s1, False, bias=self.b1, epilogue="bias_gelu")
        o = self._experts(h, r.counts, self.w2, self.s2, False)
        place = torch.empty_like(order)
        place[order] = torch.arange(order.numel(), device=x.device)
        per_choice = torch.where(r.experts[..., None] >= 0, o[place].view(T, k, -1), 0)
        y = (per_choice.float() * r.weights[..., None]).sum(1).to(x.dtype)
        return y, r.loss, (x, logits, r, order, rows, z, h, per_choice) if training else None

    def backward(self, saved, dy: torch.Tensor, d_loss: torch.Tensor):
        """Gradients (x, gate, w1, b1, w2) from y's ``dy`` and the loss's ``d_loss`` (fp32 scalars of one element)."""
        x, logits, r, order, rows, z, h, per_choice = saved
        k = self.top_k
        d_weights = (per_choice.float() * dy.float()[:, None]).sum(-1)
        w = r.weights.flatten()[order]
        d_o = (dy[order // k].float() * w[:, None]).to(dy.dtype)
        d_h = self._experts(d_o, r.counts, self.w2, self.s2, True, to=GRAD)
        with torch.enable_grad():
            leaf = z.detach().requires_grad_(True)
            (d_z,) = torch.autograd.grad(F.gelu(leaf, approximate="tanh"), leaf, d_h)
        d_rows = self._experts(d_z, r.counts, self.w1, self.s1, True, to=GRAD)
        d_logits = moe_router_backward(logits, r, d_weights.contiguous(), d_loss)
        counts = r.counts.tolist()                     # the weights' products need the rows' places on the host
        live = sum(counts)
        dx = torch.zeros_like(x, dtype=torch.float32)
        dx.index_add_(0, order[:live] // k, d_rows[:live].float())
        pad = -self.gate.shape[0] % 8                  # the bf16 products need rows of a multiple of 16 bytes
        dg16 = F.pad(d_logits, (0, pad)).to(x.dtype)
        dx += gemm(dg16, F.pad(self.gate, (0, 0, 0, pad)), out_dtype=torch.float32)
        d_gate = d_logits.t() @ x.float()
        d_w1 = torch.zeros(self.w1.shape, dtype=torch.float32, device=x.device)
        d_w2 = torch.zeros(self.w2.shape, dtype=torch.float32, device=x.device)
        d_b1 = torch.zeros(self.b1.shape, dtype=torch.float32, device=x.device)
        at = 0
        for g, m in enumerate(counts):
            part = slice(at, at + m)
            at += m
            if m:
                _weight_gradient(d_o[part], h[part], d_w2[g])
                _weight_gradient(d_z[part], rows[part], d_w1[g])
                d_b1[g] = d_z[part].float().sum(0)
        return dx.to(x.dtype), d_gate, d_w1, d_b1, d_w2


def _weight_gradient(d_out: torch.Tensor, inp: torch.Tensor, out: torch.Tensor) -> None:
    """out[N, K] = d_out[m, N]^T inp[m, K], both in blocks of 128 along the m tokens."""
    a, sa = quantize_fp8(d_out, (128, 1), dtype=GRAD)
    b, sb = quantize_fp8(inp, (128, 1))
    gemm_fp8(a.t(), sa.t(), b, sb, out)


def choose(logits, top_k, score="softmax", bias=None, groups=1, top_groups=None, group_top=1, weight_scale=1.0):
    """(experts, renormalised weights) of moe_router in 64 bits."""
    p = torch.sigmoid(logits.double()) if score == "sigmoid" else torch.softmax(logits.double(), 1)
    v = p if bias is None else p + bias.double()
    if groups > 1:
        value = v.view(v.shape[0], groups, -1).topk(group_top, 2).values.sum(2)
        kept = torch.zeros_like(value, dtype=torch.bool).scatter_(1, value.topk(top_groups or groups, 1).indices, True)
        v = v.masked_fill(~kept.repeat_interleave(v.shape[1] // groups, 1), float("-inf"))
    e = v.topk(top_k, 1).indices
    w = p.gather(1, e)
    return e, weight_scale * w / w.sum(1, keepdim=True)


def reference(gate, w1, b1, w2, top_k, x, **routing):
    """The layer in 64 bits with the choice of the same logits (rounded as the gate's product rounds them)."""
    logits = gemm(x, gate.t(), out_dtype=torch.float32).double()
    e, w = choose(logits, top_k, **routing)
    y = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    for g in range(gate.shape[0]):
        t, j = torch.nonzero(e == g, as_tuple=True)
        hidden = F.gelu(x[t].double() @ w1[g].double().t() + b1[g].double(), approximate="tanh")
        y.index_add_(0, t, (hidden @ w2[g].double().t()) * w[t, j, None])
    return y


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 4096), ("experts", 16), ("top-k", 4), ("dim", 1024), ("hidden", 1536)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--score", choices=("softmax", "sigmoid"), default="softmax")
    ap.add_argument("--groups", type=int, default=1, help="groups of neighbouring experts")
    ap.add_argument("--top-groups", type=int, help="groups to choose from (default: all)")
    ap.add_argument("--block", action="store_true", help="a residual stream's norm in front")
    a = ap.parse_args()
    gen = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).bfloat16()

    x = randn(a.tokens, a.dim)
    gate = randn(a.experts, a.dim, scale=a.dim ** -0.5)
    w1, w2 = randn(a.experts, a.hidden, a.dim, scale=a.dim ** -0.5), randn(a.experts, a.dim, a.hidden, scale=a.hidden ** -0.5)
    b1 = randn(a.experts, a.hidden, scale=0.1)
    routing = dict(score=a.score, groups=a.groups, top_groups=a.top_groups)
    layer = MoELayer(gate, w1, b1, w2, a.top_k, norm=torch.ones(a.dim, device="cuda") if a.block else None, **routing)
    dy, d_loss = randn(a.tokens, a.dim), torch.ones(1, device="cuda")
    residual = randn(a.tokens, a.dim) if a.block else None

    def forward(training=False):
        return layer.block(x, residual, training) if a.block else layer.forward(x, training)

    def step():
        *_, saved = forward(training=True)
        layer.backward_block(saved, dy, dy, d_loss) if a.block else layer.backward(saved, dy, d_loss)

    def timed(f, n=10):
        for _ in range(3):
            f()
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        for _ in range(n):
            f()
        end.record()
        torch.cuda.synchronize()
        return begin.elapsed_time(end) / n

    y, *_, loss, _ = forward()
    inputs = rmsnorm(x, layer.norm, layer.eps, residual=residual).y if a.block else x
    want = reference(gate, w1, b1, w2, a.top_k, inputs, **routing)
    off = float((y.double() - want).norm() / want.norm())
    print(f"tokens {a.tokens}, experts {a.experts}, top-k {a.top_k}, dim {a.dim}, hidden {a.hidden}")
    print(f"balance loss {float(loss):.4f}, relative distance from 64 bits {off:.4f}")
    print(f"forward {timed(forward):.3f} ms, forward and backward {timed(step):.3f} ms")


if __name__ == "__main__":
    main()
