"""64-bit references of the 8-bit expert layer's operators (plain torch on whatever device the inputs are on)."""
from __future__ import annotations

import math

import torch

BLOCK = 128
TOP = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}
SIZE = {"row": (1, BLOCK), "column": (BLOCK, 1), "square": (BLOCK, BLOCK)}


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def quantize(x: torch.Tensor, block, dtype):
    """(q, scale) by the definition, block by block: the smallest power of two s >= 2^-126 with amax <= top * s."""
    M, K = x.shape
    br, bc = block
    q = torch.zeros(M, K, dtype=torch.float64, device=x.device)
    s = torch.empty(-(-M // br), -(-K // bc), dtype=torch.float64, device=x.device)
    xd = x.double()
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            part = xd[i * br:(i + 1) * br, j * bc:(j + 1) * bc]
            amax = float(part.abs().max())
            if not math.isfinite(amax) or bool(torch.isnan(part).any()):
                s[i, j] = float("nan")
                continue
            scale = 1.0
            if amax > 0:
                while amax > TOP[dtype] * scale:
                    scale *= 2.0
                while scale > 2.0 ** -126 and amax <= TOP[dtype] * scale * 0.5:
                    scale *= 0.5
            s[i, j] = scale
            q[i * br:(i + 1) * br, j * bc:(j + 1) * bc] = part / scale
    # the quotients are exact in fp32 unless far below the 8-bit type's smallest value
    return q.float().to(dtype), s.float()


def expand(s: torch.Tensor, shape) -> torch.Tensor:
    """Scales [.., ..] spread over the elements of a matrix of that shape."""
    out = s.double()
    for dim in (0, 1):
        if out.shape[dim] != shape[dim]:
            out = out.repeat_interleave(BLOCK, dim).narrow(dim, 0, shape[dim])
    return out


def gelu(y: torch.Tensor) -> torch.Tensor:
    return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))


def product(a, sa, b, sb, bias=None, epilogue="none"):
    """(C, S, z): the product with its epilogue, sum |a' b'| and the value before the GELU, in 64 bits."""
    x = a.float().double() * expand(sa, a.shape)
    y = b.float().double() * expand(sb, b.shape)
    z = x @ y
    size = x.abs() @ y.abs()
    if epilogue != "none":
        z = z + bias.double()
    return (gelu(z) if epilogue == "bias_gelu" else z), size, z


def product_bound(want, size, z, K, epilogue, dtype):
    """How far an fp32 sum in any order (each of at most K + K / 128 + 4 additions and scalings off by 2^-23 of the
    running magnitude), tanh to 2^-10 absolute and one rounding to dtype may be from the 64-bit value."""
    eps = torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 2.0 ** -24
    pre = (K + blocks(K) + 4) * 2.0 ** -23 * size + 2.0 ** -23 * z.abs()
    if epilogue == "bias_gelu":
        pre = 1.2 * pre + 2.0 ** -10 * 0.5 * z.abs()       # |gelu'| < 1.13
    tiny = torch.finfo(dtype).tiny * 2.0 ** -9               # half a step among fp16's subnormals
    return (pre + eps * (want.abs() + pre)) * 1.001 + max(tiny, 1e-30)


def route(logits: torch.Tensor, k: int, renormalize: bool):
    """(experts, weights, counts, loss, p, rows, chosen) in 64 bits, row by row."""
    x = logits.detach().double()
    T, G = x.shape
    top = x.amax(1, keepdim=True) if T else x.new_zeros(0, 1)
    live = (x > float("-inf")).any(1) | torch.isnan(x).any(1)
    e = torch.exp(x - top)
    p = torch.where(live[:, None], e / e.sum(1, keepdim=True), torch.zeros_like(x))
    experts = torch.full((T, k), -1, dtype=torch.int32)
    xc = x.cpu()
    for t in range(T):
        row = xc[t].tolist()
        order = sorted((g for g in range(G) if row[g] != float("-inf")),
                       key=lambda g: (0 if math.isnan(row[g]) else 1, 0.0 if math.isnan(row[g]) else -row[g], g))
        for j, g in enumerate(order[:k]):
            experts[t, j] = g
    experts = experts.to(x.device)
    chosen = experts >= 0
    w = torch.where(chosen, p.gather(1, experts.clamp(min=0).long()), torch.zeros(T, k, dtype=torch.float64, device=x.device))
    if renormalize:
        w = torch.where(chosen, w / w.sum(1, keepdim=True), w)
    counts = torch.bincount(experts[chosen].long().flatten(), minlength=G).int()
    n = max(1, int(live.sum()))
    loss = G * (counts.double() / (n * k) * p.sum(0) / n).sum()
    return experts, w, counts, loss, p, int(live.sum()), chosen


def route_gradient(logits, experts, counts, k, renormalize, d_weights, d_loss):
    """The gradient of (weights . d_weights + loss * d_loss) by the logits through torch's autograd in 64 bits."""
    x = logits.detach().double().requires_grad_(True)
    T, G = x.shape
    live = (x.detach() > float("-inf")).any(1)
    masked = x.masked_fill(~live[:, None], 0.0)
    p = torch.softmax(masked, 1) * live[:, None]
    chosen = experts >= 0
    w = p.gather(1, experts.clamp(min=0).long()) * chosen
    if renormalize:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(live[:, None], total, torch.ones_like(total))
    n = max(1, int(live.sum()))
    total = x.new_zeros(())
    if d_weights is not None:
        total = total + (w * torch.where(chosen, d_weights.double(), torch.zeros_like(w))).sum()
    if d_loss is not None:
        total = total + float(d_loss) * G * (counts.double() / (n * k) * p.sum(0) / n).sum()
    (d,) = torch.autograd.grad(total, x)
    return torch.where(x.detach() > float("-inf"), d, torch.zeros_like(d))
