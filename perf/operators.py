"""Cases of the 8-bit expert layer's operators: what they are given, their plain form and their exact value.

Five operators, used one after the other by a mixture-of-experts layer whose products run in 8-bit floating
point:

* ``router``    top-k choice of experts from the gate's logits, with the per-expert token counts and the balance
                loss; with ``train`` also the gradient of the logits.
* ``quantize``  a matrix to 8-bit floating point with one power-of-two scale for each block of 128 values along a
                row, along a column, or for each 128 x 128 block.
* ``gemm``      the product of two such matrices, scaled back, with the usual epilogues.
* ``moe``       the same product for experts, the rows of each given by counts that stay on the GPU.

With ``own`` false, ``run`` computes them with elementary torch operations; with ``own`` true through the library.
"""
import math

import torch

own = False

BLOCK = 128
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16,
         "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}       # largest finite value


def _blocks(n):
    return -(-n // BLOCK)


# ------------------------------------------------------------------------------------------------- the cases


def listed():
    return [
        # one decoding step of a small batch: only the latency counts
        dict(name="router_step", op="router", T=64, G=64, k=8, type="f32", renorm=True, padded=0.0, banned=0.0,
             train=False),
        # a packed prompt with padding rows and experts that some rows may not take
        dict(name="router_prompt", op="router", T=8191, G=190, k=6, type="f16", renorm=True, padded=0.1, banned=0.2,
             train=False),
        # the gate of the 64-expert layer over 65536 tokens, forward and backward
        dict(name="router_train", op="router", T=65536, G=64, k=4, type="bf16", renorm=False, padded=0.0, banned=0.0,
             train=True),
        # a wide gate over a long batch, forward and backward
        dict(name="router_train_wide", op="router", T=131072, G=256, k=8, type="f32", renorm=True, padded=0.02,
             banned=0.0, train=True),
        # activations of 65536 tokens on their way into an expert product
        dict(name="quantize_rows", op="quantize", M=65536, K=4096, type="bf16", block="row", to="e4m3"),
        # gradients for a weight's gradient: blocks along the tokens, an odd number of them
        dict(name="quantize_columns", op="quantize", M=8191, K=1544, type="bf16", block="column", to="e5m2"),
        # a weight held in 32 bits, laid out once per update
        dict(name="quantize_weight", op="quantize", M=4096, K=4096, type="f32", block="square", to="e4m3"),
        # one token through one projection
        dict(name="gemm_token", op="gemm", M=1, N=4096, K=4096, a="row", b="col", at="e4m3", bt="e4m3", sb="square",
             pow2=False, out="bf16", epi="bias"),
        # a weight's gradient: both operands read across their rows, blocks along 5000 tokens
        dict(name="gemm_weight_gradient", op="gemm", M=1536, N=4096, K=5000, a="col", b="row", at="e5m2", bt="e4m3",
             sb="column", pow2=True, out="f32", epi="none"),
        # the large dense product
        dict(name="gemm_large", op="gemm", M=8192, N=8192, K=8192, a="row", b="col", at="e4m3", bt="e4m3",
             sb="square", pow2=False, out="bf16", epi="none"),
        # 64 experts in a decoding step: a few rows each, many of them none
        dict(name="moe_step", op="moe", T=256, G=64, K=1536, N=4096, b="col", at="e4m3", skew=0.5, pow2=True,
             out="bf16", epi="none"),
        # 64 experts over 65536 tokens, split unevenly
        dict(name="moe_train", op="moe", T=65536, G=64, K=4096, N=1536, b="col", at="e4m3", skew=0.5, pow2=True,
             out="bf16", epi="none"),
    ]


def _spread(rng, lo, hi, step=1):
    """A whole number in [lo, hi], spread over its logarithm; about half of them multiples of 128 or odd ones."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    v = min(hi, max(lo, int(v)))
    kind = rng.randrange(4)
    if kind == 0 and v > BLOCK:
        v = v // BLOCK * BLOCK
    elif kind == 1 and step == 1 and v > 2:
        v -= 1 - v % 2
    return max(lo, v // step * step)


def draw(rng):
    op = rng.choice(("router", "quantize", "gemm", "moe"))
    if op == "router":
        G = rng.randrange(8, 257)
        k = rng.randrange(1, 9)
        T = _spread(rng, 1, 131072 * 256 // max(G, 64))
        T = min(T, 131072)
        return dict(op=op, T=T, G=G, k=k, type=rng.choice(("f32", "bf16", "f16")), renorm=rng.random() < 0.5,
                    padded=rng.choice((0.0, 0.1)), banned=rng.choice((0.0, 0.2)), train=rng.random() < 0.5)
    if op == "quantize":
        M, K = _spread(rng, 1, 65536), _spread(rng, 128, 8192)
        t = rng.choice(("f32", "bf16", "f16"))
        while M * K > 65536 * (2048 if t == "f32" else 4096):
            M = max(1, M // 2)
        return dict(op=op, M=M, K=K, type=t, block=rng.choice(("row", "column", "square")),
                    to=rng.choice(("e4m3", "e5m2")))
    if op == "gemm":
        M, N, K = _spread(rng, 1, 8192), _spread(rng, 64, 8192), _spread(rng, 128, 8192)
        return dict(op=op, M=M, N=N, K=K, a=rng.choice(("row", "row", "col")), b=rng.choice(("col", "col", "row")),
                    at=rng.choice(("e4m3", "e4m3", "e5m2")), bt="e4m3",
                    sb=rng.choice(("square", "square", "column")), pow2=rng.random() < 0.5,
                    out=rng.choice(("bf16", "f32", "f16")), epi=rng.choice(("none", "bias", "bias_gelu")))
    G = rng.choice((8, 16, 31, 64, 128))
    T = _spread(rng, 1, 32768)
    K, N = _spread(rng, 256, 4096, 16), _spread(rng, 256, 4096, 16)
    return dict(op=op, T=T, G=G, K=K, N=N, b=rng.choice(("col", "col", "row")),
                at=rng.choice(("e4m3", "e4m3", "e5m2")), skew=rng.choice((0.3, 0.5, 10.0)), pow2=rng.random() < 0.5,
                out=rng.choice(("bf16", "f32", "f16")), epi=rng.choice(("none", "bias", "bias_gelu")))


# ------------------------------------------------------------------------------------------------- the inputs


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, rows, cols):
    """Normal values whose columns differ in size, a few of them much larger: what a layer's input looks like."""
    x = _randn(g, rows, cols)
    size = torch.exp(0.5 * _randn(g, cols))
    size[torch.rand(cols, generator=g, device="cuda") < 0.01] *= 20.0
    return x.mul_(size)


def _row_padded(rows, cols, dtype, to):
    """An uninitialised [rows, cols] matrix whose row length in memory is a multiple of `to` elements."""
    return torch.empty(rows, -(-cols // to) * to, dtype=dtype, device="cuda")[:, :cols]


def _tile(x, rows, cols):
    """x [M, K], zero-padded, as [M / rows, rows, K / cols, cols]."""
    M, K = x.shape
    pad = (0, -K % cols, 0, -M % rows)
    if any(pad):
        x = torch.nn.functional.pad(x, pad)
    return x.view(x.shape[0] // rows, rows, x.shape[1] // cols, cols)


def _pow2_scale(amax, top):
    """The smallest power of two s, at least 2^-126, with amax <= top * s; 1 for a block of zeros."""
    m, e = torch.frexp(amax.double() / top)             # amax / top = m 2^e with m in [1/2, 1), exact enough:
    e = torch.where(m == 0.5, e - 1, e)                 # top is 7 * 2^j, so the quotient rounds onto no power of two
    s = torch.ldexp(torch.ones_like(m), e.clamp(min=-126))
    return torch.where(amax > 0, s, torch.ones_like(s)).float()


def _quantize(x, rows, cols, to, pow2=True):
    """Values of `to` as 32-bit floats in x's shape, and the blocks' scales [M / rows, K / cols]."""
    t = _tile(x.float(), rows, cols)
    amax = t.abs().amax(dim=(1, 3), keepdim=True)
    s = _pow2_scale(amax, TOP[to]) if pow2 else torch.where(amax > 0, amax / TOP[to], torch.ones_like(amax))
    q = (t / s).clamp(-TOP[to], TOP[to])
    bad = ~torch.isfinite(amax)
    s = torch.where(bad, torch.full_like(s, float("nan")), s)
    q = torch.where(bad, torch.zeros_like(q), q)
    M, K = x.shape
    q = q.to(TYPES[to]).float().view(t.shape[0] * rows, t.shape[2] * cols)[:M, :K]
    return q, s[:, 0, :, 0]


def _operand(g, rows, cols, to, br, bc, pow2, weight):
    """An 8-bit matrix in rows of a multiple of 16 bytes, and its scales."""
    x = _randn(g, rows, cols).mul_(0.02) if weight else _activations(g, rows, cols)
    q, s = _quantize(x, br, bc, to, pow2)
    out = _row_padded(rows, cols, TYPES[to], 16)
    out.copy_(q.to(TYPES[to]))
    return out, s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    state = {"case": case}
    if op == "router":
        T, G = case["T"], case["G"]
        x = _randn(g, T, G).mul_(1.5) + 0.5 * _randn(g, G)           # some experts are liked more than others
        if case["banned"]:
            x[torch.rand(T, G, generator=g, device="cuda") < case["banned"]] = float("-inf")
        if case["padded"]:
            x[torch.rand(T, generator=g, device="cuda") < case["padded"]] = float("-inf")
        state["logits"] = x.to(TYPES[case["type"]])
        if case["train"]:
            state["d_weights"] = _randn(g, T, case["k"]).mul_(0.1)
            state["d_loss"] = torch.full((), 0.01 * T, device="cuda")
    elif op == "quantize":
        x = _activations(g, case["M"], case["K"])
        state["x"] = _row_padded(case["M"], case["K"], TYPES[case["type"]], 8)
        state["x"].copy_(x)
    elif op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        if case["a"] == "row":
            state["a"], state["scale_a"] = _operand(g, M, K, case["at"], 1, BLOCK, case["pow2"], False)
            state["scale_a"] = state["scale_a"].t().contiguous().t()
        else:
            a, s = _operand(g, K, M, case["at"], BLOCK, 1, case["pow2"], False)
            state["a"], state["scale_a"] = a.t(), s.t()
        r, c = (BLOCK, BLOCK) if case["sb"] == "square" else ((1, BLOCK) if case["b"] == "col" else (BLOCK, 1))
        if case["b"] == "col":
            b, s = _operand(g, N, K, case["bt"], r, c, case["pow2"], case["sb"] == "square")
            state["b"], state["scale_b"] = b.t(), s.t()
        else:
            state["b"], state["scale_b"] = _operand(g, K, N, case["bt"], r, c, case["pow2"], case["sb"] == "square")
        state["bias"] = _randn(g, N).mul_(0.1).bfloat16() if case["epi"] != "none" else None
    else:
        T, G, K, N = case["T"], case["G"], case["K"], case["N"]
        share = torch.rand(G, generator=g, device="cuda").clamp(min=1e-6) ** (1.0 / case["skew"])
        pick = torch.multinomial(share, T, replacement=True, generator=g)
        state["counts"] = torch.bincount(pick, minlength=G).int()
        state["rows"] = state["counts"].tolist()                     # for the plain form's loop
        state["a"], s = _operand(g, T, K, case["at"], 1, BLOCK, case["pow2"], False)
        state["scale_a"] = s.t().contiguous().t()
        rows, cols = (N, K) if case["b"] == "col" else (K, N)
        bs, ss = [], []
        for _ in range(G):
            b, s = _operand(g, rows, cols, "e4m3", BLOCK, BLOCK, case["pow2"], True)
            bs.append(b)
            ss.append(s)
        state["b"], state["scale_b"] = torch.stack(bs), torch.stack(ss)
        if case["b"] == "col":
            state["b"], state["scale_b"] = state["b"].transpose(1, 2), state["scale_b"].transpose(1, 2)
        state["bias"] = _randn(g, G, N).mul_(0.1).bfloat16() if case["epi"] != "none" else None
    return state


# ------------------------------------------------------------------------------------------------- one pass


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    import grouped_gemm_persistent_gb300 as tg
    case = state["case"]
    op = case["op"]
    if op == "router":
        r = tg.moe_router(state["logits"], case["k"], renormalize=case["renorm"])
        out = [r.experts, r.weights, r.counts, r.loss]
        if case["train"]:
            out.append(tg.moe_router_backward(state["logits"], r, state["d_weights"], state["d_loss"]))
        return out
    if op == "quantize":
        block = {"row": (1, BLOCK), "column": (BLOCK, 1), "square": (BLOCK, BLOCK)}[case["block"]]
        return list(tg.quantize_fp8(state["x"], block, dtype=TYPES[case["to"]]))
    kw = dict(bias=state["bias"], epilogue=case["epi"], out_dtype=TYPES[case["out"]])
    if op == "gemm":
        return tg.gemm_fp8(state["a"], state["scale_a"], state["b"], state["scale_b"], **kw)
    return tg.moe_gemm_fp8(state["a"], state["scale_a"], state["b"], state["scale_b"], state["counts"], **kw)


def _run_plain(state):
    case = state["case"]
    op = case["op"]
    if op == "router":
        return _router_plain(state)
    if op == "quantize":
        r, c = {"row": (1, BLOCK), "column": (BLOCK, 1), "square": (BLOCK, BLOCK)}[case["block"]]
        q, s = _quantize(state["x"], r, c, case["to"])
        return [q.to(TYPES[case["to"]]), s]
    out = TYPES[case["out"]]
    if op == "gemm":
        return _product_plain(state["a"], state["scale_a"], state["b"], state["scale_b"], state["bias"], case["epi"],
                              out)
    y = torch.empty(case["T"], case["N"], dtype=out, device="cuda")
    r = 0
    for i, m in enumerate(state["rows"]):
        if m:
            y[r:r + m] = _product_plain(state["a"][r:r + m], state["scale_a"][r:r + m], state["b"][i],
                                        state["scale_b"][i], None if state["bias"] is None else state["bias"][i],
                                        case["epi"], out)
        r += m
    return y


def _product_plain(a, sa, b, sb, bias, epi, out):
    K, N = b.shape
    x = a.float() * sa.repeat_interleave(BLOCK, 1)[:, :K]
    s = sb.repeat_interleave(BLOCK, 0)[:K]
    if s.shape[1] != N:
        s = s.repeat_interleave(BLOCK, 1)[:, :N]
    y = x @ (b.float() * s)
    if epi != "none":
        y = y + bias.float()
    if epi == "bias_gelu":
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    return y.to(out)


def _router_plain(state):
    case = state["case"]
    G, k = case["G"], case["k"]
    x = state["logits"].float()
    top = x.amax(1, keepdim=True)
    valid = top > float("-inf")
    e = torch.where(valid, (x - top).exp(), torch.zeros_like(x))
    p = torch.where(valid, e / e.sum(1, keepdim=True), torch.zeros_like(x))
    order = torch.sort(x, dim=1, descending=True, stable=True)
    taken = order.values[:, :k] > float("-inf")
    idx = order.indices[:, :k]
    experts = torch.where(taken, idx, torch.full_like(idx, -1)).int()
    w = torch.where(taken, p.gather(1, idx), torch.zeros_like(p[:, :k]))
    total = w.sum(1, keepdim=True)
    if case["renorm"]:
        w = torch.where(taken, w / total, torch.zeros_like(w))
    counts = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    slot = torch.where(taken, idx, torch.full_like(idx, G)).flatten()
    counts.index_add_(0, slot, torch.ones_like(slot, dtype=torch.int32))
    counts = counts[:G]
    rows = valid.sum().clamp(min=1).double()
    slope = G * counts.double() / (rows * k) / rows              # the loss's derivative by each probability
    loss = (slope * p.sum(0, dtype=torch.float64)).sum().float()
    out = [experts, w, counts, loss]
    if case["train"]:
        dw = torch.where(taken, state["d_weights"], torch.zeros_like(w))
        if case["renorm"]:
            dw = torch.where(taken, (dw - (dw * w).sum(1, keepdim=True)) / total, torch.zeros_like(dw))
        dp = (slope.float() * state["d_loss"]).expand_as(p).contiguous()
        dp.scatter_add_(1, idx, dw)
        d = p * (dp - (p * dp).sum(1, keepdim=True))
        out.append(d.to(state["logits"].dtype))
    return out


# ------------------------------------------------------------------------------------------------- 64 bits


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "router":
        return _router_exact(state)
    if op == "quantize":
        return _quantize_exact(state)
    if op == "gemm":
        return _product_exact(state["a"], state["scale_a"], state["b"], state["scale_b"], state["bias"], case["epi"])
    y = torch.zeros(case["T"], case["N"], dtype=torch.float64, device="cuda")
    ends = torch.cumsum(state["counts"], 0).tolist()
    for i, end in enumerate(ends):
        begin = ends[i - 1] if i else 0
        if end > begin:
            y[begin:end] = _product_exact(state["a"][begin:end], state["scale_a"][begin:end], state["b"][i],
                                          state["scale_b"][i],
                                          state["bias"][i] if state["bias"] is not None else None, case["epi"])
    return y


def _product_exact(a, sa, b, sb, bias, epi):
    K, N = b.shape
    per_column = sb.shape[1] == N
    y = torch.zeros(a.shape[0], N, dtype=torch.float64, device="cuda")
    for j in range(_blocks(K)):
        part = a[:, j * BLOCK:(j + 1) * BLOCK].to(torch.float64) @ b[j * BLOCK:(j + 1) * BLOCK].to(torch.float64)
        col = sb[j].double() if per_column else sb[j].double()[torch.arange(N, device="cuda") // BLOCK]
        y += part * sa[:, j, None].double() * col
    if epi != "none":
        y += bias.double()
    if epi == "bias_gelu":
        u = (2 / math.pi) ** 0.5 * (y + 0.044715 * y ** 3)
        y = y * (0.5 + 0.5 * torch.tanh(u))
    return y


def _quantize_exact(state):
    """Scales found by trying powers of two against the definition; the values rounded on the type's own grid."""
    case = state["case"]
    r, c = {"row": (1, BLOCK), "column": (BLOCK, 1), "square": (BLOCK, BLOCK)}[case["block"]]
    bits, low = (3, -6) if case["to"] == "e4m3" else (2, -14)    # mantissa bits, exponent of the smallest normal
    t = _tile(state["x"].double(), r, c)
    big = t.abs().amax(dim=(1, 3), keepdim=True)
    e = torch.floor(torch.log2(torch.where(big > 0, big, torch.ones_like(big)))) - math.floor(math.log2(TOP[case["to"]])) - 1
    for _ in range(3):
        e = torch.where(big > TOP[case["to"]] * torch.exp2(e), e + 1, e)
    s = torch.where(big > 0, torch.exp2(e.clamp(min=-126)), torch.ones_like(e))
    v = t / s
    _, ev = torch.frexp(v)
    step = torch.exp2((ev.double() - 1).clamp(min=low) - bits)
    q = torch.round(v / step) * step                             # ties to even multiples of the step
    M, K = state["x"].shape
    return [q.view(t.shape[0] * r, t.shape[2] * c)[:M, :K], s[:, 0, :, 0]]


def _router_exact(state):
    case = state["case"]
    T, G, k = case["T"], case["G"], case["k"]
    x = state["logits"].double()
    lse = torch.logsumexp(x, 1)
    live = lse > float("-inf")
    p = torch.exp(x - torch.where(live, lse, torch.zeros_like(lse))[:, None])
    left = x.clone()
    experts = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    w = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    chosen = torch.zeros(T, G, dtype=torch.bool, device="cuda")
    lane = torch.arange(G, device="cuda").expand(T, G)
    for j in range(min(k, G)):
        best = left.amax(1, keepdim=True)
        i = torch.where(left == best, lane, torch.full_like(lane, G)).amin(1)      # ties: the lowest index
        ok = best[:, 0] > float("-inf")
        experts[:, j] = torch.where(ok, i, torch.full_like(i, -1)).int()
        w[:, j] = torch.where(ok, p.gather(1, i[:, None])[:, 0], torch.zeros_like(lse))
        left.scatter_(1, i[:, None], float("-inf"))
        chosen |= (lane == i[:, None]) & ok[:, None]
    counts = chosen.sum(0)
    n = max(1, int(live.sum()))
    loss = G * (counts.double() / (n * k) * (p.sum(0) / n)).sum()
    total = w.sum(1, keepdim=True)
    safe = torch.where(total > 0, total, torch.ones_like(total))
    out = [experts, w / safe if case["renorm"] else w, counts.int(), loss]
    if case["train"]:
        dl = float(state["d_loss"])
        ok = experts >= 0
        dw = state["d_weights"].double() * ok
        if case["renorm"]:
            dw = (dw - (dw * w / safe).sum(1, keepdim=True)) / safe * ok
        dp = torch.zeros(T, G, dtype=torch.float64, device="cuda")
        dp.scatter_add_(1, experts.clamp(min=0).long(), dw)
        dp += dl * G * counts.double() / (n * k) / n
        out.append(p * (dp - (p * dp).sum(1, keepdim=True)))
    return out


# ------------------------------------------------------------------------------------------------- the work


SIZE = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1, "e5m2": 1}


def work(case):
    op = case["op"]
    if op == "router":
        T, G, k = case["T"], case["G"], case["k"]
        logits = T * G * SIZE[case["type"]]
        out = T * k * 8 + G * 4 + 4
        if not case["train"]:
            return {"bytes": logits + out, "flops": 5 * T * G}
        return {"bytes": 2 * logits + out + T * k * 4 + 4, "flops": 10 * T * G}
    if op == "quantize":
        M, K = case["M"], case["K"]
        blocks = {"row": M * _blocks(K), "column": _blocks(M) * K, "square": _blocks(M) * _blocks(K)}[case["block"]]
        return {"bytes": M * K * (SIZE[case["type"]] + 1) + 4 * blocks, "flops": 3 * M * K}
    K, N = case["K"], case["N"]
    kb, nb = _blocks(K), _blocks(N)
    if op == "gemm":
        M = case["M"]
        scales = 4 * kb * (M + (nb if case["sb"] == "square" else N))
        return {"bytes": M * K + K * N + scales + M * N * SIZE[case["out"]] + (2 * N if case["epi"] != "none" else 0),
                "flops": 2 * M * N * K}
    T, G = case["T"], case["G"]
    used = min(G, T)                                             # experts that can have rows at all
    return {"bytes": T * K + used * K * N + 4 * kb * (T + used * nb) + T * N * SIZE[case["out"]]
            + (2 * used * N if case["epi"] != "none" else 0), "flops": 2 * T * N * K}
