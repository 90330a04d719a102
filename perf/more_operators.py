"""Cases of the operators between and beside the products of a mixture-of-experts block: what they are given, their
plain form and their exact value.

* ``norm``    RMS norm of a residual stream: the addition of a block's output, the normalised rows with a gain, in 16
              or 32 bits and / or in 8 bits with a power-of-two scale for each 128 values of a row; with ``train`` also
              the gradients.
* ``router``  the gate's choice of experts from sigmoid or softmax scores, with a bias for balance, groups of experts
              of which only some are looked at, and weights with a factor; with ``train`` also the logits' gradient.
* ``lora``    low-rank adapters of many requests, added to what a shared projection gave.

With ``own`` false, ``run`` computes them with elementary torch operations; with ``own`` true through the library.
"""
import math

import torch

own = False

BLOCK = 128
EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16,
         "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}       # largest finite value
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1, "e5m2": 1, "none": 0}
INF = float("inf")


def _blocks(n):
    return -(-n // BLOCK)


# ------------------------------------------------------------------------------------------------- the cases


def listed():
    return [
        # one decoding step of 64 requests, in front of an 8-bit projection with adapters beside it
        dict(name="norm_step", op="norm", M=64, K=4096, x="bf16", residual="bf16", gain="bf16", out="bf16", q="e4m3",
             train=False),
        # a packed prompt of odd sizes, the residual stream held in 32 bits
        dict(name="norm_prompt", op="norm", M=8191, K=1544, x="bf16", residual="f32", gain="f32", out="bf16",
             q="none", train=False),
        # 65536 tokens on their way into an 8-bit product
        dict(name="norm_quantize", op="norm", M=65536, K=4096, x="bf16", residual="bf16", gain="bf16", out="none",
             q="e4m3", train=False),
        # a training step over 65536 tokens, forward and backward
        dict(name="norm_train", op="norm", M=65536, K=4096, x="bf16", residual="bf16", gain="f32", out="bf16",
             q="none", train=True),
        # one decoding step: 256 experts in 8 groups, 4 of them looked at
        dict(name="router_step", op="router", T=64, G=256, k=8, type="f32", score="sigmoid", bias=True, groups=8,
             top_groups=4, group_top=2, renorm=True, scale=2.5, padded=0.0, train=False),
        # a packed prompt with padding rows; 190 experts in 10 groups, softmax without a bias
        dict(name="router_prompt", op="router", T=8191, G=190, k=6, type="f16", score="softmax", bias=False, groups=10,
             top_groups=3, group_top=1, renorm=False, scale=16.0, padded=0.1, train=False),
        # the gate of the 64-expert layer over 65536 tokens, no groups, forward and backward
        dict(name="router_train", op="router", T=65536, G=64, k=4, type="bf16", score="sigmoid", bias=True, groups=1,
             top_groups=1, group_top=1, renorm=True, scale=1.0, padded=0.0, train=True),
        # a wide gate in groups over a long batch, forward and backward
        dict(name="router_train_wide", op="router", T=131072, G=256, k=8, type="f32", score="sigmoid", bias=True,
             groups=8, top_groups=4, group_top=2, renorm=True, scale=2.5, padded=0.02, train=True),
        # one token of one request
        dict(name="lora_token", op="lora", T=1, K=4096, N=4096, r=16, G=8, type="bf16", base="bf16", requests=1,
             idle=0.0, scaled=True),
        # one decoding step: 64 requests with an adapter each
        dict(name="lora_step", op="lora", T=64, K=4096, N=4096, r=16, G=64, type="bf16", base="bf16", requests=64,
             idle=0.1, scaled=True),
        # packed prompts of 30 requests with large adapters
        dict(name="lora_prompts", op="lora", T=8191, K=4096, N=1536, r=64, G=16, type="bf16", base="bf16", requests=30,
             idle=0.1, scaled=True),
        # a long batch, the projection's result in 32 bits
        dict(name="lora_batch", op="lora", T=32768, K=1536, N=4096, r=32, G=8, type="f16", base="f32", requests=100,
             idle=0.0, scaled=False),
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
    op = rng.choice(("norm", "router", "lora"))
    if op == "norm":
        M, K = _spread(rng, 1, 65536), _spread(rng, 128, 8192)
        x = rng.choice(("bf16", "bf16", "f16", "f32"))
        train = rng.random() < 0.5
        out, q = rng.choice(((x, "none"), (x, "e4m3"), ("none", "e4m3"), ("none", "e5m2")))
        while M * K > 65536 * (1024 if x == "f32" else 2048):
            M = max(1, M // 2)
        return dict(op=op, M=M, K=K, x=x, residual=rng.choice(("none", x, x, "f32")),
                    gain=rng.choice(("none", "f32", x)), out=out, q=q, train=train)
    if op == "router":
        groups = rng.choice((1, 1, 4, 8, 10, 16))
        each = rng.randrange(8, 257) if groups == 1 else rng.randrange(2, 256 // groups + 1)
        G = groups * each
        top_groups = rng.randrange(1, groups + 1)
        k = rng.randrange(1, min(8, top_groups * each) + 1)
        T = min(131072, _spread(rng, 1, 131072 * 256 // max(G, 64)))
        return dict(op=op, T=T, G=G, k=k, type=rng.choice(("f32", "bf16", "f16")),
                    score=rng.choice(("sigmoid", "sigmoid", "softmax")), bias=rng.random() < 0.6, groups=groups,
                    top_groups=top_groups, group_top=rng.choice((1, 2)), renorm=rng.random() < 0.7,
                    scale=rng.choice((1.0, 2.5)), padded=rng.choice((0.0, 0.1)), train=rng.random() < 0.5)
    T = _spread(rng, 1, 16384)
    t = rng.choice(("bf16", "f16"))
    return dict(op=op, T=T, K=_spread(rng, 256, 4096, 8), N=_spread(rng, 256, 4096, 8), r=rng.choice((8, 16, 32, 64)),
                G=rng.choice((1, 4, 16, 64) if T <= 1024 else (1, 4, 16)), type=t, base=rng.choice((t, t, "f32")),
                requests=rng.choice((1, max(1, T // 300), max(1, min(T, 64)))), idle=rng.choice((0.0, 0.1)),
                scaled=rng.random() < 0.7)


# ------------------------------------------------------------------------------------------------- the inputs


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, rows, cols):
    """Normal values whose columns differ in size, a few of them much larger: what a layer's input looks like."""
    x = _randn(g, rows, cols)
    size = torch.exp(0.5 * _randn(g, cols))
    size[torch.rand(cols, generator=g, device="cuda") < 0.01] *= 20.0
    return x.mul_(size)


def _rows(x, dtype, to=8):
    """x in a matrix whose row length in memory is a multiple of `to` elements."""
    rows, cols = x.shape
    out = torch.empty(rows, -(-cols // to) * to, dtype=dtype, device="cuda")[:, :cols]
    return out.copy_(x)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    state = {"case": case}
    if op == "norm":
        M, K = case["M"], case["K"]
        state["x"] = _rows(_activations(g, M, K), TYPES[case["x"]])
        state["residual"] = None
        if case["residual"] != "none":
            state["residual"] = _rows(_activations(g, M, K).mul_(2.0), TYPES[case["residual"]])
        state["gain"] = None
        if case["gain"] != "none":
            state["gain"] = (1.0 + 0.2 * _randn(g, K)).to(TYPES[case["gain"]])
        if case["train"]:
            state["dy"] = _rows(_randn(g, M, K).mul_(0.1), TYPES[case["x"]])
            state["d_hidden"] = None
            if state["residual"] is not None:
                state["d_hidden"] = _rows(_randn(g, M, K).mul_(0.1), TYPES[case["residual"]])
    elif op == "router":
        T, G = case["T"], case["G"]
        liked = 0.5 * _randn(g, G)                                   # some experts are liked more than others
        x = _randn(g, T, G).mul_(1.2) + liked
        if case["padded"]:
            x[torch.rand(T, generator=g, device="cuda") < case["padded"]] = -INF
        state["logits"] = x.to(TYPES[case["type"]])
        state["bias"] = None
        if case["bias"]:                                             # what a balancing rule has arrived at
            state["bias"] = -0.15 * liked + 0.01 * _randn(g, G)
        if case["train"]:
            state["d_weights"] = _randn(g, T, case["k"]).mul_(0.1)
            state["d_loss"] = torch.full((), 0.01 * T, device="cuda")
    else:
        T, K, N, r, G = case["T"], case["K"], case["N"], case["r"], case["G"]
        t = TYPES[case["type"]]
        # requests are neighbours: row i belongs to the request that the cut points below i count
        cuts = torch.randint(0, T + 1, (case["requests"] - 1,), generator=g, device="cuda")
        if case["requests"] >= T:
            request = torch.arange(T, device="cuda")
        else:
            request = (torch.arange(T, device="cuda")[:, None] >= cuts).sum(1)
        which = torch.randint(0, G, (max(case["requests"], T),), generator=g, device="cuda")
        which[torch.rand(which.shape, generator=g, device="cuda") < case["idle"]] = -1      # requests without one
        state["adapters"] = which[request].int()
        state["x"] = _activations(g, T, K).to(t)
        state["a"] = _randn(g, G, r, K).mul_(K ** -0.5).to(t)
        state["b"] = _randn(g, G, N, r).mul_(0.3 * r ** -0.5).to(t)
        state["base"] = _randn(g, T, N).to(TYPES[case["base"]])
        state["scale"] = torch.rand(G, generator=g, device="cuda") * 1.5 + 0.5 if case["scaled"] else None
    return state


# ------------------------------------------------------------------------------------------------- one pass


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    import grouped_gemm_persistent_gb300 as tg
    case = state["case"]
    op = case["op"]
    if op == "norm":
        n = tg.rmsnorm(state["x"], state["gain"], EPS, residual=state["residual"],
                       out_dtype=TYPES.get(case["out"]), fp8_dtype=TYPES.get(case["q"]))
        out = [v for v in (n.y, n.q, n.scale) if v is not None] + [n.hidden, n.row_scale]
        if case["train"]:
            out += [v for v in tg.rmsnorm_backward(n, state["dy"], state["gain"], state["d_hidden"]) if v is not None]
        return out
    if op == "router":
        r = tg.moe_router(state["logits"], case["k"], renormalize=case["renorm"], score=case["score"],
                          bias=state["bias"], groups=case["groups"], top_groups=case["top_groups"],
                          group_top=min(case["group_top"], case["G"] // case["groups"]), weight_scale=case["scale"])
        out = [r.experts, r.weights, r.counts, r.loss]
        if case["train"]:
            out.append(tg.moe_router_backward(state["logits"], r, state["d_weights"], state["d_loss"]))
        return out
    return tg.lora_add(state["base"], state["x"], state["a"], state["b"], state["adapters"], state["scale"])


def _run_plain(state):
    op = state["case"]["op"]
    return _norm_plain(state) if op == "norm" else _router_plain(state) if op == "router" else _lora_plain(state)


def _pow2_scale(amax, top):
    """The smallest power of two s, at least 2^-126, with amax <= top * s; 1 for a block of zeros."""
    m, e = torch.frexp(amax.double() / top)             # amax / top = m 2^e with m in [1/2, 1), exact enough:
    e = torch.where(m == 0.5, e - 1, e)                 # top is 7 * 2^j, so the quotient rounds onto no power of two
    s = torch.ldexp(torch.ones_like(m), e.clamp(min=-126))
    return torch.where(amax > 0, s, torch.ones_like(s)).float()


def _norm_plain(state):
    """The row factor is worked out in 64 bits and rounded once: an 8-bit value next to a border, and a scale next to
    a power of two, would otherwise fall on either side with the order of a sum."""
    case = state["case"]
    M, K = case["M"], case["K"]
    x, residual = state["x"], state["residual"]
    hidden = x if residual is None else (x.float() + residual.float()).to(residual.dtype)
    h = hidden.float()
    r = (h.double().square().mean(1) + EPS).rsqrt().float()
    y = h * r[:, None]
    if state["gain"] is not None:
        y = y * state["gain"].float()
    out = []
    if case["out"] != "none":
        out.append(y.to(TYPES[case["out"]]))
    if case["q"] != "none":
        t = torch.nn.functional.pad(y, (0, -K % BLOCK)).view(M, _blocks(K), BLOCK)
        s = _pow2_scale(t.abs().amax(2), TOP[case["q"]])
        q = (t / s[:, :, None]).clamp(-TOP[case["q"]], TOP[case["q"]]).to(TYPES[case["q"]])
        out += [q.view(M, -1)[:, :K], s]
    out += [hidden, r]
    if case["train"]:
        dy = state["dy"].float()
        if state["gain"] is not None:
            d = dy * state["gain"].float()
            d_gain = (dy * h * r[:, None]).sum(0, dtype=torch.float64).float()
        else:
            d, d_gain = dy, None
        c = (d * h).sum(1, keepdim=True, dtype=torch.float64).float() * r[:, None] ** 3 / K
        dh = d * r[:, None] - h * c
        if state["d_hidden"] is not None:
            dh = dh + state["d_hidden"].float()
        out.append(dh.to(hidden.dtype))
        if d_gain is not None:
            out.append(d_gain)
    return out


def _router_plain(state):
    """The choice is made on scores in 64 bits: with 32, two experts next to each other change places."""
    case = state["case"]
    T, G, k = case["T"], case["G"], case["k"]
    groups, each = case["groups"], case["G"] // case["groups"]
    x = state["logits"].double()
    live = x > -INF
    if case["score"] == "softmax":
        top = x.amax(1, keepdim=True)
        e = torch.where(live, (x - torch.where(top > -INF, top, torch.zeros_like(top))).exp(), torch.zeros_like(x))
        s = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        s = 1.0 / (1.0 + (-x).exp())
    v = s if state["bias"] is None else s + state["bias"].double()
    v = torch.where(live, v, torch.full_like(v, -INF))
    best = v.view(T, groups, each).topk(min(case["group_top"], each), dim=2).values
    score = torch.where(best > -INF, best, torch.zeros_like(best)).sum(2)
    score = torch.where(best[:, :, 0] > -INF, score, torch.full_like(score, -INF))
    kept = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
    looked = torch.zeros(T, groups, dtype=torch.bool, device="cuda").scatter_(1, kept, True).repeat_interleave(each, 1)
    by = torch.where(looked, x if state["bias"] is None else v, torch.full_like(v, -INF))
    order = torch.sort(by, dim=1, descending=True, stable=True)
    taken = order.values[:, :k] > -INF
    idx = order.indices[:, :k]
    experts = torch.where(taken, idx, torch.full_like(idx, -1)).int()
    s = s.float()
    chosen = torch.where(taken, s.gather(1, idx), torch.zeros(T, k, device="cuda"))
    total = chosen.sum(1, keepdim=True).clamp(min=1e-37)
    factor = case["scale"] / total if case["renorm"] else torch.full_like(total, case["scale"])
    w = chosen * factor
    counts = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    slot = torch.where(taken, idx, torch.full_like(idx, G)).flatten()
    counts.index_add_(0, slot, torch.ones_like(slot, dtype=torch.int32))
    counts = counts[:G]
    rows = live.any(1).sum().clamp(min=1).double()
    slope = G * counts.double() / (rows * k) / rows              # the loss's derivative by each share
    whole = s.sum(1, keepdim=True).clamp(min=1e-37)
    p = s / whole
    loss = (slope * p.sum(0, dtype=torch.float64)).sum().float()
    out = [experts, w, counts, loss]
    if case["train"]:
        dw = torch.where(taken, state["d_weights"], torch.zeros_like(w))
        if case["renorm"]:
            dw = dw - (dw * chosen).sum(1, keepdim=True) / total
        dw = torch.where(taken, dw * factor, torch.zeros_like(dw))
        u = (slope.float() * state["d_loss"])[None]
        ds = (u - (p * u).sum(1, keepdim=True)) / whole          # by each score
        ds = ds.scatter_add(1, idx, dw)
        if case["score"] == "softmax":
            d = s * (ds - (s * ds).sum(1, keepdim=True))
        else:
            d = s * (1.0 - s) * ds
        out.append(torch.where(live, d, torch.zeros_like(d)).to(state["logits"].dtype))
    return out


def _lora_plain(state):
    """Every adapter's first product for every row, the rows' own kept, then the second products summed."""
    case = state["case"]
    G, r, K, N = case["G"], case["r"], case["K"], case["N"]
    u = state["x"].float() @ state["a"].float().view(G * r, K).t()
    mine = state["adapters"][:, None] == torch.arange(G, device="cuda")
    factor = mine.float() if state["scale"] is None else mine * state["scale"]
    u = (u.view(-1, G, r) * factor[:, :, None]).view(-1, G * r)
    y = u @ state["b"].float().transpose(1, 2).reshape(G * r, N)
    return (state["base"].float() + y).to(state["base"].dtype)


# ------------------------------------------------------------------------------------------------- 64 bits


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    return _norm_exact(state) if op == "norm" else _router_exact(state) if op == "router" else _lora_exact(state)


def _norm_exact(state):
    case = state["case"]
    M, K = case["M"], case["K"]
    h = state["x"].double()
    if state["residual"] is not None:                                # the stream is held in the residual's type
        h = (h + state["residual"].double()).float().to(state["residual"].dtype).double()
    norm = torch.linalg.vector_norm(h, dim=1, keepdim=True)
    r = 1.0 / torch.sqrt(norm * norm / K + EPS)
    g = torch.ones(K, dtype=torch.float64, device="cuda") if state["gain"] is None else state["gain"].double()
    y = h * (r * g)
    out = [y] if case["out"] != "none" else []
    if case["q"] != "none":
        bits, low = (3, -6) if case["q"] == "e4m3" else (2, -14)     # mantissa bits, exponent of the smallest normal
        top = TOP[case["q"]]
        pad = torch.zeros(M, _blocks(K) * BLOCK, dtype=torch.float64, device="cuda")
        pad[:, :K] = y
        t = pad.view(M, -1, BLOCK)
        big = t.abs().amax(2, keepdim=True)
        e = torch.floor(torch.log2(torch.where(big > 0, big, torch.ones_like(big)))) - math.floor(math.log2(top)) - 1
        for _ in range(3):
            e = torch.where(big > top * torch.exp2(e), e + 1, e)
        s = torch.where(big > 0, torch.exp2(e.clamp(min=-126)), torch.ones_like(e))
        v = t / s
        _, ev = torch.frexp(v)
        step = torch.exp2((ev.double() - 1).clamp(min=low) - bits)
        q = torch.round(v / step) * step                             # ties to even multiples of the step
        out += [q.view(M, -1)[:, :K], s[:, :, 0]]
    out += [h, r[:, 0]]
    if case["train"]:
        dy = state["dy"].double()
        n = h * r
        dn = dy * g
        dh = r * (dn - n * (dn * n).mean(1, keepdim=True))
        if state["d_hidden"] is not None:
            dh = dh + state["d_hidden"].double()
        out.append(dh)
        if state["gain"] is not None:
            out.append((dy * n).sum(0))
    return out


def _router_exact(state):
    case = state["case"]
    T, G, k = case["T"], case["G"], case["k"]
    groups, each = case["groups"], case["G"] // case["groups"]
    x = state["logits"].double()
    none = torch.full_like(x, -INF)
    if case["score"] == "softmax":
        lse = torch.logsumexp(x, 1, keepdim=True)
        s = torch.exp(x - torch.where(lse > -INF, lse, torch.zeros_like(lse)))
    else:
        s = torch.sigmoid(x)
    v = s + state["bias"].double() if state["bias"] is not None else s
    v = torch.where(x == -INF, none, v)
    # a group's score: its largest value, and the largest left
    left = v.clone().view(T, groups, each)
    score = left.amax(2)
    if min(case["group_top"], each) == 2:
        left.scatter_(2, left.argmax(2, keepdim=True), -INF)
        second = left.amax(2)
        score = torch.where(second > -INF, score + second, score)
    kept = torch.zeros(T, groups, dtype=torch.bool, device="cuda")
    lane = torch.arange(groups, device="cuda").expand(T, groups)
    for _ in range(case["top_groups"]):
        best = score.amax(1, keepdim=True)
        i = torch.where(score == best, lane, torch.full_like(lane, groups)).amin(1, keepdim=True)
        kept.scatter_(1, i, True)
        score = score.scatter(1, i, -INF)
    left = torch.where(kept[:, :, None].expand(T, groups, each).reshape(T, G),
                       x if state["bias"] is None else v, none)
    experts = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    chosen = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    lane = torch.arange(G, device="cuda").expand(T, G)
    for j in range(k):
        best = left.amax(1, keepdim=True)
        i = torch.where(left == best, lane, torch.full_like(lane, G)).amin(1)      # ties: the lowest index
        ok = best[:, 0] > -INF
        experts[:, j] = torch.where(ok, i, torch.full_like(i, -1)).int()
        chosen[:, j] = s.gather(1, i[:, None])[:, 0] * ok
        left.scatter_(1, i[:, None], -INF)
    ok = experts >= 0
    at = experts.clamp(min=0).long()
    counts = torch.zeros(G, dtype=torch.float64, device="cuda").index_add_(0, at.flatten(), ok.flatten().double())
    n = max(1, int((x > -INF).any(1).sum()))
    whole = s.sum(1, keepdim=True)
    safe = torch.where(whole > 0, whole, torch.ones_like(whole))
    p = s / safe
    loss = G * (counts / (n * k) * (p.sum(0) / n)).sum()
    total = chosen.sum(1, keepdim=True)
    total = torch.where(total > 0, total, torch.ones_like(total)) if case["renorm"] else torch.ones_like(total)
    w = case["scale"] * chosen / total
    out = [experts, w, counts.int(), loss]
    if case["train"]:
        dw = state["d_weights"].double() * ok * case["scale"]
        if case["renorm"]:
            dw = (dw - (dw * chosen / total).sum(1, keepdim=True)) / total * ok
        dp = float(state["d_loss"]) * G * counts / (n * k) / n
        ds = (dp - (p * dp).sum(1, keepdim=True)) / safe
        ds = ds.scatter_add(1, at, dw)
        if case["score"] == "softmax":
            d = s * (ds - (s * ds).sum(1, keepdim=True))
        else:
            d = s * torch.sigmoid(-x) * ds
        out.append(torch.where(x == -INF, torch.zeros_like(d), d))
    return out


def _lora_exact(state):
    y = state["base"].double()
    for g in range(state["a"].shape[0]):
        rows = torch.nonzero(state["adapters"] == g)[:, 0]
        if rows.numel():
            low = state["x"][rows].double() @ state["a"][g].double().t()
            add = low @ state["b"][g].double().t()
            y[rows] += add if state["scale"] is None else add * state["scale"][g].double()
    return y


# ------------------------------------------------------------------------------------------------- the work


def work(case):
    op = case["op"]
    if op == "norm":
        M, K = case["M"], case["K"]
        hidden = case["x"] if case["residual"] == "none" else case["residual"]
        each = SIZE[case["x"]] + SIZE[case["out"]] + SIZE[case["q"]]
        if case["residual"] != "none":
            each += 2 * SIZE[hidden]
        flops = 6
        if case["train"]:
            each += SIZE[case["x"]] + 2 * SIZE[hidden] + (SIZE[hidden] if case["residual"] != "none" else 0)
            flops += 12
        scales = 4 * M * _blocks(K) if case["q"] != "none" else 0
        return {"bytes": M * K * each + scales + 4 * M + K * SIZE[case["gain"]], "flops": flops * M * K}
    if op == "router":
        T, G, k = case["T"], case["G"], case["k"]
        logits = T * G * SIZE[case["type"]]
        out = T * k * 8 + G * 4 + 4 + (G * 4 if case["bias"] else 0)
        if not case["train"]:
            return {"bytes": logits + out, "flops": 6 * T * G}
        return {"bytes": 2 * logits + out + T * k * 4 + 4, "flops": 12 * T * G}
    T, K, N, r = case["T"], case["K"], case["N"], case["r"]
    used = min(case["G"], T, case["requests"])                       # adapters that can have rows at all
    s = SIZE[case["type"]]
    return {"bytes": T * K * s + 2 * T * N * SIZE[case["base"]] + used * r * (K + N) * s + 4 * T,
            "flops": 2 * T * r * (K + N)}
