"""The gate with sigmoid scores, a bias, groups and a factor: refusals and the reference itself (CPU), parity with 64 bits
(GPU)."""
import subprocess

import pytest
import torch

import grouped_gemm_persistent_gb300 as tg
from grouped_gemm_persistent_gb300 import _binding
from grouped_gemm_persistent_gb300.build import INCLUDE, build

PTR = 0x10000
INF = float("inf")
BF, HF, F = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24      # half a step of fp32
BAD, NO = tg.TG_ERR_INVALID_ARG, tg.TG_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build()
    return tg.load()


# ------------------------------------------------------------------------------------------ refusals (CPU)

FORWARD = dict(T=4, G=64, k=2, logits=PTR, ld=64, bias=2 * PTR, groups=8, top_groups=4, group_top=2, experts=PTR, weights=PTR,
               counts=PTR, loss=PTR, slope=PTR, scale=1.0, dt=1, score=1, renorm=0)
BACKWARD = dict(T=4, G=64, k=2, logits=PTR, ld=64, experts=PTR, slope=PTR, dw=PTR, dl=PTR, out=2 * PTR, ldd=64,
                scale=1.0, dt=1, score=1, renorm=0)


def forward(lib, **kw):
    return lib.tg_moe_router_scored(_binding._ROUTER.pack(*{**FORWARD, **kw}.values()), None)


def backward(lib, **kw):
    return lib.tg_moe_router_scored_backward(_binding._ROUTER_BACKWARD.pack(*{**BACKWARD, **kw}.values()), None)


SHARED = [(dict(dt=3), BAD), (dict(T=-1), BAD), (dict(k=0), BAD), (dict(k=65), BAD), (dict(G=1025, ld=1025), NO),
          (dict(logits=0), BAD), (dict(ld=63), BAD), (dict(logits=PTR + 2), BAD), (dict(score=2), BAD), (dict(score=-1), BAD),
          (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD), (dict(scale=INF), BAD), (dict(scale=float("nan")), BAD)]


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(groups=0), BAD), (dict(groups=7), BAD), (dict(groups=128), BAD), (dict(top_groups=0), BAD), (dict(top_groups=9), BAD),
    (dict(group_top=0), BAD), (dict(group_top=3), BAD), (dict(groups=64, top_groups=4, group_top=2), BAD),
    (dict(k=9, top_groups=1), BAD), (dict(groups=64, top_groups=4, group_top=1), NO),
    (dict(G=1000, ld=1000, groups=40, group_top=1), NO), (dict(experts=0), BAD), (dict(weights=0), BAD), (dict(counts=0), BAD),
    (dict(loss=0), BAD), (dict(slope=0), BAD), (dict(weights=PTR + 2), BAD), (dict(bias=PTR + 2), BAD),
])
def test_forward_refusals(lib, kw, code):
    assert forward(lib, **kw) == code
    assert lib.tg_last_error_message()


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(experts=0), BAD), (dict(slope=0), BAD), (dict(out=0), BAD), (dict(ldd=63), BAD),
    (dict(out=PTR + 2), BAD), (dict(dl=PTR + 1), BAD)])
def test_backward_refusals(lib, kw, code):
    assert backward(lib, **kw) == code
    assert lib.tg_last_error_message()


def test_null_record_and_no_rows(lib):
    assert lib.tg_moe_router_scored(None, None) == BAD
    assert lib.tg_moe_router_scored_backward(None, None) == BAD
    assert backward(lib, T=0, logits=0, out=0) == tg.TG_OK


def test_records_match_the_header(tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "tg.h"\nint main(void) {\n'
                   'printf("%zu %zu %zu %zu\\n", sizeof(tg_router_args), offsetof(tg_router_args, weight_scale),'
                   ' sizeof(tg_router_backward_args), offsetof(tg_router_backward_args, weight_scale)); return 0; }\n')
    subprocess.run(["gcc", "-I", INCLUDE, str(src), "-o", str(tmp_path / "sizes")], check=True)
    out = subprocess.run([str(tmp_path / "sizes")], capture_output=True, text=True, check=True).stdout.split()
    f, b = _binding._ROUTER.size, _binding._ROUTER_BACKWARD.size
    assert [int(v) for v in out] == [f, f - 16, b, b - 16]


def test_binding_refusals():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        tg.moe_router(x, 2, score="tanh")
    with pytest.raises(ValueError):
        tg.moe_router(x, 2, score="sigmoid", bias=torch.zeros(7))
    with pytest.raises(ValueError):
        tg.moe_router(x, 2, score="sigmoid", bias=torch.zeros(8).half())
    with pytest.raises(ValueError, match="CUDA"):
        tg.moe_router(x, 2, score="sigmoid", groups=4)


# ------------------------------------------------------------------------------------------ the reference


def scores(x, score):
    """Scores of the rows in 64 bits, 0 where the logit is -infinity."""
    x = x.double()
    if score == "sigmoid":
        return torch.sigmoid(x)
    top = x.amax(1, keepdim=True)
    e = (x - torch.where(top == -INF, torch.zeros_like(top), top)).exp()
    return e / torch.where(top == -INF, torch.ones_like(top), e.sum(1, keepdim=True))


def choose(x, k, score, bias, groups, top_groups, group_top):
    """experts [T, k] by the definition, one row and one choice at a time."""
    T, G = x.shape
    each = G // groups
    v = scores(x, score) + (0 if bias is None else bias.double())
    v = torch.where(x.double() == -INF, torch.full_like(v, -INF), v)
    parts = v.view(T, groups, each).sort(dim=2, descending=True).values[:, :, :group_top]
    value = torch.where(parts > -INF, parts, torch.zeros_like(parts)).sum(2)
    value = torch.where(parts[:, :, 0] > -INF, value, torch.full_like(value, -INF))
    if bias is None and group_top == 1:
        value = x.double().view(T, groups, each).amax(2)
    kept = value.sort(dim=1, descending=True, stable=True).indices[:, :top_groups]
    open_ = torch.zeros(T, groups, dtype=torch.bool, device=x.device).scatter_(1, kept, True).repeat_interleave(each, 1)
    by = torch.where(open_, x.double() if bias is None else v, torch.full_like(v, -INF))
    got = by.sort(dim=1, descending=True, stable=True)
    return torch.where(got.values[:, :k] > -INF, got.indices[:, :k], torch.full_like(got.indices[:, :k], -1)).int()


def weigh(x, experts, score, renorm, factor):
    """(weights, chosen scores, their sum) in 64 bits."""
    s = scores(x, score)
    chosen = torch.where(experts >= 0, s.gather(1, experts.clamp(min=0).long()), torch.zeros(experts.shape, dtype=torch.float64, device=x.device))
    total = chosen.sum(1, keepdim=True)
    total = torch.where(total > 0, total, torch.ones_like(total))
    return factor * (chosen / total if renorm else chosen), chosen, total


def balance(x, experts, score):
    """(counts, loss, slope, shares, rows) in 64 bits."""
    G, k = x.shape[1], experts.shape[1]
    s = scores(x, score)
    whole = s.sum(1, keepdim=True)
    p = s / torch.where(whole > 0, whole, torch.ones_like(whole))
    counts = torch.bincount(experts[experts >= 0].long(), minlength=G)
    n = max(1, int((x > -INF).any(1).sum()))
    slope = G * counts.double() / (n * k) / n
    return counts.int(), (slope * p.sum(0)).sum(), slope, p


def gradient(x, experts, score, renorm, factor, dw, dl):
    """(d logits, a bound of the magnitudes that went into each) in 64 bits, from the formulas."""
    s = scores(x, score)
    whole = s.sum(1, keepdim=True)
    whole = torch.where(whole > 0, whole, torch.ones_like(whole))
    _, chosen, total = weigh(x, experts, score, renorm, factor)
    ok = experts >= 0
    at = experts.clamp(min=0).long()
    c = factor * dw.double() * ok
    size = c.abs()
    if renorm:
        size = (size + (size * chosen).sum(1, keepdim=True) / total) / total * ok
        c = (c - (c * chosen).sum(1, keepdim=True) / total) / total * ok
    slope = balance(x, experts, score)[2]
    u = dl * slope[None]
    p = s / whole
    ds = ((u - (p * u).sum(1, keepdim=True)) / whole).scatter_add(1, at, c)
    mag = ((u.abs() + (p * u.abs()).sum(1, keepdim=True)) / whole).scatter_add(1, at, size)
    if score == "softmax":
        return s * (ds - (s * ds).sum(1, keepdim=True)), s * (mag + (s * mag).sum(1, keepdim=True))
    f = s * torch.sigmoid(-x.double())
    return f * ds, f * mag


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_reference_gradient_against_differences(score, renorm):
    g = torch.Generator().manual_seed(0)
    T, G, k = 4, 12, 3
    x = torch.randn(T, G, generator=g, dtype=torch.float64) * 2
    x[1, 4] = -INF
    x[2] = -INF
    bias = torch.randn(G, generator=g) * 0.1
    dw, dl = torch.randn(T, k, generator=g, dtype=torch.float64), 0.7
    args = (k, score, bias, 4, 2, 2)
    experts = choose(x, *args)
    d, _ = gradient(x, experts, score, renorm, 2.5, dw, dl)

    def value(y):
        assert torch.equal(choose(y, *args), experts)             # the step does not change the choice
        return float((weigh(y, experts, score, renorm, 2.5)[0] * dw).sum() + dl * balance(y, experts, score)[1])

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


def spread(x, score):
    """How far a row's logits go: from zero (sigmoid), below its largest (softmax)."""
    x = torch.where(x.double() > -INF, x.double(), torch.zeros((), dtype=torch.float64, device=x.device))
    return (x.abs() if score == "sigmoid" else x.amax(1, keepdim=True) - x).amax(1, keepdim=True).clamp(min=1.0)


def check(x, k, r, *, score="sigmoid", bias=None, groups=1, top_groups=1, group_top=1, renorm=False, factor=1.0):
    experts = choose(x, k, score, bias, groups, top_groups, group_top)
    assert torch.equal(r.experts, experts)
    counts, loss, slope, _ = balance(x, experts, score)
    assert torch.equal(r.counts, counts)
    w, *_ = weigh(x, experts, score, renorm, factor)
    D = spread(x, score)
    # e^d: |d| half steps from the argument's rounding, (2 + 1.16 |d|) steps for the function; a sum of 32 + 6 such, a
    # reciprocal; once more for the sum of the chosen
    one = 2 * (2 + 1.16 * D) * U + D * U + (4 + 2 * D + 40) * U
    tol = 2 * one * w + 10 * U * w + 2.0 ** -120
    assert bool(((r.weights.double() - w).abs() <= tol).all())
    # each share to `one`; a lane's rows, slots, warps and blocks: at most 300 additions
    far = float(one.max()) + 300 * U
    assert abs(float(r.loss.double() - loss)) <= far * float(loss) + 2.0 ** -120
    assert bool(((r.slope.double() - slope).abs() <= 2 * U * slope).all())
    return experts


def check_gradient(x, r, experts, d, dw, dl, *, score="sigmoid", renorm=False, factor=1.0):
    want, size = gradient(x, experts, score, renorm, factor, dw, dl)
    eps = torch.finfo(x.dtype).eps
    tol = eps / 2 * want.abs() + (10 * spread(x, score) + 120) * U * size + torch.finfo(x.dtype).tiny * eps
    assert bool(((d.double() - want).abs() <= tol).all())
    assert bool((d[x == -INF] == 0).all())


def make(seed, T, G, dt, padded=0.1, banned=0.05):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, G, generator=g, device="cuda") * 1.5
    x[torch.rand(T, G, generator=g, device="cuda") < banned] = -INF
    x[torch.rand(T, generator=g, device="cuda") < padded] = -INF
    bias = torch.randn(G, generator=g, device="cuda") * 0.2
    return x.to(dt), bias, torch.randn(T, 32, generator=g, device="cuda")


CASES = [  # T, G, k, groups, top_groups, group_top
    (1, 1, 1, 1, 1, 1), (3, 8, 8, 1, 1, 1), (65, 64, 4, 1, 1, 1), (200, 256, 8, 8, 4, 2), (200, 256, 8, 8, 4, 1),
    (333, 190, 6, 10, 3, 1), (129, 160, 6, 8, 3, 2), (50, 24, 3, 12, 4, 2), (77, 32, 2, 32, 5, 1), (31, 60, 20, 3, 2, 2),
    (40, 257, 16, 1, 1, 1), (90, 512, 32, 4, 3, 2), (25, 1000, 10, 8, 5, 2), (33, 1024, 8, 32, 6, 2), (17, 1024, 32, 1, 1, 1),
    (2500, 96, 5, 6, 2, 2), (66, 128, 9, 2, 1, 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,G,k,groups,top_groups,group_top", CASES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_sizes(T, G, k, groups, top_groups, group_top, score):
    for i, (dt, with_bias) in enumerate(((F, True), (BF, True), (HF, False), (F, False), (BF, False))):
        x, bias, dw = make(i, T, G, dt)
        dw = dw[:, :k].contiguous()
        kw = dict(score=score, bias=bias if with_bias else None, groups=groups, top_groups=top_groups, group_top=group_top)
        renorm, factor = i % 2 == 0, (2.5, 1.0, 16.0)[i % 3]
        r = tg.moe_router(x, k, renormalize=renorm, weight_scale=factor, **kw)
        experts = check(x, k, r, renorm=renorm, factor=factor, **kw)
        dl = torch.full((), 0.3, device="cuda")
        d = tg.moe_router_backward(x, r, dw, dl)
        check_gradient(x, r, experts, d, dw, 0.3, score=score, renorm=renorm, factor=factor)
    tg.device_status()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F, BF])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_many_rows(dt, score):
    """More rows than one pass of the grid, twice the same."""
    x, bias, dw = make(7, 30000, 128, dt)
    dw = dw[:, :4].contiguous()
    kw = dict(score=score, bias=bias, groups=8, top_groups=3, group_top=2)
    r = tg.moe_router(x, 4, renormalize=True, weight_scale=2.5, **kw)
    experts = check(x, 4, r, renorm=True, factor=2.5, **kw)
    dl = torch.full((), 20.0, device="cuda")
    d = tg.moe_router_backward(x, r, dw, dl)
    check_gradient(x, r, experts, d, dw, 20.0, score=score, renorm=True, factor=2.5)
    again = tg.moe_router(x, 4, renormalize=True, weight_scale=2.5, **kw)
    assert all(torch.equal(p, q) for p, q in zip(again[:5], r[:5]))
    assert torch.equal(tg.moe_router_backward(x, again, dw, dl), d)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("G,groups", [(64, 8), (256, 8), (512, 4)])
def test_choices_that_32_bits_do_not_tell_apart(score, group_top, G, groups):
    """A bias that takes the scores away: what is left is their rounding, about 1e-8, and rows that differ little."""
    g = torch.Generator(device="cuda").manual_seed(11)
    row = torch.randn(1, G, generator=g, device="cuda")
    x = row + torch.randn(60, G, generator=g, device="cuda") * 1e-6
    x[20:40] = row + torch.randn(20, G, generator=g, device="cuda") * 1e-3
    bias = -scores(row, score)[0].float()
    kw = dict(score=score, bias=bias, groups=groups, top_groups=3, group_top=group_top)
    r = tg.moe_router(x, 8, renormalize=True, **kw)
    check(x, 8, r, renorm=True, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("G,groups,k", [(64, 8, 8), (64, 8, 5), (256, 8, 8), (256, 16, 7), (40, 1, 6), (320, 4, 9)])
def test_a_few_choices_that_32_bits_do_not_tell_apart(score, group_top, G, groups, k):
    """Biases that bring the experts' values to within 1e-7 of steps of a fortieth: pairs and more of them next to each other."""
    g = torch.Generator(device="cuda").manual_seed(17)
    row = torch.randn(1, G, generator=g, device="cuda") * 0.5
    x = row + torch.randn(200, G, generator=g, device="cuda") * 2e-7
    s = scores(row, score)[0]
    for seed in range(3):
        wish = torch.randint(0, 40, (G,), generator=g, device="cuda") / 40
        if seed == 1:
            wish[::2] += 0.003 * torch.rand(wish[::2].shape, generator=g, device="cuda")
        bias = (wish - s).float()
        kw = dict(score=score, bias=bias, groups=groups, top_groups=max(1, groups // 2), group_top=group_top)
        check(x, k, tg.moe_router(x, k, renormalize=True, **kw), renorm=True, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dt", [F, BF, HF])
def test_ties_and_biases(score, dt):
    """Equal logits under a bias of zeros, biases that spread far, forbid an expert or force one."""
    x, bias, _ = make(12, 300, 64, dt)
    x[:100] = torch.round(x[:100] * 2) / 2                        # many equal ones
    x[100] = 0.25                                                 # all of them
    x[101, ::2] = 0.25
    for b in (torch.zeros(64, device="cuda"), torch.full((64,), 1000.0, device="cuda"), bias * 100, bias.clone(), bias.clone()):
        if b is not bias and float(b.abs().max()) < 5 and float(b.abs().max()) > 0:
            b[3::7] = -INF
            b[5] = 0.0
        for groups, top, group_top in ((1, 1, 1), (8, 3, 1), (8, 3, 2)):
            kw = dict(score=score, bias=b, groups=groups, top_groups=top, group_top=group_top)
            check(x, 6, tg.moe_router(x, 6, renormalize=True, **kw), renorm=True, **kw)
    far = bias.clone()
    far[10:20] = -1e9                                             # a mask by a large number
    far[40] = INF
    for groups, top, group_top in ((1, 1, 1), (8, 5, 2)):
        kw = dict(score=score, bias=far, groups=groups, top_groups=top, group_top=group_top)
        r = tg.moe_router(x, 6, **kw)
        check(x, 6, r, **kw)
        assert bool((r.experts[100] == 40).any())
    for groups, top, group_top in ((1, 1, 1), (8, 3, 1), (8, 3, 2)):
        kw = dict(score=score, bias=None, groups=groups, top_groups=top, group_top=group_top)
        check(x, 6, tg.moe_router(x, 6, weight_scale=2.0, **kw), factor=2.0, **kw)


@pytest.mark.gpu
def test_special_rows():
    x, bias, dw = make(13, 8, 32, F, padded=0.0, banned=0.0)
    x[0] = -INF                                                   # padding
    x[1, 5:] = -INF                                               # fewer experts than choices
    x[2] = -200.0                                                 # scores that are 0 in fp32
    x[3, 7] = INF
    x[4, 9] = float("nan")
    x[5] = 60.0                                                   # scores that are all 1
    r = tg.moe_router(x, 8, renormalize=True, score="sigmoid", bias=bias, groups=4, top_groups=2, group_top=2)
    assert bool((r.experts[0] == -1).all()) and bool((r.weights[0] == 0).all())
    assert int((r.experts[1] >= 0).sum()) == 5 and bool((r.weights[1][r.experts[1] < 0] == 0).all())
    assert bool((r.experts[2] >= 0).all()) and bool((r.weights[2] == 0).all())
    assert bool((r.experts[3] == 7).any()) and bool(r.weights[3].isfinite().all())
    assert int(r.experts[4, 0]) == 9 and bool(r.weights[4].isnan().all()) and bool(r.loss.isnan())
    rest = torch.tensor([0, 1, 3, 5, 6, 7], device="cuda")
    want = choose(x[rest], 8, "sigmoid", bias, 4, 2, 2)
    assert torch.equal(r.experts[rest], want)
    y = x[rest].contiguous()
    part = tg.moe_router(y, 8, renormalize=True, score="sigmoid", bias=bias, groups=4, top_groups=2, group_top=2)
    d = tg.moe_router_backward(y, part, dw[rest, :8].contiguous(), torch.ones((), device="cuda"))
    assert bool(d.isfinite().all()) and bool((d[0] == 0).all()) and bool((d[1, 5:] == 0).all()) and float(d[2, 7]) == 0.0
    both = tg.moe_router_backward(x, r, dw[:, :8].contiguous(), torch.ones((), device="cuda"))
    assert bool(both[4].isnan().all())


@pytest.mark.gpu
@pytest.mark.parametrize("G", [48, 63, 300])
@pytest.mark.parametrize("score,away,zero", [("sigmoid", 60.0, False), ("sigmoid", 86.0, False), ("sigmoid", 88.4, True),
                                             ("sigmoid", 100.0, True), ("softmax", 60.0, False), ("softmax", 78.0, False),
                                             ("softmax", 84.5, True), ("softmax", 86.5, True), ("softmax", 100.0, True)])
def test_chosen_scores_near_the_smallest_number(G, score, away, zero):
    """The bias takes the experts whose scores are next to nothing: their weights and gradients are those of real numbers while the
    scores are above 2^-126, and 0 below it.

    Scores: e^-(away +- 0.2), over 38 to 291 for softmax (the nine at the end have no more than the bias gives them), so on
    either side of 2^-126 = e^-87.34 as `zero` says.  An exponential of -x is off by x 2^-24 for the logit's difference,
    x 2^-24 for its product with log2 e and 2^-22 for itself: 2 * 88 * 2^-24 + 2^-22 < 1.2e-5.  A weight is a quotient of sums of
    them, off by twice that (and 8 roundings): < 2.6e-5 of itself.  A gradient w (1 - s) (g - sum w g) takes 4 times the largest |g|
    of that at most."""
    k = 4
    gen = torch.Generator(device="cuda").manual_seed(G)
    x = torch.zeros(37, G, device="cuda")
    if score == "sigmoid":
        x -= 120.0
    x[:, -9:] = -away + 0.4 * (torch.rand(37, 9, device="cuda", generator=gen) - 0.5)
    bias = torch.zeros(G, device="cuda")
    bias[-9:] = 2.0
    dw = torch.randn(37, k, device="cuda", generator=gen)
    r = tg.moe_router(x, k, renormalize=True, score=score, bias=bias, weight_scale=1.5)
    assert bool((r.experts >= G - 9).all())
    d = tg.moe_router_backward(x, r, dw)
    if zero:
        assert bool((r.weights == 0).all()) and bool((d == 0).all())
        return
    want = weigh(x, r.experts, score, True, 1.5)[0]
    assert float((r.weights - want).abs().max()) <= 2.6e-5 * 1.5
    grad = gradient(x, r.experts, score, True, 1.5, dw, 0.0)[0]
    assert float((d - grad).abs().max()) <= 4 * 2.6e-5 * 1.5 * float(dw.abs().max())


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(), dict(score="sigmoid"), dict(weight_scale=2.0), dict(score="sigmoid", groups=4, top_groups=2)])
def test_a_routing_put_together_by_hand(kw):
    x, bias, dw = make(16, 50, 64, F)
    r = tg.moe_router(x, 4, renormalize=True, **kw)
    again = tg.Routing(r.experts, r.weights, r.counts, r.loss, r.slope, True, r.score, r.weight_scale)
    one = torch.ones((), device="cuda")
    dw = dw[:, :4].contiguous()
    assert torch.equal(tg.moe_router_backward(x, r, dw, one), tg.moe_router_backward(x, again, dw, one))


@pytest.mark.gpu
def test_parts_of_the_gradient():
    x, bias, dw = make(14, 70, 40, F)
    dw = dw[:, :3].contiguous()
    kw = dict(score="sigmoid", bias=bias)
    r = tg.moe_router(x, 3, weight_scale=1.5, **kw)
    experts = check(x, 3, r, factor=1.5, **kw)
    zero = torch.zeros_like(dw)
    check_gradient(x, r, experts, tg.moe_router_backward(x, r, None, torch.ones((), device="cuda")), zero, 1.0, factor=1.5)
    check_gradient(x, r, experts, tg.moe_router_backward(x, r, dw), dw, 0.0, factor=1.5)
    assert bool((tg.moe_router_backward(x, r) == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F, BF])
def test_rows_off_the_16_byte_boundaries(dt):
    x, bias, dw = make(15, 90, 72, dt)
    wide = torch.zeros(90, 80, dtype=dt, device="cuda")
    for at in (0, 1, 3):
        y = wide[:, at:at + 72]
        y.copy_(x)
        kw = dict(score="sigmoid", bias=bias, groups=3, top_groups=2, group_top=2)
        r = tg.moe_router(y, 4, renormalize=True, **kw)
        experts = check(x, 4, r, renorm=True, **kw)
        out = torch.full((92, 80), 7.0, dtype=dt, device="cuda")
        d = tg.moe_router_backward(y, r, dw[:, :4].contiguous(), None, out[1:91, at:at + 72])
        check_gradient(x, r, experts, d, dw[:, :4], 0.0, renorm=True)
        d.fill_(7.0)
        assert bool((out == 7.0).all())


@pytest.mark.gpu
def test_no_rows():
    x = torch.zeros(0, 16, device="cuda")
    r = tg.moe_router(x, 2, score="sigmoid", groups=2, top_groups=1)
    assert bool((r.counts == 0).all()) and float(r.loss) == 0.0 and bool((r.slope == 0).all())
    assert tg.moe_router_backward(x, r).shape == (0, 16)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [64, 5000])
def test_other_stream_and_graph(T):
    x, bias, dw = make(16, T, 128, F)
    dw = dw[:, :4].contiguous()
    dl = torch.ones((), device="cuda")
    kw = dict(renormalize=True, score="sigmoid", bias=bias, groups=8, top_groups=3, group_top=2, weight_scale=2.5)
    want = tg.moe_router(x, 4, **kw)
    want_d = tg.moe_router_backward(x, want, dw, dl)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    r = tg.moe_router(x, 4, stream=side, **kw)
    d = tg.moe_router_backward(x, r, dw, dl, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(r[:5], want[:5])) and torch.equal(d, want_d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = tg.moe_router(x, 4, **kw)
        d = tg.moe_router_backward(x, r, dw, dl)
    for _ in range(2):
        for t in (*r[:5], d):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(r[:5], want[:5])) and torch.equal(d, want_d)
