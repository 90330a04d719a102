"""An expert with a bias of -infinity is not chosen, whatever the row's scores are (GPU)."""
import pytest
import torch

import grouped_gemm_persistent_gb300 as tg
from test_router_scored import BF, F, INF, lib  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top_groups,group_top", [(1, 1, 1), (8, 4, 1), (8, 4, 2)])
@pytest.mark.parametrize("G", [64, 256, 512])
@pytest.mark.parametrize("dt", [F, BF])
def test_forbidden_beside_scores_that_are_nan(score, groups, top_groups, group_top, G, dt):
    """A NaN logit (with softmax an infinite one too) makes scores NaN, which come before all numbers; a forbidden one stays out."""
    k, each = 6, G // groups
    g = torch.Generator(device="cuda").manual_seed(60)
    x = torch.randn(9, G, generator=g, device="cuda").to(dt)
    bias = torch.randn(G, generator=g, device="cuda") * 0.1
    bias[::3] = -INF
    bias[each:2 * each] = -INF                     # (a whole group, where there are groups)
    if groups == 1:
        bias[1::2] = 0.0
    x[1, 0] = float("nan")                         # a forbidden expert's
    x[2, 5] = float("nan")                         # one that may be chosen
    x[3, 3], x[3, 4] = float("nan"), INF
    x[4, 6] = INF
    r = tg.moe_router(x, k, score=score, bias=bias, groups=groups, top_groups=top_groups, group_top=group_top)
    assert bool((r.experts >= 0).all())
    assert bool((bias[r.experts.long()] > -INF).all())
    assert int(r.counts[bias == -INF].sum()) == 0
    if score == "softmax":                         # all of the row is NaN: the lowest indices that may be chosen
        free = torch.nonzero(bias > -INF)[:, 0]
        if groups > 1:
            free = free[(free // each < 5) & (free // each != 1)]      # the four first groups that have any
        want = free[:k].int()
        for t in (1, 2, 3, 4):
            assert torch.equal(r.experts[t], want)
    else:
        assert int(r.experts[2, 0]) == 5
