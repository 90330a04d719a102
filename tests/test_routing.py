"""Routing, what the gate returns: a tuple of six as before there were other scores, and one that loses nothing with them."""
import copy
import pickle

import pytest
import torch

import grouped_gemm_persistent_gb300 as tg
from grouped_gemm_persistent_gb300.build import build

SIX = (torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), torch.zeros(8, dtype=torch.int32), torch.zeros(()), torch.zeros(8), True)


def test_six_entries():
    r = tg.Routing(*SIX)
    experts, weights, counts, loss, slope, renormalize = r
    assert all(p is q for p, q in zip((experts, weights, counts, loss, slope, renormalize), SIX)) and len(r) == 6
    assert (r.score, r.weight_scale, r.plain) == ("softmax", 1.0, True)
    assert r.experts is SIX[0] and r.slope is SIX[4] and r.renormalize is True
    assert len(tg.Routing(*SIX, "softmax", 1.0)) == 6
    other = r._replace(slope=SIX[3])
    assert other.slope is SIX[3] and other.experts is SIX[0] and len(other) == 6
    assert list(r._asdict()) == ["experts", "weights", "counts", "loss", "slope", "renormalize"]
    assert "renormalize=True" in repr(r) and "score" not in repr(r)


@pytest.mark.parametrize("kw", [dict(score="sigmoid"), dict(weight_scale=2.5), dict(plain=False), dict(score="sigmoid", weight_scale=2.5, plain=False)])
@pytest.mark.parametrize("again", [lambda r: tg.Routing(*r), tg.Routing._make, copy.copy, lambda r: pickle.loads(pickle.dumps(r)),
                                   lambda r: r._replace(renormalize=False), lambda r: tg.Routing(**r._asdict())])
def test_other_scores_are_not_lost(kw, again):
    r = tg.Routing(*SIX, **kw)
    want = {**dict(score="softmax", weight_scale=1.0, plain=True), **kw}
    for one in (r, again(r)):
        assert isinstance(one, tg.Routing)
        assert {name: getattr(one, name) for name in want} == want
        assert torch.equal(one.weights, SIX[1]) and len(one[:5]) == 5
    assert r._replace(score="softmax", weight_scale=1.0, plain=True).score == "softmax"
    assert f"score={want['score']!r}" in repr(r)


@pytest.mark.gpu
def test_the_gate_unpacks():
    build()
    x = torch.randn(50, 64, device="cuda")
    experts, weights, counts, loss, slope, renormalize = tg.moe_router(x, 4)
    assert experts.shape == weights.shape == (50, 4) and int(counts.sum()) == 200 and renormalize is False
    _, _, _, _, _, renormalize = tg.moe_router(x, 4, renormalize=True, groups=1, top_groups=1)
    assert renormalize is True
    dw = torch.randn(50, 4, device="cuda")
    for kw in (dict(), dict(score="sigmoid"), dict(groups=8, top_groups=3), dict(weight_scale=2.5)):
        r = tg.moe_router(x, 4, **kw)
        d = tg.moe_router_backward(x, r, dw)
        assert torch.equal(d, tg.moe_router_backward(x, tg.Routing(*r), dw))
        assert torch.equal(d, tg.moe_router_backward(x, r._replace(loss=r.loss.clone()), dw))
