"""What a row's result with its adapter depends on: not on the other rows, and on the batch's size in its last bits alone (GPU)."""
import pytest
import torch

import grouped_gemm_persistent_gb300 as tg
from test_lora import BF, F, HF, check, lib, make  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]


@pytest.mark.parametrize("T", [1, 64, 700, 5000])
@pytest.mark.parametrize("r", [16, 40])
@pytest.mark.parametrize("dt", [BF, HF])
def test_other_rows_do_not_enter(T, r, dt):
    """The same rows in a batch of the same size, all others and their adapters changed: the same bits."""
    base, x, a, b, ids, scale = make(70, T, 1100, 264, r, 6, dt, F, "rows")
    keep = torch.arange(T, device="cuda") % 5 == 0
    want = tg.lora_add(base, x, a, b, ids, scale)
    base2, x2, _, _, ids2, _ = make(71, T, 1100, 264, r, 6, dt, F, "requests")
    base2[keep], x2[keep], ids2[keep] = base[keep], x[keep], ids[keep]
    x2[~keep] *= 100
    assert torch.equal(tg.lora_add(base2, x2, a, b, ids2, scale)[keep], want[keep])


@pytest.mark.parametrize("r", [16, 40])
@pytest.mark.parametrize("dt", [BF, HF])
def test_alone_and_in_larger_batches(r, dt):
    """A row by itself, among 100 and among 5000, and with more adapters loaded: each within the bound of its sums."""
    base, x, a, b, ids, scale = make(72, 5000, 1100, 264, r, 200, dt, F, "rows")
    ids[0] = 3
    for T in (1, 100, 5000):
        for G in (6, 200):
            part = torch.where(ids[:T] < G, ids[:T], -1)
            check(base[:T], x[:T], a[:G], b[:G], part, scale[:G], tg.lora_add(base[:T], x[:T], a[:G], b[:G], part, scale[:G]))
