"""The norm, the gate and the adapters called by several threads at once, each on a stream of its own: the results of one after the
other (GPU)."""
import threading

import pytest
import torch

import grouped_gemm_persistent_gb300 as tg
import test_lora
import test_residual_norm
import test_router_scored
from grouped_gemm_persistent_gb300.build import build

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def norm(seed, M, K):
    x, residual, gain = test_residual_norm.make(seed, M, K, BF, BF, F)

    def call():
        n = tg.rmsnorm(x, gain, residual=residual, fp8_dtype=torch.float8_e4m3fn)
        dx, d_gain = tg.rmsnorm_backward(n, x, gain, residual)
        return n.y, n.q.view(torch.uint8), n.scale, n.hidden, n.row_scale, dx, d_gain
    return call


def gate(seed, T, G, groups):
    x, bias, dw = test_router_scored.make(seed, T, G, F)
    dw = dw[:, :6].contiguous()

    def call():
        r = tg.moe_router(x, 6, renormalize=True, score="sigmoid", bias=bias, groups=groups, top_groups=2 if groups > 1 else 1)
        return *r[:5], tg.moe_router_backward(x, r, dw, r.loss)
    return call


def adapters(seed, T, G, r):
    base, x, a, b, ids, scale = test_lora.make(seed, T, 264, 136, r, G, BF, BF, "rows")
    return lambda: (tg.lora_add(base, x, a, b, ids, scale),)


def test_calls_of_several_threads():
    """Sizes on either side of what a kernel has of shared memory without asking, of the rows' and tiles' forms, of one cluster and many
    blocks, in another order in each thread."""
    build()
    calls = [norm(80, 300, 32768), norm(81, 300, 16400), norm(82, 500, 12200), norm(83, 40, 4096), gate(84, 64, 256, 8),
             gate(85, 3000, 1000, 8), gate(86, 2000, 96, 6), adapters(87, 20, 5, 16), adapters(88, 5000, 370, 8), adapters(89, 4500, 700, 40)]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(4)

    def work(n):
        try:
            start.wait()
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for turn in range(6):
                    order = torch.randperm(len(calls), generator=torch.Generator().manual_seed(10 * n + turn)).tolist()
                    got = {i: calls[i]() for i in order}
                    stream.synchronize()
                    wrong.extend((n, i) for i in order if not all(torch.equal(p, q) for p, q in zip(got[i], want[i])))
        except Exception as e:                      # (it would end with its thread)
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(n,)) for n in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == []
    tg.device_status()
