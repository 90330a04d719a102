"""Outputs of the 8-bit calls and the gate belong to the stream they are written on, however it is named (GPU)."""
import pytest
import torch

import grouped_gemm_persistent_gb300 as tg

pytestmark = pytest.mark.gpu

E4 = torch.float8_e4m3fn


def calls():
    x = torch.randn(700, 1024, device="cuda").bfloat16()
    q, s = tg.quantize_fp8(x)
    b = torch.randn(2, 640, 1024, device="cuda").to(E4).transpose(1, 2)
    sb = torch.ones(2, 8, 5, device="cuda")
    counts = torch.tensor([300, 400], dtype=torch.int32, device="cuda")
    logits = torch.randn(5000, 200, device="cuda")
    r = tg.moe_router(logits, 4)
    dw = torch.randn(5000, 4, device="cuda")
    return {
        "quantize_fp8": lambda st: tg.quantize_fp8(x, stream=st)[:1],
        "gemm_fp8": lambda st: (tg.gemm_fp8(q, s, b[0], sb[0], stream=st),),
        "moe_gemm_fp8": lambda st: (tg.moe_gemm_fp8(q, s, b, sb, counts, stream=st),),
        "moe_router": lambda st: tg.moe_router(logits, 4, stream=st)[:2],
        "moe_router_backward": lambda st: (tg.moe_router_backward(logits, r, dw, stream=st),),
    }


@pytest.mark.parametrize("name", ["quantize_fp8", "gemm_fp8", "moe_gemm_fp8", "moe_router", "moe_router_backward"])
@pytest.mark.parametrize("form", ["object", "handle"])
def test_outputs_are_allocated_in_the_streams_order(name, form):
    call = calls()[name]
    want = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = call(side if form == "object" else side.cuda_stream)
    side.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # once freed, a block of the side stream is not handed out on the current one, which may be ahead of it
    for t in out:
        nbytes, at = t.untyped_storage().nbytes(), t.untyped_storage().data_ptr()
        del t
    del out, a, b
    other = [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(o.data_ptr() != at for o in other)


def test_default_stream_handles():
    call = calls()["gemm_fp8"]
    want = call(None)[0]
    for handle in (0, 1, 2):                               # NULL, the legacy and the per-thread default stream
        got = call(handle)[0]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        with torch.cuda.stream(torch.cuda.Stream()):       # allocated in the default stream's order, not this one's
            out = call(handle)[0]
            nbytes, at = out.untyped_storage().nbytes(), out.data_ptr()
            del out
            other = [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(4)]
            assert all(o.data_ptr() != at for o in other)
        torch.cuda.synchronize()
