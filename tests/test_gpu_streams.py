"""Calls on another stream than the current one: what they allocate is that
stream's memory, results and temporaries, so that no work still queued on the
current stream holds it and none there gets it while the call runs."""

import pytest
import torch

import weight_only_quantized_prologue_b200 as dq

pytestmark = pytest.mark.gpu


def stream_of(t):
    """The stream whose memory t lies in, by the allocator's own account."""
    p = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= p < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's")


@pytest.fixture(params=["stream", "address"])
def given(request):
    st = torch.cuda.Stream()
    yield st if request.param == "stream" else st.cuda_stream, st
    torch.cuda.synchronize()


def calls():
    K, N, M = 256, 128, 40
    x = torch.randn(M, K, device="cuda").to(torch.bfloat16)
    w = torch.randn(N, K, device="cuda")
    blk = dq.QuantizedLinear.from_float("fp8_block", w)
    sta = dq.QuantizedLinear.from_float("fp8_static", w, act_scale=0.01)
    i4 = dq.QuantizedLinear.from_float("int4", w)
    ex = dq.QuantizedExperts.from_float("fp8_block", w.repeat(3, 1, 1))
    off = torch.tensor([0, 10, 10, M], dtype=torch.int32, device="cuda")
    q, s = dq.quantize_act_fp8_block(x)
    big = x.repeat(10, 1)                  # static FP8: quantized ahead, into a temporary
    return [
        lambda st: blk(x, stream=st), lambda st: blk.from_codes(q, scales=s, stream=st), lambda st: blk.dequantize(stream=st),
        lambda st: ex(x, off, stream=st), lambda st: ex.from_codes(q, s, off, stream=st), lambda st: ex.dequantize(stream=st),
        lambda st: sta(big, stream=st), lambda st: sta.quantized_out(big, 0.02, stream=st), lambda st: sta.quantized_out(x, 0.02, stream=st),
        lambda st: i4(x, stream=st), lambda st: i4.dequantize(stream=st),
        lambda st: dq.rmsnorm(x, residual=x, quant="fp8_block", stream=st), lambda st: dq.rmsnorm(x, stream=st),
        lambda st: dq.silu_mul(x, stream=st), lambda st: dq.silu_mul(x, quant="fp8_static", s_out=0.1, stream=st),
        lambda st: dq.quantize_act_fp8_block(x, stream=st),
    ]


def test_results_are_memory_of_the_calls_stream(given):
    arg, st = given
    fns = calls()
    torch.cuda.synchronize()
    for i, f in enumerate(fns):
        ref, got = f(None), f(arg)
        torch.cuda.synchronize()
        for r, g in zip(*((t if isinstance(t, tuple) else (t,)) for t in (ref, got))):
            assert stream_of(g) == st.cuda_stream, i
            assert stream_of(r) == 0 and torch.equal(r, g), i


def test_temporaries_are_memory_of_the_calls_stream(given):
    arg, st = given
    K, N, M = 512, 256, 4096
    w = torch.randn(N, K, device="cuda")
    x = torch.randn(M, K, device="cuda").to(torch.bfloat16)
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    for lin in (dq.QuantizedLinear.from_float("fp8_static", w, act_scale=0.01), dq.QuantizedLinear.from_float("fp8_block", w)):
        torch.cuda.synchronize()
        held = torch.cuda.memory_stats()["allocation.all.allocated"]
        before = {s["address"] for s in torch.cuda.memory_snapshot()}
        lin(x, out=out, stream=arg)
        torch.cuda.synchronize()
        assert torch.cuda.memory_stats()["allocation.all.allocated"] == held + 1
        new = [s for s in torch.cuda.memory_snapshot() if s["address"] not in before]
        # a stream that has no memory yet gets a segment of its own for it
        assert all(s["stream"] == st.cuda_stream for s in new) and (new or lin.fmt != "fp8_static")


def test_the_default_stream_by_its_address():
    x = torch.randn(4, 256, device="cuda")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        y = dq.rmsnorm(x, stream=0)
    torch.cuda.synchronize()
    assert stream_of(y) == 0 and torch.equal(y, dq.rmsnorm(x))
