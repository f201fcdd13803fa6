"""One layer, one set of experts and the row operators called from several host
threads at once, their first calls among them; and first calls that a graph captures."""

import subprocess
import sys
import threading
from pathlib import Path

import pytest
import torch

import weight_only_quantized_prologue_b200 as dq

pytestmark = pytest.mark.gpu


def test_first_calls_from_many_threads():
    K, N, E = 1024, 640, 4
    w = torch.randn(E, N, K, device="cuda")
    xs = [torch.randn(M, K, device="cuda").to(torch.bfloat16) for M in (1, 7, 16, 33, 64, 100, 200, 700)]
    offs = [torch.tensor([0, x.shape[0] // 2, x.shape[0] // 2, x.shape[0], x.shape[0]], dtype=torch.int32, device="cuda") for x in xs]

    def run(lin, ex, i):
        x = xs[i % len(xs)]
        q, s, r = dq.rmsnorm(x, residual=x, quant="fp8_block")
        return [lin(x), lin.from_codes(q, scales=s), ex(x, offs[i % len(xs)]), dq.silu_mul(x), q, s, r]

    make = lambda: (dq.QuantizedLinear.from_float("fp8_block", w[0]), dq.QuantizedExperts.from_float("fp8_block", w))  # noqa: E731
    lin, ex = make()
    refs = [run(lin, ex, i) for i in range(len(xs))]
    torch.cuda.synchronize()
    for _ in range(3):
        lin, ex = make()                    # nothing known to the new handles yet
        got, bad = [None] * 16, []
        start = threading.Barrier(16)

        def work(i):
            try:
                st = torch.cuda.Stream()
                start.wait()
                with torch.cuda.stream(st):
                    for k in range(10):
                        got[i] = run(lin, ex, i + k)
                st.synchronize()
            except Exception as e:  # noqa: BLE001
                bad.append(e)

        threads = [threading.Thread(target=work, args=(i,)) for i in range(16)]
        [t.start() for t in threads]
        [t.join() for t in threads]
        assert not bad, bad
        for i in range(16):
            assert all(torch.equal(a, b) for a, b in zip(got[i], refs[(i + 9) % len(xs)]))
        assert lin.last_error() == 0 and ex.last_error() == 0


CAPTURE = """
import torch
import weight_only_quantized_prologue_b200 as dq
x = torch.randn(40, 512, device="cuda").to(torch.bfloat16)
w = torch.randn(3, 256, 512, device="cuda")
lin, ex = dq.QuantizedLinear.from_float("fp8_block", w[0]), dq.QuantizedExperts.from_float("fp8_block", w)
off = torch.tensor([0, 10, 10, 40], dtype=torch.int32, device="cuda")
def run():
    q, s, r = dq.rmsnorm(x, residual=x, quant="fp8_block")
    return [q, s, r, lin(x), lin.from_codes(q, scales=s), ex(x, off), ex.from_codes(q, s, off), dq.silu_mul(x),
            *dq.silu_mul(x, quant="fp8_block"), *dq.quantize_act_fp8_block(x), lin(x[:3].contiguous())]
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = run()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, run()))
print("captured")
"""


def test_first_calls_may_be_captured():
    r = subprocess.run([sys.executable, "-c", CAPTURE], cwd=Path(__file__).resolve().parent.parent, capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
