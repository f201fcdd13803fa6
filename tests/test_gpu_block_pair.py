"""The CTA-pair kernel of block-scaled FP8 layers, at sizes whose plan is that
kernel (asserted), against the fp64 oracle with the bound of test_gpu_block."""

import numpy as np
import pytest
import torch

import weight_only_quantized_prologue_b200 as dq
from oracle import block as B
from test_gpu_block import bound, check, cuda, randn, rows, weights

pytestmark = pytest.mark.gpu


def layer(M, K, N, seed, bias=False):
    wq, ws = weights(1, N, K, seed)
    b = randn((N,), seed + 1).to(torch.bfloat16) if bias else None
    lin = dq.QuantizedLinear("fp8_block", K, N, cuda(wq[0]), cuda(ws[0]), bias=None if b is None else b.cuda())
    assert lin.plan(M)["bn"] == 256, lin.plan(M)
    return lin, wq[0], ws[0], None if b is None else b.double().numpy()


# one block of K and many; whole tiles, rows and channels that end inside one;
# the tile's second 128 channels cut (N % 256 > 128) or absent; N a multiple
# of 8 (rows leave by bulk copies) or not; one tile a pair and several
SIZES = [(2048, 128, 2048), (2057, 400, 2001), (2100, 272, 1928), (2300, 144, 1900), (2300, 2064, 1888), (4500, 128, 1000),
         (9000, 640, 500), (5000, 640, 2500), (18900, 16, 129)]


@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("bias", [False, True])
def test_linear_on_pairs(M, K, N, bias):
    _, q, s = rows(M, K, 201)
    lin, wq, ws, bv = layer(M, K, N, 203, bias)
    out = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    if N % 8:
        y = lin.from_codes(cuda(q), scales=cuda(s))
    else:
        y = lin.from_codes(cuda(q), scales=cuda(s), out=out[:M])
    torch.cuda.synchronize()
    assert lin.last_error() == 0 and (out[M:] == 7).all()
    ref = B.linear(q, s, wq, ws, bv)
    check(y, ref, bound(q, s, wq, ws, ref, bv))


@pytest.mark.parametrize("M,K,N", [(5000, 640, 2500), (2057, 2064, 2001), (9000, 128, 1024)])
def test_results_do_not_change_from_call_to_call(M, K, N):
    _, q, s = rows(M, K, 211)
    lin, *_ = layer(M, K, N, 213, True)
    q, s = cuda(q), cuda(s)
    first = lin.from_codes(q, scales=s)
    out = torch.empty_like(first)
    for i in range(200):
        out.fill_(float("nan"))
        assert torch.equal(first, lin.from_codes(q, scales=s, out=out)), i
    assert lin.last_error() == 0


def test_spoiled_rows_stay_alone():
    M, K, N = 2300, 384, 1900
    x, _, _ = rows(M, K, 221)
    lin, *_ = layer(M, K, N, 223)
    clean = lin(x.cuda())
    x[7, 5] = float("nan")
    x[1300, 200] = float("inf")
    x[2299] = 0
    y = lin(x.cuda())
    assert torch.isnan(y[7]).all() and torch.isnan(y[1300]).all() and (y[2299] == 0).all()
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[[7, 1300, 2299]] = False
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("M,K,N", [(2057, 2064, 2001), (5000, 640, 2500), (2048, 128, 2048)])
def test_wait_limit_expires_and_the_next_call_is_right(M, K, N):
    """What a call leaves whose waits gave up: elements as they were or right."""
    _, q, s = rows(M, K, 231)
    lin, *_ = layer(M, K, N, 233)
    q, s = cuda(q), cuda(s)
    ref = lin.from_codes(q, scales=s)
    for limit in (1, 2000, 20000):
        for _ in range(5):
            dq.dqgemm_set_wait_limit(lin.handle, limit)
            out = torch.full((M, N), 5.0, dtype=torch.bfloat16, device="cuda")
            lin.from_codes(q, scales=s, out=out)
            torch.cuda.synchronize()
            err = lin.last_error()
            assert err in (0, dq._native.DQ_ERR_TIMEOUT) and (err or limit > 1)
            assert ((out == 5) | (out == ref)).all() and (err or torch.equal(out, ref))
            dq.dqgemm_set_wait_limit(lin.handle, 0)
            assert torch.equal(lin.from_codes(q, scales=s, out=out), ref)
            torch.cuda.synchronize()
            assert lin.last_error() == 0


def test_many_experts_and_rows_on_one_of_them():
    # as many experts as a handle takes, and all rows of a call on one or two of a few
    E, K, N, M = 1024, 128, 136, 300
    wq, ws = weights(E, N, K, 241)
    ex = dq.QuantizedExperts("fp8_block", E, K, N, cuda(wq), cuda(ws))
    _, q, s = rows(M, K, 243)
    counts = np.zeros(E, np.int64)
    counts[[0, 1, 31, 32, 500, 1022, 1023]] = [1, 100, 2, 64, 33, 65, 35]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    y = ex.from_codes(cuda(q), cuda(s), cuda(off))
    for e in np.nonzero(counts)[0]:
        a, z = off[e], off[e + 1]
        ref = B.linear(q[a:z], s[a:z], wq[e], ws[e])
        check(y[a:z], ref, bound(q[a:z], s[a:z], wq[e], ws[e], ref))
    E, K, N, M = 8, 384, 520, 1000
    wq, ws = weights(E, N, K, 245)
    ex = dq.QuantizedExperts("fp8_block", E, K, N, cuda(wq), cuda(ws))
    assert ex.plan(M)["bn"] == 256
    _, q, s = rows(M, K, 247)
    for counts in ([0, 0, 0, 1000, 0, 0, 0, 0], [999, 0, 0, 0, 0, 0, 0, 1]):
        off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        y = ex.from_codes(cuda(q), cuda(s), cuda(off))
        assert ex.last_error() == 0
        for e in np.nonzero(counts)[0]:
            a, z = off[e], off[e + 1]
            ref = B.linear(q[a:z], s[a:z], wq[e], ws[e])
            check(y[a:z], ref, bound(q[a:z], s[a:z], wq[e], ws[e], ref))
