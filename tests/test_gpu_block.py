"""Block-scaled FP8 layers and experts against the fp64 oracle.

Tolerance of an output.  The products of a block are exact in fp32; the tensor
core adds 128 of them and the kernel adds ceil(K / 128) scaled partials (plus
the ranks of a split and the bias), each addition or product within 2^-23 of
the magnitudes it adds, whatever its rounding direction.  So with A the sum of
|x w| over k, the fp32 result is within (128 + ceil(K / 128) + 16) 2^-23 A of the
exact one, and the bf16 output within half a step more, 2^-8 of the value."""

import numpy as np
import pytest
import torch

import weight_only_quantized_prologue_b200 as dq
from oracle import block as B
from oracle import formats as F

pytestmark = pytest.mark.gpu


def randn(shape, seed):
    return torch.randn(shape, generator=torch.Generator("cpu").manual_seed(seed))


def rows(M, K, seed):
    """Codes and scales of rows of unequal size, made by the oracle."""
    x = (randn((M, K), seed) * (0.2 + randn((M, 1), seed + 1).abs())).to(torch.bfloat16)
    q, s = B.quantize_rows(x.double().numpy())
    return x, q, s


def weights(E, N, K, seed):
    w = randn((E, N, K), seed).numpy() * np.exp2(np.arange(E) % 3)[:, None, None]
    qs = [B.quantize_weight(w[e]) for e in range(E)]
    return np.stack([q for q, _ in qs]), np.stack([s for _, s in qs])


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bound(q, s, wq, ws, ref, bias=None):
    A = np.abs(B.dequantize_rows(q, s)) @ np.abs(B.dequantize_weight(wq, ws)).T
    if bias is not None:
        A = A + np.abs(bias)
    return np.abs(ref) * 2.0 ** -8 + (128 + s.shape[1] + 16) * 2.0 ** -23 * A + 2.0 ** -133


def check(y, ref, b):
    err = np.abs(y.double().cpu().numpy() - ref)
    bad = ~(err <= b)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5].tolist(), float(err[bad].max()) if bad.any() else 0)


SIZES = [(1, 16, 1), (1, 128, 128), (2, 144, 7), (15, 400, 130), (16, 1024, 256), (17, 1040, 100), (33, 2064, 260),
         (64, 256, 1000), (65, 640, 384), (128, 1024, 512), (129, 144, 257), (300, 2064, 512), (257, 128, 128),
         (1, 4096, 2048), (5, 8192, 128), (100, 4096, 256)]


@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("bias", [False, True])
def test_linear_on_codes(M, K, N, bias):
    _, q, s = rows(M, K, 1)
    wq, ws = weights(1, N, K, 3)
    b = randn((N,), 5).to(torch.bfloat16) if bias else None
    lin = dq.QuantizedLinear("fp8_block", K, N, cuda(wq[0]), cuda(ws[0]), bias=None if b is None else b.cuda())
    bv = None if b is None else b.double().numpy()
    out = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    y = lin.from_codes(cuda(q), scales=cuda(s), out=out[:M])
    torch.cuda.synchronize()
    assert lin.last_error() == 0, lin.plan(M)
    ref = B.linear(q, s, wq[0], ws[0], bv)
    check(y, ref, bound(q, s, wq[0], ws[0], ref, bv))
    assert (out[M:] == 7).all()


@pytest.mark.parametrize("M,K,N", [(512, 512, 2048), (2048, 1040, 2000), (777, 4096, 1001), (4096, 256, 300)])
def test_linear_on_pairs_of_ctas(M, K, N):
    _, q, s = rows(M, K, 11)
    wq, ws = weights(1, N, K, 13)
    lin = dq.QuantizedLinear("fp8_block", K, N, cuda(wq[0]), cuda(ws[0]))
    y = lin.from_codes(cuda(q), scales=cuda(s))
    torch.cuda.synchronize()
    assert lin.last_error() == 0, lin.plan(M)
    ref = B.linear(q, s, wq[0], ws[0])
    check(y, ref, bound(q, s, wq[0], ws[0], ref))


def test_the_plan_reaches_both_kernels_and_every_tile_and_split():
    seen = set()
    for N, K in ((128, 1024), (2048, 512), (14336, 512)):
        wq = torch.zeros((N, K), dtype=torch.uint8, device="cuda")
        lin = dq.QuantizedLinear("fp8_block", K, N, wq, torch.ones((N // 128, K // 128), device="cuda"))
        for M in (1, 17, 33, 65, 129, 2048):
            p = lin.plan(M)
            seen.add((p["bn"], p["max_segments"]))
    assert {b for b, _ in seen} == {16, 32, 64, 128, 256}
    assert {s for _, s in seen} >= {1, 8}


@pytest.mark.parametrize("M", [1, 40, 300])
def test_linear_on_bf16_is_the_quantizer_and_the_product(M):
    K, N = 1040, 520
    x, q, s = rows(M, K, 21)
    wq, ws = weights(1, N, K, 23)
    lin = dq.QuantizedLinear("fp8_block", K, N, cuda(wq[0]), cuda(ws[0]))
    xc = x.cuda()
    y = lin(xc)
    ref = B.linear(q, s, wq[0], ws[0])
    check(y, ref, bound(q, s, wq[0], ws[0], ref))
    # the C entry with the handle's own workspace gives the same, also when it grows and shrinks
    for m in (1, M, 1, M):
        y2 = torch.empty((m, N), dtype=torch.bfloat16, device="cuda")
        dq.dqgemm_run(lin.handle, xc[:m].contiguous(), m, y2)
        y1 = lin(xc[:m].contiguous())
        assert torch.equal(y1, y2)


@pytest.mark.parametrize("M,K,N", [(1, 16, 1), (1, 8192, 128), (1, 2064, 14336), (3, 144, 130), (8, 4096, 512), (7, 400, 300),
                                   (8, 2064, 1000), (5, 128, 128), (9, 1040, 100), (32, 2064, 1000)])
def test_few_rows_quantized_in_the_products_kernel_give_the_same_bits(M, K, N):
    x, _, _ = rows(M, K, 25)
    wq, ws = weights(1, N, K, 27)
    b = randn((N,), 28).to(torch.bfloat16).cuda()
    lin = dq.QuantizedLinear("fp8_block", K, N, cuda(wq[0]), cuda(ws[0]), bias=b)
    assert (lin.plan(M)["workspace_bytes"] == 0) == (M <= 8)
    x[0, ::3] = 0
    x = x.cuda()
    q, s = dq.quantize_act_fp8_block(x)
    out = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    y = lin(x, out=out[:M])
    assert torch.equal(y, lin.from_codes(q, scales=s)) and (out[M:] == 7).all() and lin.last_error() == 0


@pytest.mark.parametrize("counts", [[0, 3, 0, 1], [1] * 16, [16, 0], [9, 0, 7, 0, 17, 0, 0, 0, 0, 3, 1, 0], [40, 0, 0, 2, 1, 0, 7],
                                    [0, 0, 33]], ids=str)
@pytest.mark.parametrize("K,N", [(400, 300), (1024, 128)])
def test_experts_on_bf16_give_the_bits_of_their_codes(counts, K, N):
    E, M = len(counts), sum(counts)
    x, _, _ = rows(M, K, 33)
    wq, ws = weights(E, N, K, 35)
    ex = dq.QuantizedExperts("fp8_block", E, K, N, cuda(wq), cuda(ws))
    off = cuda(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    x = x.cuda()
    q, s = dq.quantize_act_fp8_block(x)
    ref = ex.from_codes(q, s, off)
    assert torch.equal(ex(x, off), ref) and ex.last_error() == 0
    ws = torch.empty(M * (K + 4 * ((K + 127) // 128)) + 256, dtype=torch.uint8, device="cuda")
    y = torch.empty_like(ref)
    dq.dqgemm_run_fp8_block(ex.handle, x, M, off, y, ws, ws.numel())
    assert torch.equal(y, ref)
    need = ex.plan(M)["workspace_bytes"]
    assert need <= ws.numel() and (need > 0 or M <= 16)
    if need:
        with pytest.raises(dq.DQError):
            dq.dqgemm_run_fp8_block(ex.handle, x, M, off, y, ws, need - 1)


def test_packers_and_dequantize_are_bit_exact():
    N, K = 200, 336
    w = (randn((N, K), 31) * 0.1).float()
    w[:128, 128:256] = 0
    q, s = B.quantize_weight(w.double().numpy())
    hq, hs, _ = dq.dqgemm_pack_host("fp8_block", w.numpy())
    assert np.array_equal(hq, q) and np.array_equal(hs, s)
    for entry in (dq.dqgemm_pack_device, dq.dqgemm_pack_device_noalloc):
        dq_, ds = torch.empty((N, K), dtype=torch.uint8, device="cuda"), torch.empty((2, 3), device="cuda")
        assert entry("fp8_block", w.cuda(), dq_, ds) == 1.0
        assert np.array_equal(dq_.cpu().numpy(), q) and np.array_equal(ds.cpu().numpy(), s)
    lin = dq.QuantizedLinear.from_float("fp8_block", w.cuda())
    d = lin.dequantize().double().cpu().numpy()
    want = F.bf16((F.e4m3_decode(q) * np.repeat(np.repeat(s.astype(np.float64), 128, 0), 128, 1)[:N, :K]).astype(np.float32))
    assert np.array_equal(d, want)


COUNTS = [[0, 5, 0, 1, 17, 0, 64, 3], [1], [0, 0, 300], [130, 0, 1, 129], [16] * 40, [700, 20, 0, 513, 256, 257],
          [0] * 63 + [2]]


@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("K,N", [(256, 128), (400, 300), (128, 1)])
@pytest.mark.parametrize("bias", [False, True])
def test_experts(counts, K, N, bias):
    E, lead, tail = len(counts), 3, 5            # rows before the first and behind the last expert stay
    M = lead + sum(counts) + tail
    _, q, s = rows(M, K, 41)
    wq, ws = weights(E, N, K, 43)
    b = randn((E, N), 45).to(torch.bfloat16) if bias else None
    off = np.concatenate([[lead], lead + np.cumsum(counts)]).astype(np.int32)
    ex = dq.QuantizedExperts("fp8_block", E, K, N, cuda(wq), cuda(ws), bias=None if b is None else b.cuda())
    out = torch.full((M, N), 3.0, dtype=torch.bfloat16, device="cuda")
    y = ex.from_codes(cuda(q), cuda(s), cuda(off), out=out)
    torch.cuda.synchronize()
    assert ex.last_error() == 0, ex.plan(M)
    for e in range(E):
        a, z = off[e], off[e + 1]
        if z > a:
            bv = None if b is None else b[e].double().numpy()
            ref = B.linear(q[a:z], s[a:z], wq[e], ws[e], bv)
            check(y[a:z], ref, bound(q[a:z], s[a:z], wq[e], ws[e], ref, bv))
    assert (out[:lead] == 3).all() and (out[M - tail:] == 3).all()


def test_experts_clamp_offsets_outside_the_rows():
    E, K, N, M = 4, 256, 200, 37
    x, q, s = rows(M, K, 51)
    wq, ws = weights(E, N, K, 53)
    ex = dq.QuantizedExperts("fp8_block", E, K, N, cuda(wq), cuda(ws))
    off = np.array([-9, 10, 10, 30, 2 ** 31 - 1], np.int32)
    y = ex(x.cuda(), cuda(off))
    torch.cuda.synchronize()
    for e, a, z in ((0, 0, 10), (2, 10, 30), (3, 30, M)):
        ref = B.linear(q[a:z], s[a:z], wq[e], ws[e])
        check(y[a:z], ref, bound(q[a:z], s[a:z], wq[e], ws[e], ref))
    # no expert has a row (ends before starts, all of them past the end): y stays
    for off in ([37, 37, 37, 37, 37], [30, 20, 10, 5, -1], [2 ** 31 - 1] * 5):
        y2 = ex(x.cuda(), cuda(np.array(off, np.int32)), out=torch.full((M, N), 3.0, dtype=torch.bfloat16, device="cuda"))
        assert (y2 == 3).all()
    assert ex.last_error() == 0
    assert ex(x[:0].cuda(), cuda(np.zeros(5, np.int32))).shape == (0, N)


@pytest.mark.parametrize("M", [3, 50, 400])
def test_a_spoiled_row_or_block_stays_alone(M):
    # NaN and infinite activations reach their own rows only; zero scales give zeros
    K, N = 384, 300
    x, _, _ = rows(M, K, 61)
    wq, ws = weights(1, N, K, 63)
    lin = dq.QuantizedLinear("fp8_block", K, N, cuda(wq[0]), cuda(ws[0]))
    clean = lin(x.cuda())
    x[0, 5] = float("nan")
    x[2, 200] = float("inf")
    x[1] = 0
    y = lin(x.cuda())
    assert torch.isnan(y[0]).all() and torch.isnan(y[2]).all() and (y[1] == 0).all()
    assert torch.equal(y[3:], clean[3:])


def test_two_streams_at_once_and_a_replayed_graph():
    K, N, M = 2048, 1024, 48
    wq, ws = weights(1, N, K, 73)
    lin = dq.QuantizedLinear("fp8_block", K, N, cuda(wq[0]), cuda(ws[0]))
    xs = [rows(M, K, 80 + 2 * i)[0].cuda() for i in range(4)]
    refs = [lin(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for given in (False, True):
        got = []
        for rep in range(20):
            for i, x in enumerate(xs):
                st = streams[i % 2]
                if given:
                    got.append((i, lin(x, stream=st, out=torch.empty_like(refs[0]))))
                else:
                    with torch.cuda.stream(st):
                        got.append((i, lin(x)))
        torch.cuda.synchronize()
        assert all(torch.equal(y, refs[i]) for i, y in got)
    x, out = xs[0].clone(), torch.empty_like(refs[0])
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]     # two graphs on one layer
    for g in graphs:
        with torch.cuda.graph(g):
            lin(x, out=out)
    for i in (1, 2, 3):
        x.copy_(xs[i])
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(out, refs[i])


def test_offsets_change_between_replays():
    E, K, N, M = 8, 512, 384, 200
    x, q, s = rows(M, K, 91)
    wq, ws = weights(E, N, K, 93)
    ex = dq.QuantizedExperts("fp8_block", E, K, N, cuda(wq), cuda(ws))
    xc, off, out = x.cuda(), torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    ex(xc, off, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ex(xc, off, out=out)
    for cut in ([0, 200, 200, 200, 200, 200, 200, 200, 200], [0, 1, 2, 3, 100, 100, 150, 199, 200]):
        off.copy_(torch.tensor(cut, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ex(xc, off))


def test_results_do_not_change_from_call_to_call():
    for M, K, N in ((1, 4096, 512), (64, 2048, 256), (600, 1024, 2048)):
        _, q, s = rows(M, K, 95)
        wq, ws = weights(1, N, K, 97)
        lin = dq.QuantizedLinear("fp8_block", K, N, cuda(wq[0]), cuda(ws[0]))
        qc, sc = cuda(q), cuda(s)
        first = lin.from_codes(qc, scales=sc)
        for _ in range(10):
            assert torch.equal(first, lin.from_codes(qc, scales=sc))


def test_weight_codes_and_scales_outside_the_format_are_refused():
    K = N = 128
    wq, ws = weights(1, N, K, 99)
    for bad in (0x7F, 0xFF):
        w = wq[0].copy()
        w[77, 33] = bad
        with pytest.raises(dq.DQError):
            dq.QuantizedLinear("fp8_block", K, N, cuda(w), cuda(ws[0]))
    for bad in (-1.0, np.inf, np.nan):
        s = ws[0].copy()
        s[0, 0] = bad
        with pytest.raises(dq.DQError):
            dq.QuantizedLinear("fp8_block", K, N, cuda(wq[0]), cuda(s))


def test_operands_are_checked_before_the_launch():
    K, N, M = 256, 128, 4
    wq, ws = weights(2, N, K, 101)
    lin = dq.QuantizedLinear("fp8_block", K, N, cuda(wq[0]), cuda(ws[0]))
    ex = dq.QuantizedExperts("fp8_block", 2, K, N, cuda(wq), cuda(ws))
    _, q, s = rows(M, K, 103)
    q, s, off = cuda(q), cuda(s), torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="scales"):
        lin.from_codes(q)
    with pytest.raises(ValueError):
        lin.from_codes(q, scales=s[:, :1])
    with pytest.raises(TypeError):
        lin.from_codes(q, scales=s.half())
    with pytest.raises(ValueError):
        ex.from_codes(q, s, off[:2])
    with pytest.raises(TypeError):
        ex.from_codes(q, s, off.long())
    with pytest.raises(ValueError):
        ex.from_codes(q, s, off.cpu())
    with pytest.raises(dq.DQError):
        lin.quantized_out(torch.zeros((M, K), dtype=torch.bfloat16, device="cuda"), 1.0)
    with pytest.raises(ValueError):
        dq.QuantizedExperts("int4", 2, K, N, cuda(wq), cuda(ws))
    lib = dq._native.lib()
    assert lib.dqgemm_run_fp8_block_quantized(ex.handle, q.data_ptr(), s.data_ptr(), M, q.data_ptr(), None) == 2
    assert lib.dqgemm_run(ex.handle, q.data_ptr(), M, q.data_ptr(), None) == 2
    assert lib.dqgemm_run_fp8_block_quantized(lin.handle, q.data_ptr() + 1, s.data_ptr(), M, q.data_ptr(), None) == 3


def test_feed_forward_block_dense_and_by_experts():
    """norm -> gate|up -> gated SiLU -> down, 8-bit activations between the
    products, against the same chain in fp64 on the same codes.  An activation
    is off by half an e4m3 step (2^-4) where the chain's own values stand near a
    border; most are the oracle's: 2 % of the output's norm bounds what one code
    in a few hundred, 2^-4 off each, can move."""
    M, D, H, E = 96, 512, 640, 4
    x, r = randn((M, D), 111).to(torch.bfloat16), randn((M, D), 112).to(torch.bfloat16)
    w = randn((D,), 113).to(torch.bfloat16)
    up, down = weights(E, 2 * H, D, 115), weights(E, D, H, 117)
    off = np.array([0, 10, 10, 90, M], np.int32)
    q, s, r2 = dq.rmsnorm(x.cuda(), w.cuda(), 1e-5, residual=r.cuda(), quant="fp8_block")
    v, _ = B.rmsnorm(x.double().numpy(), w.double().numpy(), 1e-5, r.double().numpy())
    oq, os_ = B.quantize_rows(v)
    # dense: expert 0's weights
    l1 = dq.QuantizedLinear("fp8_block", D, 2 * H, cuda(up[0][0]), cuda(up[1][0]))
    l2 = dq.QuantizedLinear("fp8_block", H, D, cuda(down[0][0]), cuda(down[1][0]))
    hq, hs = dq.silu_mul(l1.from_codes(q, scales=s), quant="fp8_block")
    y = l2.from_codes(hq, scales=hs)
    h = F.bf16(B.linear(oq, os_, up[0][0], up[1][0]))
    gq, gs = B.quantize_rows(B.silu_mul(h))
    ref = B.linear(gq, gs, down[0][0], down[1][0])
    assert np.linalg.norm(y.double().cpu().numpy() - ref) <= 0.02 * np.linalg.norm(ref)
    # by experts
    e1 = dq.QuantizedExperts("fp8_block", E, D, 2 * H, cuda(up[0]), cuda(up[1]))
    e2 = dq.QuantizedExperts("fp8_block", E, H, D, cuda(down[0]), cuda(down[1]))
    o = cuda(off)
    hq, hs = dq.silu_mul(e1.from_codes(q, s, o), quant="fp8_block")
    y = e2.from_codes(hq, hs, o)
    h = F.bf16(B.experts(oq, os_, up[0], up[1], off))
    gq, gs = B.quantize_rows(B.silu_mul(h))
    ref = B.experts(gq, gs, down[0], down[1], off)
    assert np.linalg.norm(y.double().cpu().numpy() - ref) <= 0.02 * np.linalg.norm(ref)


@pytest.mark.parametrize("M,K,N", [(1, 4096, 512), (32, 4096, 1024), (100, 4096, 512), (1500, 2048, 4096), (16, 128, 128)])
def test_wait_limit_expires_and_the_next_call_is_right(M, K, N):
    # a limit so short that the first wait that does not complete at once gives
    # up: no output, an error to read, and a layer and context that go on
    _, q, s = rows(M, K, 121)
    wq, ws = weights(1, N, K, 123)
    lin = dq.QuantizedLinear("fp8_block", K, N, cuda(wq[0]), cuda(ws[0]))
    q, s = cuda(q), cuda(s)
    ref = lin.from_codes(q, scales=s)
    out = torch.full((M, N), 5.0, dtype=torch.bfloat16, device="cuda")
    dq.dqgemm_set_wait_limit(lin.handle, 1)
    lin.from_codes(q, scales=s, out=out)
    torch.cuda.synchronize()
    assert lin.last_error() == dq._native.DQ_ERR_TIMEOUT, lin.plan(M)
    # a tile is written whole or not at all
    o = out.float()
    assert ((o == 5) | (o == ref.float())).all()
    dq.dqgemm_set_wait_limit(lin.handle, 0)
    assert torch.equal(lin.from_codes(q, scales=s, out=out), ref)
    torch.cuda.synchronize()
    assert lin.last_error() == 0


@pytest.mark.parametrize("counts", [[3, 0, 9], [300, 20, 700, 0]], ids=str)
def test_experts_wait_limit_expires(counts):
    E, K, N, M = len(counts), 1024, 512, sum(counts)
    x, q, s = rows(M, K, 125)
    wq, ws = weights(E, N, K, 127)
    ex = dq.QuantizedExperts("fp8_block", E, K, N, cuda(wq), cuda(ws))
    off = cuda(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    q, s = cuda(q), cuda(s)
    ref = ex.from_codes(q, s, off)
    dq.dqgemm_set_wait_limit(ex.handle, 1)
    ex.from_codes(q, s, off)
    ex(x.cuda(), off)
    torch.cuda.synchronize()
    assert ex.last_error() == dq._native.DQ_ERR_TIMEOUT
    dq.dqgemm_set_wait_limit(ex.handle, 0)
    assert torch.equal(ex.from_codes(q, s, off), ref)
    assert torch.equal(ex(x.cuda(), off), ref)
    torch.cuda.synchronize()
    assert ex.last_error() == 0


def test_offsets_past_32_bits():
    # 4.6e9 weight bytes: the last experts' rows lie past 2^32
    E, N, K, M = 70, 8192, 8192, 6
    ex = dq.QuantizedExperts("fp8_block", E, K, N, torch.full((E, N, K), 0x38, dtype=torch.uint8, device="cuda"),
                             torch.arange(1, E + 1, device="cuda", dtype=torch.float32)[:, None, None].expand(E, 64, 64).contiguous())
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = 2
    off[E - 1:] = 4
    off[E] = 6
    x = torch.ones((M, K), dtype=torch.bfloat16, device="cuda")
    y = ex(x, off.cuda()).float().cpu()        # 1.0 = code 0x38: y = K * expert
    want = torch.tensor([1, 1, E - 1, E - 1, E, E]).float()[:, None] * K
    assert (y == want.to(torch.bfloat16).float()).all()
    ex.close()
    # 2.5e9 outputs
    M, N, K = 150016, 16384, 128
    wq, ws = weights(1, 256, K, 131)
    wide = cuda(wq[0]).repeat(N // 256, 1)
    lin = dq.QuantizedLinear("fp8_block", K, N, wide, cuda(ws[0]).repeat(N // 256, 1))
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    tail, q, s = rows(5, K, 133)
    x[-5:] = tail.cuda()
    y = lin(x)
    ref = B.linear(q, s, wq[0], ws[0])
    check(y[-5:, -256:], ref, bound(q, s, wq[0], ws[0], ref))
    assert not y[:-5:997].any() and torch.equal(y[-5:, :256], y[-5:, -256:])


def test_static_codes_of_the_row_operators_feed_a_static_layer():
    K, N, M = 512, 256, 40
    torch.manual_seed(3)
    w = torch.randn(N, K, device="cuda") * 0.05
    x, r = randn((M, K), 141).to(torch.bfloat16).cuda(), randn((M, K), 142).to(torch.bfloat16).cuda()
    lin = dq.QuantizedLinear.from_float("fp8_static", w, act_scale=0.01)
    q, _ = dq.rmsnorm(x, residual=r, quant="fp8_static", s_out=0.01)
    n, _ = dq.rmsnorm(x, residual=r)
    y, y2 = lin.from_codes(q), lin(n)               # the second rounds the norm to bf16 first
    assert (y.float() - y2.float()).norm() <= 0.02 * y2.float().norm()
    g = torch.cat([x, r], 1)
    y, y2 = lin.from_codes(dq.silu_mul(g, quant="fp8_static", s_out=0.01)), lin(dq.silu_mul(g))
    assert (y.float() - y2.float()).norm() <= 0.02 * y2.float().norm()


def test_quantize_replaces_linears_by_block_scaled_ones():
    from weight_only_quantized_prologue_b200 import module as Mod

    torch.manual_seed(5)
    model = torch.nn.Sequential(torch.nn.Linear(256, 384), torch.nn.ReLU(), torch.nn.Linear(384, 64))
    model = model.to(device="cuda", dtype=torch.bfloat16)
    w = [(m.weight.float(), m.bias.detach()) for m in (model[0], model[2])]
    l1, l2 = (dq.QuantizedLinear.from_float("fp8_block", a, b) for a, b in w)
    Mod.quantize_(model, "fp8_block")
    x = randn((3, 7, 256), 151).to(torch.bfloat16).cuda()
    with torch.no_grad():
        y = model(x)
    assert torch.equal(y, l2(torch.relu(l1(x.view(-1, 256)))).view(3, 7, 64))


@pytest.mark.parametrize("E,N,K", [(3, 128, 128), (3, 384, 128), (4, 384, 1152), (5, 200, 336), (3, 1, 16), (2, 256, 256)])
def test_experts_from_float_at_any_count_of_blocks(E, N, K):
    w = (randn((E, N, K), 161) * 0.1).float()
    ex = dq.QuantizedExperts.from_float("fp8_block", w.cuda())
    d = ex.dequantize().double().cpu().numpy()
    for e in range(E):
        q, s = B.quantize_weight(w[e].double().numpy())
        wide = np.repeat(np.repeat(s.astype(np.float64), 128, 0), 128, 1)[:N, :K]
        assert np.array_equal(d[e], F.bf16((F.e4m3_decode(q) * wide).astype(np.float32)))
    M = 2 * E
    x, xq, xs = rows(M, K, 163)
    y = ex(x.cuda(), torch.arange(0, M + 1, 2, dtype=torch.int32, device="cuda"))
    for e in range(E):
        q, s = B.quantize_weight(w[e].double().numpy())
        a, z = 2 * e, 2 * e + 2
        ref = B.linear(xq[a:z], xs[a:z], q, s)
        check(y[a:z], ref, bound(xq[a:z], xs[a:z], q, s, ref))
