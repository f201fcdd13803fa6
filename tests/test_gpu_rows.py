"""The row operators (RMS norm with residual, gated SiLU, block-scaled FP8
quantizer) against the fp64 oracle.

Tolerances.  u = 2^-24 is half a step of fp32.  A row's sum of squares takes at
most K / 4096 + 7 fused multiply-adds in turn per element slot of a thread (8
of them a vector) and 9 additions across threads, each within u of its value,
so its square root is within (8 (K / 4096 + 1) + 9) / 2 + 1 of u; the residual's
sum, the reciprocal root (2 units of 2^-23), and two products add 8 u.  The
gated SiLU's hardware exponential is within 2 + 1.16 |g| units of 2^-23 and its
division within 2.  Every output then carries half a step of its type, with an
absolute part below the type's smallest normal; for a code the half step is
2^-4 of the value, or 2^-10 scales below 2^-6 scales."""

import numpy as np
import pytest
import torch

import weight_only_quantized_prologue_b200 as dq
from oracle import block as B
from oracle import formats as F

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}   # half the subnormal spacing


def gen(shape, seed, dt, scale=1.0):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(DT[dt]).cuda()


def f64(t):
    return t.double().cpu().numpy()


def norm_rel(K):
    return ((8 * (K / 4096 + 1) + 9) / 2 + 9) * U


def check_float(y, ref, dt, rel):
    bound = np.abs(ref) * (rel + HALF[dt]) + TINY[dt] + 2.0 ** -149
    bad = ~(np.abs(f64(y) - ref) <= bound)
    assert not bad.any(), (bad.sum(), np.abs(f64(y) - ref).max())


def check_codes(q, s, ref, rel):
    """Codes and scales against the unquantized fp64 values, each within rel."""
    q, s = q.cpu().numpy(), s.cpu().numpy()
    M, K = ref.shape
    pad = np.zeros((M, s.shape[1] * 128))
    pad[:, :K] = np.abs(ref)
    amax = pad.reshape(M, -1, 128).max(2)
    sw = s.astype(np.float64)
    assert (np.abs(sw - amax / 448) <= amax / 448 * (rel + 2 * U) + 2.0 ** -149).all()
    wide = np.repeat(sw, 128, 1)[:, :K]
    got = F.e4m3_decode(q) * wide
    bound = np.maximum(np.abs(ref) * 2.0 ** -4, wide * 2.0 ** -10) * 1.0001 + np.abs(ref) * (2 * rel + 4 * U) + 2.0 ** -148
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), bad.sum()


SIZES = [(1, 1), (3, 7), (2, 8), (5, 120), (1, 128), (4, 136), (9, 257), (130, 1000), (17, 2048), (33, 4096),
         (7, 5008), (2, 8200), (3, 16384), (2, 20008), (1, 40001)]


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_quantizer_is_bit_exact(M, K, dt):
    x = gen((M, K), 1, dt, 3.0)
    x.view(-1)[::7] *= -0.0                         # zeros of both signs keep them
    q, s = dq.quantize_act_fp8_block(x)
    rq, rs = B.quantize_rows(f64(x))
    assert np.array_equal(s.cpu().numpy().view(np.uint32), rs.view(np.uint32))
    assert np.array_equal(q.cpu().numpy(), rq)


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("dt,odt", [("bf16", None), ("fp16", None), ("fp32", None), ("fp32", "bf16"), ("bf16", "fp32")])
@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm_float_outputs(M, K, dt, odt, residual):
    x, w = gen((M, K), 2, dt, 2.0), gen((K,), 3, dt)
    r = gen((M, K), 4, dt, 2.0) if residual else None
    got = dq.rmsnorm(x, w, 1e-5, residual=r, out_dtype=None if odt is None else DT[odt])
    ref, rsum = B.rmsnorm(f64(x), f64(w), 1e-5, None if r is None else f64(r))
    y = got[0] if residual else got
    assert y.dtype == DT[odt or dt]
    check_float(y, ref, odt or dt, norm_rel(K))
    if residual:
        check_float(got[1], rsum, dt, U)


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_rmsnorm_block_codes(M, K, dt):
    x, w, r = gen((M, K), 5, dt), gen((K,), 6, dt), gen((M, K), 7, dt)
    q, s, r2 = dq.rmsnorm(x, w, residual=r, quant="fp8_block")
    ref, rsum = B.rmsnorm(f64(x), f64(w), 1e-6, f64(r))
    check_codes(q, s, ref, norm_rel(K))
    check_float(r2, rsum, dt, U)
    # the codes are those of the fp32 norm
    y, _ = dq.rmsnorm(x, w, residual=r, out_dtype=torch.float32)
    q2, s2 = dq.quantize_act_fp8_block(y)
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("wdt", ["bf16", "fp16", "fp32", None])
def test_rmsnorm_weight_types_and_static_codes(wdt):
    M, K = 19, 1048
    x = gen((M, K), 8, "bf16")
    w = None if wdt is None else gen((K,), 9, wdt)
    s_out = 0.0123
    q = dq.rmsnorm(x, w, quant="fp8_static", s_out=s_out)
    y = dq.rmsnorm(x, w, out_dtype=torch.float32)
    t = (f64(y) / np.float64(np.float32(s_out))).astype(np.float32).astype(np.float64)
    assert np.array_equal(q.cpu().numpy(), F.e4m3_encode(F.e4m3_round(t)))


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("dt,odt", [("bf16", None), ("fp16", None), ("fp32", None), ("bf16", "fp32")])
def test_silu_mul_float_outputs(M, K, dt, odt):
    x = gen((M, 2 * K), 10, dt, 2.0)
    y = dq.silu_mul(x, out_dtype=None if odt is None else DT[odt])
    g = np.abs(f64(x)[:, :K])
    check_float(y, B.silu_mul(f64(x)), odt or dt, (8 + 1.2 * g) * 2.0 ** -23)


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_silu_mul_codes(M, K, dt):
    x = gen((M, 2 * K), 11, dt, 2.0)
    ref = B.silu_mul(f64(x))
    rel = float((8 + 1.2 * np.abs(f64(x)[:, :K]).max()) * 2.0 ** -23)
    q, s = dq.silu_mul(x, quant="fp8_block")
    check_codes(q, s, ref, rel)
    s_out = 0.031
    got = F.e4m3_decode(dq.silu_mul(x, quant="fp8_static", s_out=s_out).cpu().numpy()) * np.float64(np.float32(s_out))
    want = np.clip(ref, -448 * s_out, 448 * s_out)
    bound = np.maximum(np.abs(want) * 2.0 ** -4, s_out * 2.0 ** -10) * 1.0001 + np.abs(want) * (2 * rel + 4 * U)
    assert (np.abs(got - want) <= bound).all()


def test_silu_mul_at_the_ends_of_the_exponential():
    # e^-g overflows below -88: the result tends to 0 with g's sign; large g gives g * u
    g = torch.tensor([[-1e4, -120.0, -89.0, -0.0, 0.0, 89.0, 1e4, 3e38]])
    x = torch.cat([g, torch.full_like(g, 2.0)], 1).cuda()
    for dt in (torch.float32, torch.bfloat16):
        y = dq.silu_mul(x, out_dtype=dt)[0].float().cpu()
        assert (y[:3].abs() < 1e-30).all() and (y[3:5] == 0).all()
        assert torch.allclose(y[5:7], torch.tensor([178.0, 2e4]), rtol=2 ** -7) and y[7] == float("inf")


def test_strided_rows_and_given_outputs():
    M, K = 21, 384
    wide = gen((M, 3 * K + 8), 12, "bf16")
    for at in (0, 8, K, K + 3):                    # an offset of 3 leaves the vector path
        x = wide[:, at:at + K]
        q, s = dq.quantize_act_fp8_block(x)
        q2, s2 = dq.quantize_act_fp8_block(x.contiguous())
        assert torch.equal(q, q2) and torch.equal(s, s2)
        assert torch.equal(dq.rmsnorm(x), dq.rmsnorm(x.contiguous()))
        x2 = wide[:, at:at + 2 * K]
        assert torch.equal(dq.silu_mul(x2), dq.silu_mul(x2.contiguous()))
    x, r = gen((M, K), 13, "bf16"), gen((M, K), 14, "bf16")
    ref = dq.rmsnorm(x, residual=r, quant="fp8_block")
    out, sc = torch.empty((M, K), dtype=torch.uint8, device="cuda"), torch.empty((M, 3), device="cuda")
    got = dq.rmsnorm(x, residual=r, quant="fp8_block", out=out, scales=sc, residual_out=r)   # in place
    assert got[0] is out and got[1] is sc and got[2] is r
    for a, b in zip(ref, got):
        assert torch.equal(a, b)
    # many rows a CTA, the new residual in the place of x
    x, r = gen((5000, 520), 20, "bf16"), gen((5000, 520), 21, "bf16")
    ref = dq.rmsnorm(x, residual=r)
    got = dq.rmsnorm(x, residual=r, residual_out=x)
    assert got[1] is x and all(torch.equal(a, b) for a, b in zip(ref, got))


@pytest.mark.parametrize("dt,odt", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp16"), ("fp32", "fp32"), ("bf16", "fp8_block")])
@pytest.mark.parametrize("K", [1, 3, 7, 15, 17, 129, 511, 515, 1031, 4100])
def test_rows_that_start_anywhere(dt, odt, K):
    """Every offset of each buffer from a 16-byte boundary gives the same bits,
    and nothing beside the outputs is written."""
    M, gap = 3, 5
    quant = odt if odt == "fp8_block" else None
    ot = torch.uint8 if quant else DT[odt]
    xv, rv, w = gen((M, 2 * K), 1, dt), gen((M, K), 2, dt), gen((K,), 3, dt)

    def place(v, at, ld):                      # v [M, cols] with rows ld apart, `at` elements into its buffer
        buf = torch.full((at + ld * M,), 9.0, dtype=v.dtype, device="cuda")
        view = buf.as_strided(v.shape, (ld, 1), at)
        view.copy_(v)
        return view

    def empty(t, at):                          # [M, K] inside a buffer of a known value
        buf = torch.full((at + M * K + 40,), 77, dtype=t, device="cuda")
        return buf, buf[at:at + M * K].view(M, K)

    first = None
    for at in range(17):
        x, g = place(xv[:, :K], at, K + gap), place(xv, at, 2 * K + gap)
        res = place(rv, (3 * at) % 17, K)
        wt = place(w.view(1, K), (5 * at) % 17, K).view(K)
        outs = [empty(ot, (7 * at) % 17), empty(ot, (11 * at) % 17), empty(DT[dt], at)]
        kw = dict(quant=quant) if quant else dict(out_dtype=ot)
        got = dq.rmsnorm(x, wt, residual=res, out=outs[0][1], residual_out=outs[2][1], **kw)
        gate = dq.silu_mul(g, out=outs[1][1], **kw)
        all_ = list(got) + (list(gate) if quant else [gate])
        same = dq.rmsnorm(x, wt, residual=res, residual_out=res, **kw)   # in place
        all_ += list(same)
        if quant:
            all_ += list(dq.quantize_act_fp8_block(x, out=empty(ot, at)[1]))
        bits = [t.contiguous().clone().view(torch.uint8) for t in all_]
        for (buf, view), o in zip(outs, ((7 * at) % 17, (11 * at) % 17, at)):
            assert (buf[:o] == 77).all() and (buf[o + M * K:] == 77).all()
        if first is None:
            first = bits
        for a, b in zip(first, bits):
            assert torch.equal(a, b)


@pytest.mark.parametrize("K", [256, 200])
def test_special_values(K):
    x = gen((6, K), 15, "fp32")
    x[0] = 0
    x[1, 130] = float("nan")
    x[2, 3] = float("inf")
    x[3, :128] = 1e-45                              # amax / 448 underflows: scale and codes 0
    x[4, :128] = 1e-40                              # a subnormal scale
    x[5, :128] = 3e38
    q, s = dq.quantize_act_fp8_block(x)
    v = F.e4m3_decode(q.cpu().numpy())
    s = s.cpu().numpy()
    assert (v[0] == 0).all() and (s[0] == 0).all()
    assert np.isnan(s[1, 1]) and np.isnan(v[1, 128:]).all() and np.isfinite(v[1, :128]).all()
    assert np.isinf(s[2, 0]) and np.isnan(v[2, 3]) and (np.delete(v[2, :128], 3) == 0).all()
    assert s[3, 0] == 0 and (v[3, :128] == 0).all()
    xs = x.double().cpu().numpy()
    for row in (4, 5):
        rq, rs = B.quantize_rows(xs[row:row + 1])
        assert np.array_equal(s[row], rs[0]) and np.array_equal(q.cpu().numpy()[row], rq[0])
    # a NaN or an infinity spoils its own row of the norm only
    y = dq.rmsnorm(x, eps=1e-6).cpu()
    assert (y[0] == 0).all() and torch.isnan(y[1]).all() and torch.isnan(y[2, 3]) and torch.isfinite(y[3:5]).all()


@pytest.mark.parametrize("op,dt", [("norm", "bf16"), ("norm", "fp32"), ("gate", "bf16"), ("gate", "fp32")])
def test_few_codes_differ_from_the_exact_ones(op, dt):
    """A value whose error is d of it changes its code where a border between
    two codes lies in between: for one of |q| / step d <= 16 d of the values.
    With u = 2^-24, d is for the norm half of the sum's (8 + 6 + 8) u and of the
    mean's 2 u, the root's 4 u, two products' 2 u and the quotient's u: 19 u in
    all.  For the gate with g > 0: the exponential's (4 u + 1.45 u g) e^-g /
    (1 + e^-g) <= 2.1 u, the sum 1 + e^-g u, its reciprocal 2 u, two products
    2 u, the quotient u: 8.1 u."""
    M, K, s = 2048, 4096, 0.013
    x = gen((M, K if op == "norm" else 2 * K), 5, dt)
    if op == "norm":
        w = gen((K,), 6, dt)
        q = dq.rmsnorm(x, w, quant="fp8_static", s_out=s)
        r = x.double()
        ref, d = r * torch.rsqrt(r.square().mean(1, keepdim=True) + 1e-6) * w.double(), 19 * U
    else:
        x[:, :K] = x[:, :K].abs()
        q = dq.silu_mul(x, quant="fp8_static", s_out=s)
        g, u = x.double().chunk(2, 1)
        ref, d = g * torch.sigmoid(g) * u, 8.1 * U
    exact = (ref / float(np.float32(s))).float().clamp(-448, 448).to(torch.float8_e4m3fn)
    other = (q.view(torch.float8_e4m3fn).float() != exact.float()).sum().item()
    assert other <= 16 * d * M * K, other


def test_empty_batch():
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    q, s = dq.quantize_act_fp8_block(x)
    assert q.shape == (0, 256) and s.shape == (0, 2)
    assert dq.rmsnorm(x, residual=x)[0].shape == (0, 256) and dq.silu_mul(x).shape == (0, 128)


def test_offsets_past_32_bits():
    M, K = 70000, 32768                             # 2.3e9 elements
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[-3:] = gen((3, K), 16, "bf16")
    q, s = dq.quantize_act_fp8_block(x)
    q2, s2 = dq.quantize_act_fp8_block(x[-3:].contiguous())
    assert torch.equal(q[-3:], q2) and torch.equal(s[-3:], s2) and not q[:-3].any()
    n = dq.rmsnorm(x, out=x.clone())
    assert torch.equal(n[-3:], dq.rmsnorm(x[-3:].contiguous()))


def test_offsets_past_32_bits_of_rows_that_start_anywhere():
    M, K = 70000, 32771
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[-3:] = gen((3, K), 16, "bf16")
    last = x[-3:].clone()
    q, s = dq.quantize_act_fp8_block(x)
    q2, s2 = dq.quantize_act_fp8_block(last)
    assert torch.equal(q[-3:], q2) and torch.equal(s[-3:], s2) and not q[:-3].any()
    del q, s
    n, r = dq.rmsnorm(x, residual=x, residual_out=x)          # r = 2 x, in place
    n2, r2 = dq.rmsnorm(last, residual=last)
    assert torch.equal(n[-3:], n2) and torch.equal(x[-3:], r2) and not n[:-3].any() and not x[:-3].any()


def test_streams_and_graphs():
    x, r = gen((64, 4096), 17, "bf16"), gen((64, 4096), 18, "bf16")
    ref = dq.rmsnorm(x, residual=r, quant="fp8_block")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    for kw, ctx in (({"stream": st}, torch.cuda.stream(torch.cuda.current_stream())), ({}, torch.cuda.stream(st))):
        with ctx:
            got = dq.rmsnorm(x, residual=r, quant="fp8_block", **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
    outs = [torch.zeros_like(t) for t in ref]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dq.rmsnorm(x, residual=r, quant="fp8_block", out=outs[0], scales=outs[1], residual_out=outs[2])
        dq.silu_mul(outs[2], quant="fp8_block")
    x2 = gen((64, 4096), 19, "bf16")
    want = dq.rmsnorm(x2, residual=r, quant="fp8_block")
    x.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


@pytest.mark.parametrize("dt,odt", [("bf16", "bf16"), ("fp32", "fp32"), ("fp32", "bf16"), ("fp32", "fp16"), ("bf16", "fp32")])
@pytest.mark.parametrize("K", [4096, 4100, 4099])
def test_silu_mul_far_below_zero_with_large_factors(dt, odt, K):
    """e^-g leaves fp32 at -88.7 and its reciprocal the normal numbers at -87.3; u
    up to 3e38 makes ordinary numbers of the results down to g = -180.  The
    tolerance is the gate's: e^(g/4) four times is within 4 x 2 units of 2^-23,
    its products within 5 more halves."""
    M = 6
    g = torch.linspace(-205, -60, M * K, dtype=torch.float64).reshape(K, M).T
    up = torch.exp2(torch.linspace(0, 95 if odt == "fp16" else 126, K)[torch.randperm(K, generator=torch.Generator().manual_seed(1))])
    u = up * (1 - 2 * (torch.arange(M)[:, None] % 2)) * (1 + torch.rand((M, K), generator=torch.Generator().manual_seed(2)) / 2)
    x = torch.cat([g, u.double()], 1).to(DT[dt]).cuda()
    ref = B.silu_mul(f64(x))
    rel = (8 + 1.2 * np.abs(f64(x)[:, :K])) * 2.0 ** -23
    check_float(dq.silu_mul(x, out_dtype=DT[odt]), ref, odt, rel)
    # a row of blocks by size, so that a block's scale is its own elements'
    order = torch.arange(K) * 61 % K if K % 61 else torch.arange(K)
    near = torch.cat([torch.linspace(-95, -85, K)[order].expand(M, K), torch.full((M, K), 2.0 ** 120)], 1).to(DT[dt]).cuda()
    q, s = dq.silu_mul(near, quant="fp8_block")
    check_codes(q, s, B.silu_mul(f64(near)), float((8 + 1.2 * 96) * 2.0 ** -23))
    # an element does not depend on its neighbours
    mixed = x.clone()
    mixed[:, :K][:, 1::2] = 1.0
    a, b = dq.silu_mul(x, out_dtype=DT[odt]), dq.silu_mul(mixed, out_dtype=DT[odt])
    assert torch.equal(a[:, 0::2], b[:, 0::2])
    x[:, :K] = x[:, :K].clamp(min=-79)
    mixed = x.clone()
    mixed[:, :K][:, 1::2] = -150.0
    a, b = dq.silu_mul(x, out_dtype=DT[odt]), dq.silu_mul(mixed, out_dtype=DT[odt])
    assert torch.equal(a[:, 0::2], b[:, 0::2])


def test_gradients_raise_where_they_would_be_missing():
    x, r, w = gen((4, 256), 31, "bf16"), gen((4, 256), 32, "bf16"), gen((256,), 33, "bf16")
    ref = dq.rmsnorm(x, w, residual=r)
    for which in (0, 1, 2):
        a = [x.clone(), w.clone(), r.clone()]
        a[which].requires_grad_(True)
        y, r2 = dq.rmsnorm(a[0], a[1], residual=a[2])
        assert torch.equal(y, ref[0]) and torch.equal(r2, ref[1])
        with pytest.raises(RuntimeError, match="inference only"):
            y.float().sum().backward()
        q, s, r3 = dq.rmsnorm(a[0], a[1], residual=a[2], quant="fp8_block")
        assert r3.requires_grad == (which != 1)        # the new residual has no weight in it
        if which != 1:
            with pytest.raises(RuntimeError, match="inference only"):
                r3.float().sum().backward()
    g = torch.cat([x, r], 1).requires_grad_(True)
    with pytest.raises(RuntimeError, match="inference only"):
        dq.silu_mul(g).float().sum().backward()
    with torch.no_grad():
        assert not dq.silu_mul(g).requires_grad and not dq.rmsnorm(x.clone().requires_grad_(True)).requires_grad
    ex = dq.QuantizedExperts.from_float("fp8_block", torch.randn(2, 128, 256, device="cuda"))
    off = torch.tensor([0, 1, 4], dtype=torch.int32, device="cuda")
    y = ex(x.clone().requires_grad_(True), off)
    assert torch.equal(y, ex(x, off))
    with pytest.raises(RuntimeError, match="inference only"):
        y.float().sum().backward()


@pytest.mark.parametrize("exponent", [-80, 0, 100])
def test_every_significand_of_a_blocks_maximum(exponent):
    """Scales and codes of blocks with each of the 2^23 significands of amax (of a
    binade), the other elements next to the borders between codes times the scale:
    the fp32 quotients decide those codes, so they test the scale, its reciprocal
    and the quotient's correction.  The definition in 64 bits: a quotient of two
    fp32 numbers rounded to fp64 and then to fp32 is the one rounded once (53 >=
    2 * 24 + 2)."""
    t = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    border = (t[:-1] + t[1:]) / 2                                   # 126 of them, exact
    step = 1 << 17
    for at in range(0, 1 << 23, step):
        m = torch.arange(at, at + step, device="cuda", dtype=torch.int32)
        a = (m + ((127 + exponent) << 23)).view(torch.float32)
        s = (a.double() / torch.tensor(448.0, dtype=torch.float64, device="cuda")).float()
        v = (s.double()[:, None] * border).float()                  # the nearest to the border, and one unit off
        off = (torch.arange(126, device="cuda") + m[:, None]) % 3 - 1
        v = (v.view(torch.int32) + off.int()).view(torch.float32)
        v[:, -1] = torch.minimum(v[:, -1], a)                       # (the largest border is below amax)
        x = torch.cat([a[:, None], v, -v[:, :1]], 1)
        q, sc = dq.quantize_act_fp8_block(x)
        assert torch.equal(sc[:, 0], s)
        want = (x.double() / s.double()[:, None]).float().to(torch.float8_e4m3fn)
        assert torch.equal(q, want.view(torch.uint8)), at
