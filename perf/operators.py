"""The operators of a feed-forward block in block-scaled FP8, as they are measured.

Four operators: ``norm`` (root-mean-square norm of x + residual), ``gate``
(silu(g) * u), ``linear`` (FP8 product with a scale per 128 x 128 weight block
and per 128 activations) and ``experts`` (the same product for rows grouped by
expert).  ``run`` computes them in plain 32-bit torch, or through the package
where ``own`` is true.  8-bit outputs come as e4m3 tensors beside their
scales.  The plain form of ``experts`` pads every expert's rows to the largest
count, which the state holds.
"""

import math

import torch

own = False

EPS = 1e-6
BLOCK = 128
E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token's hidden state on its way into a projection
        {"name": "norm token", "op": "norm", "M": 1, "K": 4096, "dtype": "bf16", "quant": "fp8_block", "residual": True},
        # an fp32 residual stream of a ragged batch, the width no multiple of the block, 16-bit output
        {"name": "norm ragged fp32", "op": "norm", "M": 777, "K": 5008, "dtype": "fp32", "quant": "bf16", "residual": True},
        # a prompt batch
        {"name": "norm prompt", "op": "norm", "M": 16384, "K": 4096, "dtype": "bf16", "quant": "fp8_block", "residual": True},
        # a decode batch's gate, codes for a static-FP8 layer, odd width
        {"name": "gate decode", "op": "gate", "M": 17, "K": 5004, "dtype": "fp16", "quant": "fp8_static"},
        # a prompt's gate in front of the down projection
        {"name": "gate prompt", "op": "gate", "M": 8192, "K": 14336, "dtype": "bf16", "quant": "fp8_block"},
        # one token through the up projection
        {"name": "linear token", "op": "linear", "M": 1, "K": 4096, "N": 14336, "codes": False, "bias": False},
        # a decode batch through a square projection
        {"name": "linear decode", "op": "linear", "M": 32, "K": 4096, "N": 4096, "codes": False, "bias": True},
        # a ragged prompt, K and N inside a block
        {"name": "linear ragged", "op": "linear", "M": 777, "K": 1040, "N": 5000, "codes": True, "bias": True},
        # a prompt batch through the up projection, on the norm's codes
        {"name": "linear prompt", "op": "linear", "M": 8192, "K": 4096, "N": 14336, "codes": True, "bias": False},
        # a small mixture: seven rows over five of eight experts
        {"name": "experts small", "op": "experts", "M": 7, "K": 1024, "N": 768, "E": 8, "used": 5, "codes": False},
        # a decode batch: 32 experts, most of them with a row or two
        {"name": "experts decode", "op": "experts", "M": 64, "K": 4096, "N": 2048, "E": 32, "used": 24, "codes": False},
        # a prompt over 16 experts with ragged counts
        {"name": "experts prompt", "op": "experts", "M": 8192, "K": 4096, "N": 4096, "E": 16, "used": 15, "codes": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "gate", "linear", "experts"])
    if op in ("norm", "gate"):
        K = _log(rng, 200, 14000)
        M = min(_log(rng, 1, 16000), 60_000_000 // K)
        c = {"op": op, "M": M, "K": K, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
             "quant": rng.choice(["fp8_block", "fp8_block", "fp8_static", "bf16"])}
        if op == "norm":
            c["residual"] = rng.random() < 0.7
        return c
    K = 16 * _log(rng, 8, 512)
    N = _log(rng, 100, 14000)
    if op == "linear":
        M = min(_log(rng, 1, 8000), 400_000_000_000 // (2 * K * N) + 1)
        return {"op": op, "M": M, "K": K, "N": N, "codes": rng.random() < 0.5, "bias": rng.random() < 0.5}
    E = rng.randint(2, max(2, min(64, 250_000_000 // (K * N))))
    M = min(_log(rng, 1, 8000), 100_000_000_000 // (2 * K * N) + 1)
    return {"op": op, "M": M, "K": K, "N": N, "E": E, "used": rng.randint(1, min(E, M)), "codes": rng.random() < 0.5}


def _e4m3(u8):
    return u8.view(torch.float8_e4m3fn)


def _blocks(v):
    """v [..., K] with K padded with zeros to whole blocks: [..., K / 128, 128]."""
    v = torch.nn.functional.pad(v, (0, -v.shape[-1] % BLOCK))
    return v.unflatten(-1, (-1, BLOCK))


def _quantize_rows(v):
    """v fp32 [M, K] -> e4m3 codes [M, K], scales fp32 [M, ceil(K / 128)]."""
    b = _blocks(v)
    s = b.abs().amax(-1) / E4M3_MAX
    q = torch.where(s[..., None] > 0, b / s[..., None], torch.zeros_like(b))
    return q.flatten(-2)[..., :v.shape[-1]].to(torch.float8_e4m3fn).contiguous(), s


def _quantize_weight(w):
    """w fp32 [E, N, K] -> codes u8 [E, N, K], scales fp32 [E, N / 128, K / 128] (rounded up)."""
    E, N, K = w.shape
    p = torch.nn.functional.pad(w, (0, -K % BLOCK, 0, -N % BLOCK))
    p = p.view(E, p.shape[1] // BLOCK, BLOCK, p.shape[2] // BLOCK, BLOCK)
    s = p.abs().amax((2, 4)) / E4M3_MAX
    q = (p / s[:, :, None, :, None]).view(E, p.shape[1] * BLOCK, -1)[:, :N, :K]
    return q.to(torch.float8_e4m3fn).contiguous().view(torch.uint8), s


def _widen(s, rows, cols):
    """A scale per block of the last two dims, spread over rows x cols elements."""
    return s.repeat_interleave(BLOCK, -2)[..., :rows, :].repeat_interleave(BLOCK, -1)[..., :cols]


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    randn = lambda *n: torch.randn(n, generator=g, device="cuda")  # noqa: E731
    M, K = case["M"], case["K"]
    st = {"case": case}
    if case["op"] == "norm":
        dt = DTYPES[case["dtype"]]
        st["x"] = (randn(M, K) * (0.5 + randn(M, 1).abs())).to(dt)
        st["residual"] = (randn(M, K) * 2).to(dt) if case["residual"] else None
        st["weight"] = (1 + 0.2 * randn(K)).to(dt)
        st["s_out"] = 0.011
        return st
    if case["op"] == "gate":
        st["x"] = (randn(M, 2 * K) * (0.5 + randn(M, 1).abs())).to(DTYPES[case["dtype"]])
        st["s_out"] = 0.023
        return st
    N, E = case["N"], case.get("E", 1)
    w = (torch.rand((E, N, K), generator=g, device="cuda") * 2 - 1) / math.sqrt(K)
    st["w"], st["sw"] = _quantize_weight(w)
    del w
    x = (randn(M, K) * (0.5 + randn(M, 1).abs())).to(torch.bfloat16)
    if case["codes"]:
        q, st["sx"] = _quantize_rows(x.float())
        st["q"] = q.view(torch.uint8)
    else:
        st["x"] = x
    if case["op"] == "linear":
        st["bias"] = randn(N).to(torch.bfloat16) if case["bias"] else None
    else:
        # ragged counts: `used` experts, each with a row at least, the rest of the rows skewed
        h = torch.Generator("cpu").manual_seed(seed)
        ids = torch.randperm(E, generator=h)[:case["used"]]
        share = torch.rand(case["used"], generator=h) + 0.1
        more = torch.multinomial(share, M - case["used"], replacement=True, generator=h) if M > case["used"] else ids[:0]
        counts = torch.bincount(torch.cat([ids, ids[more]]), minlength=E)
        st["cap"] = int(counts.max())
        st["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32).cuda()
    if own:
        import weight_only_quantized_prologue_b200 as dq

        if case["op"] == "linear":
            st["layer"] = dq.QuantizedLinear("fp8_block", K, N, st["w"][0], st["sw"][0], bias=st["bias"])
        else:
            st["layer"] = dq.QuantizedExperts("fp8_block", E, K, N, st["w"], st["sw"])
    return st


def _run_own(st):
    import weight_only_quantized_prologue_b200 as dq

    c = st["case"]
    if c["op"] in ("norm", "gate"):
        quant = None if c["quant"] == "bf16" else c["quant"]
        kw = {"quant": quant}
        if quant is None:
            kw["out_dtype"] = torch.bfloat16
        elif quant == "fp8_static":
            kw["s_out"] = st["s_out"]
        if c["op"] == "norm":
            r = dq.rmsnorm(st["x"], st["weight"], EPS, residual=st["residual"], **kw)
        else:
            r = dq.silu_mul(st["x"], **kw)
        r = r if isinstance(r, tuple) else (r,)
        return [_e4m3(t) if t.dtype == torch.uint8 else t for t in r]
    if c["op"] == "linear":
        return [st["layer"].from_codes(st["q"], scales=st["sx"]) if c["codes"] else st["layer"](st["x"])]
    if c["codes"]:
        return [st["layer"].from_codes(st["q"], st["sx"], st["offsets"])]
    return [st["layer"](st["x"], st["offsets"])]


def _out(y, c, st):
    if c["quant"] == "bf16":
        return [y.to(torch.bfloat16)]
    if c["quant"] == "fp8_static":
        return [(y / st["s_out"]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)]
    return list(_quantize_rows(y))


def run(st):
    if own:
        return _run_own(st)
    c = st["case"]
    if c["op"] == "norm":
        r = st["x"].float()
        if c["residual"]:
            r = r + st["residual"].float()
        y = r / (r.square().mean(-1, keepdim=True) + EPS).sqrt() * st["weight"].float()
        return _out(y, c, st) + ([r.to(st["x"].dtype)] if c["residual"] else [])
    if c["op"] == "gate":
        g, u = st["x"].float().chunk(2, -1)
        return _out(g / (1 + (-g).exp()) * u, c, st)
    q, s = (_e4m3(st["q"]), st["sx"]) if c["codes"] else _quantize_rows(st["x"].float())
    K, N = c["K"], c["N"]
    x = q.float() * s.repeat_interleave(BLOCK, -1)[:, :K]
    w = _e4m3(st["w"]).float() * _widen(st["sw"], N, K)
    if c["op"] == "linear":
        y = x @ w[0].T
        if c["bias"]:
            y = y + st["bias"].float()
        return [y.to(torch.bfloat16)]
    o = st["offsets"].long()
    row = torch.arange(c["M"], device="cuda")
    e = (row[:, None] >= o[None, 1:]).sum(-1)
    at = row - o[e]
    padded = torch.zeros((c["E"], st["cap"], K), device="cuda")
    padded[e, at] = x
    return [torch.bmm(padded, w.transpose(1, 2))[e, at].to(torch.bfloat16)]


def work(case):
    M, K = case["M"], case["K"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if case["op"] in ("norm", "gate"):
        b = size[case["dtype"]]
        out = 2 * M * K if case["quant"] == "bf16" else M * K
        if case["quant"] == "fp8_block":
            out += 4 * M * -(-K // BLOCK)
        if case["op"] == "gate":
            return {"bytes": 2 * b * M * K + out, "flops": 6 * M * K}
        return {"bytes": b * M * K * (3 if case["residual"] else 1) + b * K + out, "flops": 6 * M * K}
    N, kb = case["N"], -(-K // BLOCK)
    weights = case.get("used", 1) * (N * K + 4 * -(-N // BLOCK) * kb)
    x = M * K + 4 * M * kb if case["codes"] else 2 * M * K
    return {"bytes": x + weights + 2 * M * N, "flops": 2 * M * N * K}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def _round_e4m3(a):
    """The nearest e4m3 value of each element (ties to even), as fp64."""
    a = a.clamp(-E4M3_MAX, E4M3_MAX)
    step = torch.exp2(torch.floor(torch.log2(a.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(a / step) * step


def _exact_codes(v):
    """Codes and scales of v [M, K]: the scale of a block is the fp32 nearest to amax / 448, the code
    the e4m3 nearest to the fp32 quotient (16-bit inputs put many quotients on a border)."""
    M, K = v.shape
    kb = -(-K // BLOCK)
    p = torch.zeros((M, kb * BLOCK), dtype=torch.float64, device=v.device)
    p[:, :K] = v
    p = p.reshape(M, kb, BLOCK)
    s = (p.abs().max(-1).values / E4M3_MAX).float().double()
    q = _round_e4m3((p / s.unsqueeze(-1).masked_fill(s.unsqueeze(-1) == 0, 1.0)).float().double())
    return q.reshape(M, -1)[:, :K], s


def exact(case, seed):
    st = prepare(case, seed)
    c, K = case, case["K"]
    if c["op"] in ("norm", "gate"):
        x = st["x"].double()
        if c["op"] == "gate":
            y = x[:, :K] * torch.sigmoid(x[:, :K]) * x[:, K:]
            more = []
        else:
            more = []
            if c["residual"]:
                x = x + st["residual"].double()
                more = [x]
            y = x * torch.rsqrt((x * x).sum(1, keepdim=True) / K + EPS) * st["weight"].double()
        if c["quant"] == "bf16":
            return [y] + more
        if c["quant"] == "fp8_static":
            # the scale is a 32-bit argument
            return [_round_e4m3(y / float(torch.tensor(st["s_out"], dtype=torch.float32)))] + more
        return list(_exact_codes(y)) + more
    if c["codes"]:
        q, s = _e4m3(st["q"]).double(), st["sx"].double()
    else:
        q, s = _exact_codes(st["x"].double())
    M, N = c["M"], c["N"]
    col = torch.arange(K, device="cuda") // BLOCK
    row = torch.arange(N, device="cuda") // BLOCK
    x = q * s[:, col]
    bounds = st["offsets"].tolist() if c["op"] == "experts" else [0, M]
    y = torch.empty((M, N), dtype=torch.float64, device="cuda")
    for e in range(len(bounds) - 1):
        if bounds[e + 1] > bounds[e]:
            w = _e4m3(st["w"][e]).double() * st["sw"][e].double()[row][:, col]
            y[bounds[e]:bounds[e + 1]] = x[bounds[e]:bounds[e + 1]] @ w.T
    return [y + st["bias"].double() if c.get("bias") else y]
