"""The row operators of a feed-forward block on torch tensors: RMS norm with the
residual's addition, gated SiLU, and the block-scaled FP8 activation quantizer.

Each is one launch of ``libdqgemm`` (``dqgemm_rmsnorm``, ``dqgemm_silu_mul``,
``dqgemm_quantize_act_fp8_block``); this module checks the tensors, which the
library sees only as addresses, and allocates the results.  ``quant`` names the
output:

    None          a tensor of ``out_dtype`` (the input's type if not given)
    "fp8_block"   (codes uint8 [M, K], scales fp32 [M, ceil(K / 128)]): what an
                  "fp8_block" layer's ``from_codes`` takes
    "fp8_static"  codes uint8 [M, K] under the per-tensor scale ``s_out``: what
                  an "fp8_static" layer calibrated with that scale takes

Results are allocated if not given (``out``, ``scales``, ``residual_out``) and
must not overlap the inputs, except where a function says so.  Inference only:
there is no backward.  In grad mode, with an input that requires a gradient, the
floating results carry a step that raises when a gradient reaches it, as the
``dqgemm::linear`` op does.  A call runs on
``stream``, or on the current stream of the tensors' device, which must be the
current device; its new tensors belong to that stream.
"""

import math

import torch

from . import _empty, _native, _require

_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}   # _native.ROW_TYPES, ROW_OUTS
_U8, _F32 = torch.uint8, torch.float32
_new = torch.empty_strided   # (the cheapest of torch's allocating calls on the host)
_MAX_M, _MAX_K = 1 << 31, 1 << 28
_one_device = None


def check_current(dev):
    """Calls go to the current device: it has to be the tensors' own.  (With
    one visible GPU it can only be that one.)"""
    global _one_device
    if _one_device is None:
        _one_device = torch.cuda.device_count() <= 1
    if not _one_device and torch.cuda.current_device() != dev:
        raise ValueError(f"the tensors live on cuda:{dev}; make it the current device "
                         "(torch.cuda.set_device / torch.cuda.device) before the call")


class _NoBackward(torch.autograd.Function):
    @staticmethod
    def forward(ctx, name, y, *inputs):
        ctx.name = name
        return y

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"{ctx.name} is inference only: it has no backward")


def no_backward(name, y, *inputs):
    """y, with a step that raises in backward where an input wants a gradient
    (without it the gradient would be missing without a word)."""
    wanted = [t for t in inputs if t is not None and t.requires_grad]
    if wanted and torch.is_grad_enabled():
        return _NoBackward.apply(name, y, *wanted)
    return y


def _rows(x, name, halves=1):
    """(M, K, row stride) of a 2-D operand whose rows are contiguous."""
    try:                     # the common operand, checked in a few steps
        if x.is_cuda and x.dtype in _TYPES and x.is_contiguous():
            M, width = x.shape
            if width and not width % halves and M < _MAX_M and width <= _MAX_K:
                return M, width // halves, width
    except (AttributeError, ValueError):
        pass
    if getattr(x, "dim", lambda: 0)() != 2:
        raise ValueError(f"{name} must be 2-D")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.dtype not in _TYPES:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {x.dtype}")
    M, width = x.shape
    if width % halves or width == 0:
        raise ValueError(f"{name} must hold {halves} halves of at least one column" if halves > 1
                         else f"{name} must have at least one column")
    if M >= _MAX_M or width // halves > _MAX_K:   # (the library takes them as 32-bit numbers)
        raise ValueError(f"{name} must have fewer than 2^31 rows and at most 2^28 columns{' a half' if halves > 1 else ''}")
    ld, inner = x.stride()
    if (inner != 1 and width != 1) or (M > 1 and ld < width):
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return M, width // halves, ld if M > 1 else width


def _given(t, name, M, K, dtype, x):
    """A given [M, K] operand of x's device: checked the short way, and only a
    misfit by _require, which names it."""
    if not (t.dtype is dtype and t.dim() == 2 and t.shape[0] == M and t.shape[1] == K and t.is_contiguous()
            and t.get_device() == x.get_device() and t.is_cuda):
        _require(t, name, shape=(M, K), dtype=dtype, device=x.device)


def _outputs(x, M, K, quant, s_out, out_dtype, out, scales, stream=None):
    """(kind, s_out, out, scales) with what is not given allocated."""
    if quant == "fp8_block":
        if out_dtype is not None:
            raise ValueError("out_dtype goes with quant=None")
        if s_out is not None:
            raise ValueError("s_out goes with quant='fp8_static'")
        dev = x.device
        if out is None:
            out = _new((M, K), (K, 1), dtype=_U8, device=dev) if stream is None else _empty((M, K), _U8, dev, stream)
        else:
            _given(out, "out", M, K, _U8, x)
        kb = (K + 127) // 128
        if scales is None:
            scales = _new((M, kb), (kb, 1), dtype=_F32, device=dev) if stream is None else _empty((M, kb), _F32, dev, stream)
        else:
            _given(scales, "scales", M, kb, _F32, x)
        return 3, 1.0, out, scales
    if scales is not None:
        raise ValueError("scales go with quant='fp8_block'")
    if quant is None:
        if s_out is not None:
            raise ValueError("s_out goes with quant='fp8_static'")
        dt = x.dtype if out_dtype is None else out_dtype
        if dt not in _TYPES:
            raise TypeError(f"out_dtype must be bfloat16, float16 or float32, got {dt}")
        kind, s_out = _TYPES[dt], 1.0
    elif quant == "fp8_static":
        if out_dtype is not None:
            raise ValueError("out_dtype goes with quant=None")
        if s_out is None or not (math.isfinite(s_out) and s_out > 0):
            raise ValueError("quant='fp8_static' needs a finite s_out > 0")
        dt, kind, s_out = torch.uint8, 4, float(s_out)
    else:
        raise ValueError(f"unknown quant {quant!r}; None, 'fp8_block' or 'fp8_static'")
    if out is None:
        out = _new((M, K), (K, 1), dtype=dt, device=x.device) if stream is None else _empty((M, K), dt, x.device, stream)
    else:
        _given(out, "out", M, K, dt, x)
    return kind, s_out, out, None


def rmsnorm(x, weight=None, eps=1e-6, residual=None, quant=None, s_out=None, out_dtype=None, out=None, scales=None,
            residual_out=None, stream=None):
    """Root-mean-square norm of r = x + residual:  r * weight / sqrt(mean(r^2) + eps).

    x: [M, K] bf16, fp16 or fp32 (rows may be a slice of a wider tensor);
    weight [K] of any of these types, or None for ones; residual [M, K]
    contiguous, of x's type.  The norm is of the unrounded sum.  Returns the
    output (see the module); with a residual also the new one, r rounded to
    x's type, as the last of a tuple.  ``residual_out`` may be ``residual``
    itself, or a contiguous x."""
    M, K, ld = _rows(x, "x")
    dt = x.dtype
    dev = x.get_device()
    if _one_device is not True:
        check_current(dev)
    wt = wp = rp = np = None
    if weight is not None:
        wt = _TYPES.get(weight.dtype)
        if wt is None:
            raise TypeError(f"weight must be bfloat16, float16 or float32, got {weight.dtype}")
        if not (weight.dim() == 1 and weight.shape[0] == K and weight.is_contiguous() and weight.get_device() == dev):
            _require(weight, "weight", shape=(K,), device=x.device)
        wp = weight.data_ptr()
    if residual is not None:
        _given(residual, "residual", M, K, dt, x)
        if residual_out is None:
            residual_out = (_new((M, K), (K, 1), dtype=dt, device=x.device) if stream is None
                            else _empty((M, K), dt, x.device, stream))
        elif residual_out is not residual:
            _given(residual_out, "residual_out", M, K, dt, x)
        rp, np = residual.data_ptr(), residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if not 0 <= eps < math.inf:
        raise ValueError(f"eps must be finite and not negative, got {eps}")
    kind, s_out, out, scales = _outputs(x, M, K, quant, s_out, out_dtype, out, scales, stream)
    if M:
        st = _native.lib().dqgemm_rmsnorm(_TYPES[dt], x.data_ptr(), ld, rp, np, wt or 0, wp, eps, M, K, kind, s_out,
                                          out.data_ptr(), None if scales is None else scales.data_ptr(),
                                          _native.device_stream(stream, dev))
        if st:
            raise _native.DQError(st, "dqgemm_rmsnorm")
    if x.requires_grad or weight is not None and weight.requires_grad or residual is not None and residual.requires_grad:
        if quant is None:
            out = no_backward("rmsnorm", out, x, weight, residual)
        if residual is not None:
            residual_out = no_backward("rmsnorm", residual_out, x, residual)
    if residual is None:
        return out if scales is None else (out, scales)
    return (out, residual_out) if scales is None else (out, scales, residual_out)


def silu_mul(x, quant=None, s_out=None, out_dtype=None, out=None, scales=None, stream=None):
    """Gated SiLU: x [M, 2K] = [g | u] (the output of a fused gate and up
    projection) gives g / (1 + exp(-g)) * u, [M, K].  Types, strides and
    outputs as for ``rmsnorm``."""
    M, K, ld = _rows(x, "x", 2)
    dev = x.get_device()
    if _one_device is not True:
        check_current(dev)
    kind, s_out, out, scales = _outputs(x, M, K, quant, s_out, out_dtype, out, scales, stream)
    if M:
        st = _native.lib().dqgemm_silu_mul(_TYPES[x.dtype], x.data_ptr(), ld, M, K, kind, s_out, out.data_ptr(),
                                           None if scales is None else scales.data_ptr(),
                                           _native.device_stream(stream, dev))
        if st:
            raise _native.DQError(st, "dqgemm_silu_mul")
    if quant is None and x.requires_grad:
        out = no_backward("silu_mul", out, x)
    return out if scales is None else (out, scales)


def quantize_act_fp8_block(x, out=None, scales=None, stream=None):
    """e4m3 codes of x [M, K] with a scale per 128 along K: (uint8 [M, K],
    fp32 [M, ceil(K / 128)]).  Types and strides as for ``rmsnorm``."""
    M, K, ld = _rows(x, "x")
    dev = x.get_device()
    if _one_device is not True:
        check_current(dev)
    _, _, out, scales = _outputs(x, M, K, "fp8_block", None, None, out, scales, stream)
    if M:
        _native._check(_native.lib().dqgemm_quantize_act_fp8_block(
            _TYPES[x.dtype], x.data_ptr(), ld, M, K, out.data_ptr(), scales.data_ptr(),
            _native.device_stream(stream, dev)), "dqgemm_quantize_act_fp8_block")
    return out, scales
