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
must not overlap the inputs, except where a function says so.  A call runs on
``stream``, or on the current stream of the tensors' device, which must be the
current device.
"""

import math

import torch

from . import _native, _require

_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}   # _native.ROW_TYPES, ROW_OUTS
_QUANTS = {"fp8_block": 3, "fp8_static": 4}
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


def _rows(x, name, halves=1):
    """(M, K, row stride) of a 2-D operand whose rows are contiguous."""
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
    ld, inner = x.stride()
    if (inner != 1 and width != 1) or (M > 1 and ld < width):
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return M, width // halves, ld if M > 1 else width


def _outputs(x, M, K, quant, s_out, out_dtype, out, scales):
    """(kind, s_out, out, scales) with what is not given allocated."""
    dev = x.device
    if quant is None:
        if scales is not None or s_out is not None:
            raise ValueError("scales and s_out belong to quantized outputs (quant=...)")
        dt = x.dtype if out_dtype is None else out_dtype
        if dt not in _TYPES:
            raise TypeError(f"out_dtype must be bfloat16, float16 or float32, got {dt}")
        if out is None:
            out = torch.empty((M, K), dtype=dt, device=dev)
        else:
            _require(out, "out", shape=(M, K), dtype=dt, device=dev)
        return _TYPES[dt], 1.0, out, None
    if quant not in _QUANTS:
        raise ValueError(f"unknown quant {quant!r}; None, 'fp8_block' or 'fp8_static'")
    if out_dtype is not None:
        raise ValueError("out_dtype goes with quant=None")
    if out is None:
        out = torch.empty((M, K), dtype=torch.uint8, device=dev)
    else:
        _require(out, "out", shape=(M, K), dtype=torch.uint8, device=dev)
    if quant == "fp8_static":
        if scales is not None:
            raise ValueError("scales go with quant='fp8_block'")
        if s_out is None or not (math.isfinite(s_out) and s_out > 0):
            raise ValueError("quant='fp8_static' needs a finite s_out > 0")
        return 4, float(s_out), out, None
    if s_out is not None:
        raise ValueError("s_out goes with quant='fp8_static'")
    shape = (M, (K + 127) // 128)
    if scales is None:
        scales = torch.empty(shape, dtype=torch.float32, device=dev)
    else:
        _require(scales, "scales", shape=shape, dtype=torch.float32, device=dev)
    return 3, 1.0, out, scales


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
    dev = x.get_device()
    check_current(dev)
    if weight is not None:
        if weight.dtype not in _TYPES:
            raise TypeError(f"weight must be bfloat16, float16 or float32, got {weight.dtype}")
        _require(weight, "weight", shape=(K,), device=x.device)
    if residual is not None:
        _require(residual, "residual", shape=(M, K), dtype=x.dtype, device=x.device)
        if residual_out is None:
            residual_out = torch.empty((M, K), dtype=x.dtype, device=x.device)
        else:
            _require(residual_out, "residual_out", shape=(M, K), dtype=x.dtype, device=x.device)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    eps = float(eps)
    if not (math.isfinite(eps) and eps >= 0):
        raise ValueError(f"eps must be finite and not negative, got {eps}")
    kind, s_out, out, scales = _outputs(x, M, K, quant, s_out, out_dtype, out, scales)
    if M:
        _native._check(_native.lib().dqgemm_rmsnorm(
            _TYPES[x.dtype], x.data_ptr(), ld, None if residual is None else residual.data_ptr(),
            None if residual is None else residual_out.data_ptr(), 0 if weight is None else _TYPES[weight.dtype],
            None if weight is None else weight.data_ptr(), eps, M, K, kind, s_out, out.data_ptr(),
            None if scales is None else scales.data_ptr(), _native.device_stream(stream, dev)), "dqgemm_rmsnorm")
    r = (out,) if scales is None else (out, scales)
    if residual is not None:
        r += (residual_out,)
    return r if len(r) > 1 else out


def silu_mul(x, quant=None, s_out=None, out_dtype=None, out=None, scales=None, stream=None):
    """Gated SiLU: x [M, 2K] = [g | u] (the output of a fused gate and up
    projection) gives g / (1 + exp(-g)) * u, [M, K].  Types, strides and
    outputs as for ``rmsnorm``."""
    M, K, ld = _rows(x, "x", 2)
    dev = x.get_device()
    check_current(dev)
    kind, s_out, out, scales = _outputs(x, M, K, quant, s_out, out_dtype, out, scales)
    if M:
        _native._check(_native.lib().dqgemm_silu_mul(
            _TYPES[x.dtype], x.data_ptr(), ld, M, K, kind, s_out, out.data_ptr(),
            None if scales is None else scales.data_ptr(), _native.device_stream(stream, dev)), "dqgemm_silu_mul")
    return out if scales is None else (out, scales)


def quantize_act_fp8_block(x, out=None, scales=None, stream=None):
    """e4m3 codes of x [M, K] with a scale per 128 along K: (uint8 [M, K],
    fp32 [M, ceil(K / 128)]).  Types and strides as for ``rmsnorm``."""
    M, K, ld = _rows(x, "x")
    dev = x.get_device()
    check_current(dev)
    _, _, out, scales = _outputs(x, M, K, "fp8_block", None, None, out, scales)
    if M:
        _native._check(_native.lib().dqgemm_quantize_act_fp8_block(
            _TYPES[x.dtype], x.data_ptr(), ld, M, K, out.data_ptr(), scales.data_ptr(),
            _native.device_stream(stream, dev)), "dqgemm_quantize_act_fp8_block")
    return out, scales
