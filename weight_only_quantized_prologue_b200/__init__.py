"""B200-native quantized nn.Linear with the dequantization in the GEMM prologue.

The compute lives in ``libdqgemm.so`` (hand-written sm_100a CUDA, C ABI in
``include/dqgemm.h``); this package only marshals torch tensors to it.

    from weight_only_quantized_prologue_b200 import QuantizedLinear
    ql = QuantizedLinear.from_float("int4", W_fp32_cuda, bias_bf16_cuda)
    y = ql(x_bf16_cuda)            # y = x . deq(W)^T + b, bf16
"""

import numpy as _np

from . import _native
from ._native import (  # noqa: F401
    FORMATS,
    DQError,
    dqgemm_create,
    dqgemm_create_experts,
    dqgemm_dequantize,
    dqgemm_destroy,
    dqgemm_get_plan,
    dqgemm_last_error,
    dqgemm_pack_device,
    dqgemm_pack_device_noalloc,
    dqgemm_pack_host,
    dqgemm_quantize_act_fp4,
    dqgemm_quantize_act_fp8,
    dqgemm_quantize_act_fp8_block,
    dqgemm_rmsnorm,
    dqgemm_run,
    dqgemm_run_experts_quantized,
    dqgemm_run_fp8_block,
    dqgemm_run_fp8_block_quantized,
    dqgemm_run_fp8_static_quantized,
    dqgemm_run_fp8_static_quantized_out,
    dqgemm_run_quantized_out,
    dqgemm_run_static_mlp,
    dqgemm_selftest_timeout,
    dqgemm_set_wait_limit,
    dqgemm_silu_mul,
    dqgemm_status_string,
    storage_shapes,
)


def _require(t, name, shape=None, dtype=None, nbytes=None, device=None):
    """Checks the library cannot make itself: its entry points take bare
    device pointers, so a tensor of the wrong dtype, shape or layout would be
    read or written out of bounds on the GPU."""
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if nbytes is not None and t.numel() * t.element_size() != nbytes:
        raise ValueError(f"{name} must hold {nbytes} bytes, got {t.numel() * t.element_size()}")


def _fits(t, cols, dtype, rows=None, dev=None):
    """Fast form of the _require checks for a 2-D operand [rows, cols]: True
    exactly when _require(t, shape=(rows, cols), dtype, device) would pass,
    `dev` being that device's index (an integer compare: building the
    operand's torch.device on every call costs more than the rest)."""
    try:
        return (t.dtype is dtype and t.is_cuda and t.dim() == 2 and t.shape[1] == cols
                and (rows is None or t.shape[0] == rows) and t.is_contiguous()
                and (dev is None or t.get_device() == dev))
    except AttributeError:
        return False


_torch_mod = None


def _torch():
    """torch, imported on first use (the package itself does not need it)."""
    global _torch_mod
    if _torch_mod is None:
        import torch

        _torch_mod = torch
    return _torch_mod


def _on_current_device(device, what):
    """The library launches on, and a handle belongs to, the current device: a
    weight or layer on another one would be read there through bare pointers."""
    cuda = _torch().cuda
    if cuda.device_count() > 1 and cuda.current_device() != device.index:
        raise ValueError(f"{what} on {device}; make it the current device (torch.cuda.set_device / "
                         f"torch.cuda.device) before the call")


def _empty(shape, dtype, device, stream):
    """A new dense tensor for a call on `stream`, in that stream's memory: what
    the allocator hands out for the current stream may still be in use by work
    queued there, and goes back to that stream's next tensor when a temporary
    is dropped, while the call may still run."""
    torch = _torch()
    strides = (shape[1], 1) if len(shape) == 2 else (1,)
    if stream is None:
        return torch.empty_strided(shape, strides, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        s = _native._stream(stream)
        stream = torch.cuda.ExternalStream(s, device=device) if s else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty_strided(shape, strides, dtype=dtype, device=device)


def _storage_bytes(fmt, K, N):
    ps, pd, ss, sd = storage_shapes(fmt, K, N)
    return (int(_np.prod(ps)) * _np.dtype(pd).itemsize, int(_np.prod(ss)) * _np.dtype(sd).itemsize)


def static_mlp(l1, l2, x, out=None, h_out=None, stream=None):
    """The static-FP8 two-layer model y = l2(l1(x)) in one launch
    (dqgemm_run_static_mlp): l1, l2 are "fp8_static" QuantizedLinear layers
    with l2.K == l1.N, l1.N in {256, 512, 1024}, l2.N <= 128; x bf16
    [M, l1.K] on their device.  Returns y (``out``, allocated if None);
    ``h_out`` (bf16 [M, l1.N]) receives layer 1's output if given."""
    torch = _torch()
    if l1.fmt != "fp8_static" or l2.fmt != "fp8_static":
        raise ValueError("static_mlp needs two fp8_static layers")
    if l2.K != l1.N:
        raise ValueError(f"layer 2 takes {l2.K} inputs, layer 1 gives {l1.N}")
    if l2._dev != l1._dev:
        raise ValueError("both layers must live on the same device")
    M = l1._check_x(x, torch.bfloat16)
    out = l2._out(out, M, torch.bfloat16, stream)
    if h_out is not None:
        _require(h_out, "h_out", shape=(M, l1.N), dtype=torch.bfloat16, device=l1.device)
    if M == 0:
        return out
    dqgemm_run_static_mlp(l1.handle, l2.handle, x, M, h_out, out, stream)
    return out


def _block_call(layer, x, M, offsets, out, stream):
    """A block-scaled layer (or experts, with their offsets) on bf16 x.  With
    more than the few rows that the product's own kernel quantizes, their
    codes and scales go through a temporary of the stream the call runs on, so
    that the allocator hands it to nobody before the call is done."""
    dev = layer._dev
    s = _native.device_stream(stream, dev)
    size = ws = 0
    if M > layer._few_rows:
        size = M * (layer.K + 4 * ((layer.K + 127) // 128)) + 256
        tmp = _empty((size,), _torch().uint8, layer.device, stream)
        ws = tmp.data_ptr()
    _native._check(_native.lib().dqgemm_run_fp8_block(layer._h, x.data_ptr(), M, offsets, out.data_ptr(), ws or None, size, s),
                   "dqgemm_run_fp8_block")


class QuantizedLinear:
    """One quantized Linear layer on the current CUDA device.

    ``packed`` / ``scales`` are CUDA tensors in the canonical layout of
    ``fmt`` (see ``storage_shapes``); they are copied and re-laid-out by the
    library, so the caller may drop them afterwards."""

    # rows up to which the library quantizes a block-scaled layer's bf16 x in
    # the product's kernel, so that a call needs no workspace
    _few_rows = 8
    # static FP8 from this many rows on: quantize x once, then the FP8 GEMM
    # (the fused kernel re-quantizes x for every 128-channel tile) ...
    STATIC_PREQUANT_M = 128
    # ... and from this many when the output tiles fill more than half the
    # SMs in one wave: the GEMM on codes then takes the 128-row tile, one CTA
    # per SM over the whole K range, which the fused kernel does not (at
    # 4096 x 14336: 19.6 against 33.6 us at 32 rows; up to 16 rows the fused
    # 16-row tile is faster, 23.2 against 25.5)
    STATIC_PREQUANT_M_WIDE = 17

    def __init__(self, fmt, K, N, packed, scales, global_scale=1.0, bias=None):
        import torch

        self._h = None
        if fmt not in FORMATS:
            raise ValueError(f"unknown format {fmt!r}; one of {tuple(FORMATS)}")
        pb, sb = _storage_bytes(fmt, K, N)
        _require(packed, "packed", nbytes=pb)
        _require(scales, "scales", nbytes=sb, device=packed.device)
        if bias is not None:
            _require(bias, "bias", shape=(N,), dtype=torch.bfloat16, device=packed.device)
        self.fmt, self.K, self.N = fmt, K, N
        _on_current_device(packed.device, "packed is")
        sms = torch.cuda.get_device_properties(packed.device).multi_processor_count
        n_tiles = (N + 127) // 128
        self._static_prequant_m = (self.STATIC_PREQUANT_M_WIDE if 2 * n_tiles > sms and n_tiles <= sms
                                   else self.STATIC_PREQUANT_M)
        self.device = packed.device               # the handle belongs to this device
        self._dev = self.device.index
        # with one visible GPU the current device can only be this one
        self._check_current = torch.cuda.device_count() > 1
        self.act_scale = float(global_scale) if fmt == "fp8_static" else None
        self._h = dqgemm_create(fmt, K, N, packed, scales, global_scale, bias)

    @classmethod
    def from_float(cls, fmt, W, bias=None, act_scale=None):
        """Quantize a CUDA fp32 weight [N, K] with the GPU packer and build the
        layer.  ``act_scale`` is the static-FP8 per-tensor activation scale."""
        import torch

        if not getattr(W, "is_cuda", False) or W.dim() != 2:
            raise ValueError("W must be a 2-D CUDA tensor [N, K]")
        _on_current_device(W.device, "W is")
        W = W.detach().to(torch.float32).contiguous()
        N, K = W.shape
        ps, pd, ss, sd = storage_shapes(fmt, K, N)
        tdt = {_np.uint8: torch.uint8, _np.uint16: torch.int16, _np.float32: torch.float32}
        packed = torch.empty(ps, dtype=tdt[pd], device=W.device)
        scales = torch.empty(ss, dtype=tdt[sd], device=W.device)
        g = dqgemm_pack_device("fp8" if fmt == "fp8_static" else fmt, W, packed, scales)
        if fmt == "fp8_static":
            g = act_scale
        return cls(fmt, K, N, packed, scales, g, bias)

    def _check_x(self, x, dtype, name="x"):
        if not _fits(x, self.K, dtype, dev=self._dev):
            if getattr(x, "dim", lambda: 0)() != 2:
                raise ValueError(f"{name} must be 2-D [M, {self.K}]")
            _require(x, name, shape=(x.shape[0], self.K), dtype=dtype, device=self.device)
        if self._check_current:
            if _torch().cuda.current_device() != self._dev:
                raise ValueError(f"the layer lives on {self.device}; make it the current device "
                                 f"(torch.cuda.set_device / torch.cuda.device) before calling it")
        M = x.shape[0]
        if M >= 1 << 31:   # (the library takes it as a 32-bit number)
            raise ValueError(f"{name} must have fewer than 2^31 rows")
        return M

    def _out(self, out, M, dtype, stream):
        if out is None:
            if stream is None:   # (empty_strided: the cheapest of torch's allocating calls on the host)
                return _torch().empty_strided((M, self.N), (self.N, 1), dtype=dtype, device=self.device)
            return _empty((M, self.N), dtype, self.device, stream)
        if not _fits(out, self.N, dtype, M, self._dev):
            _require(out, "out", shape=(M, self.N), dtype=dtype, device=self.device)
        return out

    def __call__(self, x, out=None, stream=None):
        """y = x . deq(W)^T + b; x bf16 [M, K] contiguous on CUDA, y (``out``,
        allocated if None) bf16 [M, N]."""
        torch = _torch()
        M = self._check_x(x, torch.bfloat16)
        out = self._out(out, M, torch.bfloat16, stream)
        if M == 0:
            return out
        if self.fmt == "fp8_block":
            _block_call(self, x, M, None, out, stream)
        elif self.fmt == "fp8_static" and M >= self._static_prequant_m:
            q = _empty((M, self.K), torch.uint8, self.device, stream)
            dqgemm_quantize_act_fp8(x, M, self.K, self.act_scale, q, stream)
            dqgemm_run_fp8_static_quantized(self._h, q, M, out, stream)
        else:
            # (operands checked above: their pointers go straight to the entry)
            _native.run_ptrs(self._h, x.data_ptr(), M, out.data_ptr(), stream)
        return out

    def quantized_out(self, x, s_out, out=None, stream=None):
        """The layer with its result leaving as the next static-FP8 layer's
        e4m3 codes, e4m3(f32(y) / s_out) (uint8 [M, N]); x as for __call__."""
        torch = _torch()
        M = self._check_x(x, torch.bfloat16)
        out = self._out(out, M, torch.uint8, stream)
        if M == 0:
            return out
        if self.fmt == "fp8_static" and M >= self._static_prequant_m:
            q = _empty((M, self.K), torch.uint8, self.device, stream)
            dqgemm_quantize_act_fp8(x, M, self.K, self.act_scale, q, stream)
            dqgemm_run_fp8_static_quantized_out(self._h, q, M, out, s_out, stream)
        else:
            dqgemm_run_quantized_out(self._h, x, M, out, s_out, stream)
        return out

    def from_codes(self, q, out=None, stream=None, scales=None):
        """The layer on activations that are e4m3 codes already (uint8 [M, K]):
        static FP8, quantized with the layer's own scale (e.g. by
        quantized_out); "fp8_block", with their ``scales`` fp32 [M, ceil(K /
        128)] (from rmsnorm, silu_mul or quantize_act_fp8_block)."""
        torch = _torch()
        if self.fmt not in ("fp8_static", "fp8_block"):
            raise ValueError("from_codes needs a static FP8 layer or a block-scaled one")
        if (scales is None) == (self.fmt == "fp8_block"):
            raise ValueError("scales go with the codes of an fp8_block layer")
        M = self._check_x(q, torch.uint8, "q")
        if scales is not None and not _fits(scales, (self.K + 127) // 128, torch.float32, M, self._dev):
            _require(scales, "scales", shape=(M, (self.K + 127) // 128), dtype=torch.float32, device=self.device)
        out = self._out(out, M, torch.bfloat16, stream)
        if M == 0:
            return out
        if scales is not None:
            _native._check(_native.lib().dqgemm_run_fp8_block_quantized(
                self._h, q.data_ptr(), scales.data_ptr(), M, out.data_ptr(), _native.device_stream(stream, self._dev)),
                "dqgemm_run_fp8_block_quantized")
            return out
        dqgemm_run_fp8_static_quantized(self._h, q, M, out, stream)
        return out

    def dequantize(self, stream=None):
        _on_current_device(self.device, "the layer is")
        w = _empty((self.N, self.K), _torch().bfloat16, self.device, stream)
        dqgemm_dequantize(self._h, w, stream)
        return w

    def plan(self, M):
        return dqgemm_get_plan(self._h, M)

    def last_error(self):
        return dqgemm_last_error(self._h)

    @property
    def handle(self):
        return self._h

    # the object owns a library handle (device memory freed by close), so a
    # copy would destroy it twice and a pickle would carry a dead pointer
    def __copy__(self):
        raise TypeError("QuantizedLinear owns a device handle and cannot be copied; build another layer")

    def __deepcopy__(self, memo):
        self.__copy__()

    def __reduce__(self):
        raise TypeError("QuantizedLinear owns a device handle and cannot be pickled")

    def close(self):
        if self._h is not None:
            dqgemm_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class QuantizedExperts:
    """E quantized Linear weights of one shape on the current CUDA device, for
    rows that are grouped by expert: rows ``offsets[e] .. offsets[e + 1]`` go
    through weight e.

    fmt: "fp8_block".  ``packed`` uint8 [E, N, K] and ``scales`` fp32 [E,
    ceil(N / 128), ceil(K / 128)] are the weights' canonical storage (see
    ``storage_shapes``), ``bias`` bf16 [E, N] or None; all copied."""

    def __init__(self, fmt, E, K, N, packed, scales, bias=None):
        import torch

        self._h = None
        if fmt != "fp8_block":
            raise ValueError(f"experts take the format 'fp8_block', not {fmt!r}")
        _require(packed, "packed", shape=(E, N, K), dtype=torch.uint8)
        _require(scales, "scales", shape=(E, (N + 127) // 128, (K + 127) // 128), dtype=torch.float32,
                 device=packed.device)
        if bias is not None:
            _require(bias, "bias", shape=(E, N), dtype=torch.bfloat16, device=packed.device)
        _on_current_device(packed.device, "packed is")
        self.fmt, self.E, self.K, self.N = fmt, E, K, N
        self.device = packed.device
        self._dev = self.device.index
        self._check_current = torch.cuda.device_count() > 1
        self._h = dqgemm_create_experts(fmt, E, K, N, packed, scales, bias)
        # as QuantizedLinear's, by the library's rule for these sizes
        self._few_rows = next((m for m in range(16, 0, -1) if self.plan(m)["workspace_bytes"] == 0), 0)

    @classmethod
    def from_float(cls, fmt, W, bias=None):
        """Quantize CUDA weights [E, N, K] with the GPU packer."""
        import torch

        if not getattr(W, "is_cuda", False) or W.dim() != 3:
            raise ValueError("W must be a 3-D CUDA tensor [E, N, K]")
        _on_current_device(W.device, "W is")
        if fmt != "fp8_block":
            raise ValueError(f"experts take the format 'fp8_block', not {fmt!r}")
        E, N, K = W.shape
        ps, _, ss, _ = storage_shapes(fmt, K, N)
        packed = torch.empty((E, *ps), dtype=torch.uint8, device=W.device)
        scales = torch.empty((E, *ss), dtype=torch.float32, device=W.device)
        for e in range(E):
            dqgemm_pack_device_noalloc(fmt, W[e].detach().to(torch.float32).contiguous(), packed[e], scales[e])
        return cls(fmt, E, K, N, packed, scales, bias)

    # checks and results of one [M, K] operand, as a layer's
    _check_x = QuantizedLinear._check_x
    _out = QuantizedLinear._out

    def _check_offsets(self, offsets):
        t = offsets
        if not (getattr(t, "dtype", None) is _torch().int32 and t.is_cuda and t.dim() == 1 and t.shape[0] == self.E + 1
                and t.is_contiguous() and t.get_device() == self._dev):
            _require(t, "offsets", shape=(self.E + 1,), dtype=_torch().int32, device=self.device)

    def __call__(self, x, offsets, out=None, stream=None):
        """y[m] = x[m] . deq(W_e)^T + b_e for offsets[e] <= m < offsets[e + 1];
        x bf16 [M, K], offsets int32 [E + 1] on the device, not decreasing; y
        (``out``, allocated if None) bf16 [M, N].  Rows that no expert has are
        left as they were (undefined in an allocated y).  Inference only, as the
        row operators: a gradient that reaches y's raises."""
        torch = _torch()
        M = self._check_x(x, torch.bfloat16)
        self._check_offsets(offsets)
        out = self._out(out, M, torch.bfloat16, stream)
        if M:
            _block_call(self, x, M, offsets.data_ptr(), out, stream)
        if x.requires_grad:
            from . import rows

            return rows.no_backward("QuantizedExperts", out, x)
        return out

    def from_codes(self, q, scales, offsets, out=None, stream=None):
        """The same on e4m3 codes uint8 [M, K] with scales fp32 [M, ceil(K / 128)]."""
        torch = _torch()
        M = self._check_x(q, torch.uint8, "q")
        if not _fits(scales, (self.K + 127) // 128, torch.float32, M, self._dev):
            _require(scales, "scales", shape=(M, (self.K + 127) // 128), dtype=torch.float32, device=self.device)
        self._check_offsets(offsets)
        out = self._out(out, M, torch.bfloat16, stream)
        if M:
            _native._check(_native.lib().dqgemm_run_experts_quantized(
                self._h, q.data_ptr(), scales.data_ptr(), M, offsets.data_ptr(), out.data_ptr(),
                _native.device_stream(stream, self._dev)), "dqgemm_run_experts_quantized")
        return out

    def dequantize(self, stream=None):
        _on_current_device(self.device, "the layer is")
        w = _empty((self.E * self.N, self.K), _torch().bfloat16, self.device, stream)
        dqgemm_dequantize(self._h, w, stream)
        return w.view(self.E, self.N, self.K)

    plan = QuantizedLinear.plan
    last_error = QuantizedLinear.last_error
    handle = QuantizedLinear.handle
    close = QuantizedLinear.close
    __del__ = QuantizedLinear.__del__

    def __copy__(self):
        raise TypeError("QuantizedExperts owns a device handle and cannot be copied; build another one")

    def __deepcopy__(self, memo):
        self.__copy__()

    def __reduce__(self):
        raise TypeError("QuantizedExperts owns a device handle and cannot be pickled")


_ROWS = ("rmsnorm", "silu_mul", "quantize_act_fp8_block")


def __getattr__(name):
    # the row operators need torch at import: loaded on first use, as the
    # package itself does without it
    if name in _ROWS:
        from . import rows

        for n in _ROWS:
            globals()[n] = getattr(rows, n)
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
