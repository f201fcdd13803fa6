"""Refusals of the block-scaled layers and experts that need no GPU."""

import ctypes

import pytest
import torch

import weight_only_quantized_prologue_b200 as dq

BAD, UNSUP, ALIGN = dq._native.DQ_ERR_INVALID_ARG, dq._native.DQ_ERR_UNSUPPORTED, dq._native.DQ_ERR_ALIGNMENT


def test_create_refuses_bad_shapes_formats_and_buffers():
    lib, h = dq._native.lib(), ctypes.c_void_p()
    f = dq.FORMATS["fp8_block"]
    assert lib.dqgemm_create(ctypes.byref(h), f, 24, 128, 16, 16, 1.0, None) == BAD
    assert lib.dqgemm_create(ctypes.byref(h), f, 128, 128, None, 16, 1.0, None) == BAD
    assert lib.dqgemm_create(ctypes.byref(h), f, 128, 128, 17, 16, 1.0, None) == ALIGN
    ex = lib.dqgemm_create_experts
    assert ex(None, f, 2, 128, 128, 16, 16, None) == BAD
    assert ex(ctypes.byref(h), f, 0, 128, 128, 16, 16, None) == BAD
    assert ex(ctypes.byref(h), f, 2, 120, 128, 16, 16, None) == BAD
    assert ex(ctypes.byref(h), f, 2, 128, 128, 16, None, None) == BAD
    assert ex(ctypes.byref(h), f, 2, 128, 128, 16, 24, None) == ALIGN
    assert ex(ctypes.byref(h), f, 1025, 128, 128, 16, 16, None) == UNSUP
    assert ex(ctypes.byref(h), 3, 2, 128, 128, 16, 16, None) == UNSUP
    assert ex(ctypes.byref(h), 9, 2, 128, 128, 16, 16, None) == BAD
    assert h.value is None


def test_run_refuses_null_arguments():
    lib = dq._native.lib()
    assert lib.dqgemm_run_fp8_block_quantized(None, 16, 16, 4, 16, None) == BAD
    assert lib.dqgemm_run_experts_quantized(None, 16, 16, 4, 16, 16, None) == BAD
    assert lib.dqgemm_run_fp8_block(None, 16, 4, None, 16, None, 0, None) == BAD


def test_python_layer_refuses_host_tensors():
    with pytest.raises(ValueError, match="CUDA"):
        dq.QuantizedLinear("fp8_block", 128, 128, torch.zeros(128, 128, dtype=torch.uint8), torch.zeros(1, 1))
    with pytest.raises(ValueError, match="CUDA"):
        dq.QuantizedExperts("fp8_block", 2, 128, 128, torch.zeros(2, 128, 128, dtype=torch.uint8), torch.zeros(2, 1, 1))
    with pytest.raises(ValueError, match="fp8_block"):
        dq.QuantizedExperts("nvfp4", 2, 128, 128, None, None)
    with pytest.raises(ValueError, match="3-D CUDA"):
        dq.QuantizedExperts.from_float("fp8_block", torch.zeros(2, 128, 128))


def test_experts_cannot_be_copied_or_pickled():
    import copy
    import pickle

    ex = dq.QuantizedExperts.__new__(dq.QuantizedExperts)
    ex._h = None
    for fn in (copy.copy, copy.deepcopy, pickle.dumps):
        with pytest.raises(TypeError, match="handle"):
            fn(ex)


def test_storage_shapes():
    import numpy as np

    assert dq.storage_shapes("fp8_block", 272, 130) == ((130, 272), np.uint8, (2, 3), np.float32)


def test_packers_take_scales_that_begin_at_any_fp32():
    # an expert's scales lie N / 128 * K / 128 values behind the one's before it
    lib, f = dq._native.lib(), dq.FORMATS["fp8_block"]
    for entry in (lib.dqgemm_pack_device, lib.dqgemm_pack_device_noalloc):
        assert entry(f, 16, 128, 128, 16, 18, None, None) == ALIGN
        assert entry(f, 20, 128, 128, 16, 16, None, None) == ALIGN
        assert entry(f, 16, 128, 128, 20, 16, None, None) == ALIGN
        assert entry(dq.FORMATS["fp8"], 16, 128, 128, 16, 20, None, None) == ALIGN
