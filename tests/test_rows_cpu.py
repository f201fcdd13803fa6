"""Refusals of the row operators, by the Python layer and by the C entry points
(no launch is reached: these run without a GPU)."""

import pytest
import torch

import weight_only_quantized_prologue_b200 as dq

BAD, ALIGN = dq._native.DQ_ERR_INVALID_ARG, dq._native.DQ_ERR_ALIGNMENT
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("fn", ["rmsnorm", "silu_mul", "quantize_act_fp8_block"])
def test_host_tensors_and_wrong_ranks_are_refused(fn):
    f = getattr(dq, fn)
    with pytest.raises(ValueError, match="CUDA"):
        f(torch.zeros(4, 256))
    with pytest.raises(ValueError, match="2-D"):
        f(torch.zeros(4, 2, 256))


def norm(type_=0, x=64, ldx=256, res=None, res_out=None, wt=0, w=None, eps=1e-6, M=2, K=256, out=0, s_out=1.0, o=64,
         sc=64):
    return dq._native.lib().dqgemm_rmsnorm(type_, x, ldx, res, res_out, wt, w, eps, M, K, out, s_out, o, sc, None)


@pytest.mark.parametrize("kw", [{"type_": 3}, {"type_": -1}, {"x": None}, {"o": None}, {"M": 0}, {"K": 0},
                                {"ldx": 255}, {"res": 64}, {"res_out": 64}, {"wt": 3}, {"eps": -1.0}, {"eps": NAN},
                                {"eps": INF}, {"out": 5}, {"out": -1}, {"out": 3, "sc": None},
                                {"out": 4, "s_out": 0.0}, {"out": 4, "s_out": NAN}, {"out": 4, "s_out": INF},
                                {"K": (1 << 28) + 8, "ldx": 1 << 40}, {"res": 128, "res_out": 64}])
def test_rmsnorm_refuses_bad_arguments(kw):
    assert norm(**kw) == BAD


@pytest.mark.parametrize("kw", [{"x": 65}, {"o": 65}, {"w": 65}, {"res": 65, "res_out": 128},
                                {"res": 256, "res_out": 129}, {"out": 3, "o": 1, "sc": 66}, {"type_": 2, "x": 66},
                                {"wt": 2, "w": 66}, {"out": 2, "o": 66}])
def test_rmsnorm_refuses_unaligned_buffers(kw):
    assert norm(**kw) == ALIGN


def test_silu_mul_and_quantizer_refuse_bad_arguments():
    lib = dq._native.lib()
    assert lib.dqgemm_silu_mul(0, 64, 511, 2, 256, 0, 1.0, 64, None, None) == BAD      # a row holds 2K columns
    assert lib.dqgemm_silu_mul(0, None, 512, 2, 256, 0, 1.0, 64, None, None) == BAD
    assert lib.dqgemm_silu_mul(0, 64, 512, 2, 256, 3, 1.0, 64, None, None) == BAD
    assert lib.dqgemm_silu_mul(0, 64, 512, 2, 256, 4, -1.0, 64, None, None) == BAD
    assert lib.dqgemm_silu_mul(2, 66, 512, 2, 256, 0, 1.0, 64, None, None) == ALIGN
    assert lib.dqgemm_silu_mul(0, 64, 1 << 30, 2, 1 << 29, 0, 1.0, 64, None, None) == BAD
    assert lib.dqgemm_quantize_act_fp8_block(0, 64, 256, 2, 256, 64, None, None) == BAD
    assert lib.dqgemm_quantize_act_fp8_block(0, 64, 256, 2, 256, None, 64, None) == BAD
    assert lib.dqgemm_quantize_act_fp8_block(0, 64, 100, 2, 256, 64, 64, None) == BAD


class Fake:
    """Stands in for a CUDA tensor: the checks read metadata only."""

    def __init__(self, t, dev=0):
        self.t, self.is_cuda, self.device, self.dtype, self.shape = t, True, torch.device("cuda", dev), t.dtype, t.shape

    def __getattr__(self, n):
        return getattr(self.t, n)


def test_layouts_and_types_are_refused():
    from weight_only_quantized_prologue_b200 import rows

    z = torch.zeros(4, 256, dtype=torch.bfloat16)
    assert rows._rows(Fake(z), "x") == (4, 256, 256)
    assert rows._rows(Fake(z[:, :100]), "x") == (4, 100, 256)
    assert rows._rows(Fake(z[:1, 3:10]), "x") == (1, 7, 7)
    assert rows._rows(Fake(z), "x", 2) == (4, 128, 256)
    with pytest.raises(ValueError, match="contiguous"):
        rows._rows(Fake(z.t()), "x")
    with pytest.raises(ValueError, match="overlap"):
        rows._rows(Fake(z[:1].expand(4, 256)), "x")
    with pytest.raises(TypeError, match="float64"):
        rows._rows(Fake(z.double()), "x")
    with pytest.raises(ValueError, match="halves"):
        rows._rows(Fake(z[:, :255]), "x", 2)
    with pytest.raises(ValueError, match="column"):
        rows._rows(Fake(z[:, :0]), "x")


def test_output_arguments_are_refused():
    from weight_only_quantized_prologue_b200 import rows

    x = Fake(torch.zeros(4, 256, dtype=torch.bfloat16))
    for args in [("fp8_row", None, None), ("fp8_static", None, None), ("fp8_static", 0.0, None),
                 ("fp8_static", INF, None), ("fp8_block", 0.1, None), ("fp8_block", None, torch.float16),
                 (None, 0.1, None)]:
        with pytest.raises(ValueError):
            rows._outputs(x, 4, 256, *args, Fake(torch.zeros(4, 256, dtype=torch.uint8)), None)
    with pytest.raises(TypeError):
        rows._outputs(x, 4, 256, None, None, torch.int8, None, None)
    with pytest.raises(ValueError, match="shape"):
        rows._outputs(x, 4, 256, "fp8_block", None, None, Fake(torch.zeros(4, 255, dtype=torch.uint8)), None)


def test_a_gradient_that_would_be_missing_is_an_error():
    from weight_only_quantized_prologue_b200 import rows

    x, y, w = torch.ones(3, requires_grad=True), torch.zeros(3), torch.ones(3)
    out = rows.no_backward("rmsnorm", y, x, None, w)
    assert out.requires_grad and out.data_ptr() == y.data_ptr() and not y.requires_grad
    with pytest.raises(RuntimeError, match="rmsnorm is inference only"):
        (out + x).sum().backward()
    assert rows.no_backward("rmsnorm", y, w, None) is y
    with torch.no_grad():
        assert rows.no_backward("rmsnorm", y, x) is y


def test_sizes_beyond_the_librarys_32_bit_numbers_are_refused():
    from weight_only_quantized_prologue_b200 import rows

    def huge(*shape):        # metadata only: no memory behind it
        return Fake(torch.empty(shape, dtype=torch.bfloat16, device="meta"))

    for x in (huge(1 << 31, 1), huge((1 << 32) + 5, 1), huge(1, (1 << 28) + 1), huge(2, (1 << 32) + 256)):
        with pytest.raises(ValueError, match="2.31 rows and at most 2.28"):
            rows._rows(x, "x")
    with pytest.raises(ValueError, match="a half"):
        rows._rows(huge(1, (1 << 29) + 2), "x", 2)
    assert rows._rows(huge(1, 1 << 29), "x", 2) == (1, 1 << 28, 1 << 29)
    assert rows._rows(huge((1 << 31) - 1, 1), "x") == ((1 << 31) - 1, 1, 1)
    lin = dq.QuantizedLinear.__new__(dq.QuantizedLinear)
    lin._h, lin.fmt, lin.K, lin.N, lin.device, lin._dev, lin._check_current = None, "fp8_block", 16, 16, torch.device("cuda", 0), 0, False
    with pytest.raises(ValueError, match="2.31 rows"):
        lin._check_x(Fake(torch.empty(((1 << 32) + 5, 16), dtype=torch.uint8, device="meta")), torch.uint8, "q")
