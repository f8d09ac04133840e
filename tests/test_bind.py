"""The native calls' own checks: whatever is passed, an exception and no
call into the library (nothing here reaches a GPU)."""
import pytest
import torch

from decode_gemv_tb_b200 import build as tbbuild
from decode_gemv_tb_b200 import tb


@pytest.fixture(scope="module")
def bind():
    tbbuild.build()
    tb.load()
    return tb._bind


W = torch.zeros(4, 64)
U8 = torch.zeros(4096, dtype=torch.uint8)
X = torch.zeros((2, 128), dtype=torch.bfloat16)
IDS, WEIGHTS = torch.zeros((2, 1), dtype=torch.int32), torch.zeros((2, 1))
Y = torch.zeros(2, 4)


@pytest.mark.parametrize("name,args,what", [
    ("mx4_quantize", (W, U8, U8, None, None), "CUDA tensors"),
    ("mx4_quantize", (W[0], U8, U8, None, None), "two dimensions"),
    ("mx4_quantize", (W[:, :40], U8, U8, None, None), "multiple of 32"),
    ("mx4_quantize", (W.t().contiguous().t(), U8, U8, None, None), "contiguous"),
    ("mx4_quantize", (W, None, U8, None, None), "codes must be a tensor"),
    ("mx4_quantize", (W, U8, U8, 7, None), "bad_count must be a tensor"),
    ("mx4_dequantize", (U8, U8, 4, 64, W, None), "CUDA tensors"),
    ("mx4_dequantize", (U8, U8, 4, 2 ** 40, W, None), "2\\^31"),
    ("mx4_dequantize", (U8, U8, 4, 2 ** 70, W, None), "64 bits"),
    ("mx4_dequantize", (U8, U8, "4", 64, W, None), "integers"),
    ("mx4_dequantize", (U8, U8, 0, 64, W, None), "N >= 1"),
    ("mx4_gemm", (U8, U8, U8, U8, 2, 4, 64, Y, 0, None), "CUDA tensors"),
    ("mx4_gemm", (U8, U8, U8, U8, 0, 4, 64, Y, 0, None), "N >= 1"),
    ("mx4_gemm", (U8, U8, U8, [], 2, 4, 64, Y, 0, None), "x_scales must be a tensor"),
    ("moe_route", (X, X, 1, True, IDS, WEIGHTS, None), "CUDA tensors"),
    ("moe_route", (X, X.float(), 1, True, IDS, WEIGHTS, None), "router must hold bf16"),
    ("moe_route", (X, X[:, :64], 1, True, IDS, WEIGHTS, None), "router must be \\[2\\]\\[128\\]"),
    ("moe_route", (X, torch.zeros((2, 256), dtype=torch.bfloat16)[:, :128], 1, True, IDS, WEIGHTS, None), "contiguous"),
    ("moe_route", (X.to_sparse(), X, 1, True, IDS, WEIGHTS, None), "."),
    ("moe", (0, 128, 0, X, IDS, WEIGHTS, Y, U8, 0, None), "CUDA tensors"),
    ("moe", (0, 64, 0, X, IDS, WEIGHTS, Y, U8, 0, None), "x must be \\[2\\]\\[64\\]"),
])
def test_refusals(bind, name, args, what):
    with pytest.raises(tb.TBError, match=what):
        getattr(bind, name)(*args)


def test_argument_counts(bind):
    for name in ("init", "mx4_quantize", "mx4_dequantize", "mx4_gemm", "moe_route", "moe"):
        with pytest.raises(TypeError):
            getattr(bind, name)(None)


def test_stays_in_step_with_the_library(bind):
    for name in tb.BOUND:
        assert name in tb.SIGNATURES


@pytest.mark.gpu
def test_refusals_on_the_gpu(bind):
    """Checks that need tensors on the device; the library's own refusals with their text."""
    dev = "cuda:0"
    w, u8, x, ids, wt, y = (t.to(dev) for t in (W, U8, X, IDS, WEIGHTS, Y))
    for name, args, what in (
            ("mx4_quantize", (w, u8[:64], u8, None, None), "codes must hold at least 128 bytes"),
            ("mx4_quantize", (w, u8, u8[:511], None, None), "scales must hold at least 512"),
            ("mx4_quantize", (w, u8, u8.float(), None, None), "scales must hold"),
            ("mx4_quantize", (w.double(), u8, u8, None, None), "weights must be float32 or bfloat16"),
            ("mx4_quantize", (w, u8[::2], u8, None, None), "codes must be contiguous"),
            ("mx4_quantize", (w, u8[1:], u8, None, None), "TB_ERR_ALIGN"),
            ("mx4_quantize", (w, u8, u8, wt, None), "bad_count must be int32"),
            ("mx4_quantize", (w, U8, u8, None, None), "different devices"),
            ("mx4_quantize", (w, u8, u8, None, "s"), "stream"),
            ("mx4_gemm", (u8, u8, u8, u8, 2, 4, 64, y.half(), 0, None), "Y must be float32 or bfloat16"),
            ("mx4_gemm", (u8, u8, u8, u8, 2, 4, 64, y, 1, None), "TB_ERR_ARG"),
            ("mx4_gemm", (u8, u8, u8, u8, 2, 4, 64, y, 1 << 32, None), "32 bits"),
            ("mx4_gemm", (u8, u8, u8, u8, 2, 4, 64, y.t(), 0, None), "Y must be \\[2\\]\\[4\\]"),
            ("moe_route", (x, x, 3, True, ids, wt, None), "weights must be|ids must be"),
            ("moe_route", (x, x, 1, True, ids.long(), wt, None), "ids must be contiguous"),
            ("moe_route", (x, x, 17, True, ids, wt, None), "TB_ERR_ARG"),
            ("moe", (0, 128, 0, x, ids, wt, y, u8, 0, None), "y must be"),
            ("moe", (0, 128, 0, x, ids, wt, x.float(), u8, 0, None), "TB_ERR_ARG"),  # no layer
            ("moe", (0, 128, 1, x, ids, wt, x.float(), u8, 0, None), "the layer on cuda:1")):
        with pytest.raises(tb.TBError, match=what):
            getattr(bind, name)(*args)
