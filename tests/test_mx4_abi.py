"""The 4-bit format's entry points on the host: sizes in closed form and
every refusal before anything is launched, and the reference implementation
of the format against worked blocks."""
import numpy as np
import pytest

from decode_gemv_tb_b200 import build as tbbuild
from decode_gemv_tb_b200 import tb
from tests import mx4_ref as R

A = 1 << 40  # aligned, never dereferenced
ARG, SHAPE, ALIGN = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    tbbuild.build()
    return tb.load()


def test_sizes(lib):
    for N, K in ((1, 32), (1, 4096), (127, 96), (128, 128), (129, 160), (17408, 5120)):
        assert tb.mx4_code_bytes(N, K) == N * K // 2
        assert tb.mx4_scale_bytes(N, K) == 512 * ((N + 127) // 128) * ((K + 127) // 128)
        idx = R.scale_index(N, K)
        assert idx.max() < tb.mx4_scale_bytes(N, K) and len(np.unique(idx)) == idx.size
    for N, K in ((0, 32), (-1, 32), (1, 0), (1, 16), (1, 33), (1, -32), (1 << 31, 32), (1, 1 << 31)):
        assert tb.mx4_code_bytes(N, K) == 0 and tb.mx4_scale_bytes(N, K) == 0


def test_quantize_refusals(lib):
    for f in ((lambda W=A, dt=0, ld=64, N=4, K=64, c=A, s=A, b=0: lib.tb_mx4_quantize(W, dt, ld, N, K, c, s, b, 0)),
              (lambda W=A, dt=0, ld=64, N=4, K=64, c=A, s=A, b=0: lib.tb_mx4_dequantize(c, s, N, K, W, dt, ld, 0))):
        assert f(W=0) == ARG and f(c=0) == ARG and f(s=0) == ARG and f(dt=2) == ARG
        assert f(N=0) == SHAPE and f(K=48) == SHAPE and f(K=0) == SHAPE and f(ld=60) == SHAPE and f(ld=-64) == SHAPE
        assert f(W=A + 8) == ALIGN and f(ld=66) == ALIGN and f(c=A + 8) == ALIGN and f(s=A + 4) == ALIGN
        assert f(dt=1, ld=68) == ALIGN
    assert lib.tb_mx4_quantize(A, 0, 64, 4, 64, A, A, A + 2, 0) == ALIGN


def test_gemm_refusals(lib):
    def f(wc=A, ws=A, xc=A, xs=A, Y=A, dt=0, ld=64, M=4, N=64, K=64, flags=0):
        return lib.tb_mx4_gemm(wc, ws, xc, xs, Y, dt, ld, M, N, K, flags, 0)
    for name in ("wc", "ws", "xc", "xs"):
        assert f(**{name: 0}) == ARG and f(**{name: A + 8}) == ALIGN
    assert f(Y=0) == ARG and f(dt=2) == ARG and f(flags=1) == ARG and f(flags=4) == ARG
    assert f(M=0) == SHAPE and f(M=65537) == SHAPE and f(N=0) == SHAPE and f(K=40) == SHAPE and f(ld=63) == SHAPE
    assert f(N=1 << 31, ld=1 << 31) == SHAPE and f(M=65536, N=(1 << 31) - 1, ld=1 << 31) == SHAPE
    assert f(Y=A + 2) == ALIGN and f(Y=A + 1, dt=1) == ALIGN


def test_binding_refusals():
    """The binding's own checks, on CPU tensors (nothing is launched)."""
    import torch
    w = torch.zeros(4, 64)
    for bad in (torch.zeros(4, 40), torch.zeros(4, 64)):
        with pytest.raises(tb.TBError):
            tb.tb_mx4_quantize(bad)  # K % 32, then: not on the GPU
    with pytest.raises(tb.TBError):
        tb.tb_mx4_quantize(w.t().contiguous().t())  # rows not contiguous
    with pytest.raises(tb.TBError):
        tb.tb_mx4_dequantize(w.to(torch.uint8), w.to(torch.uint8), 4, 64)


def test_reference_on_worked_blocks():
    """amax 7 -> scale 2^0: 7 saturates at 6, ties go to the even code; a block of zeros gets byte 0; a
    non-finite value does not enter the scale."""
    w = np.zeros((1, 96))
    w[0, :12] = [7, -7, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, 0.26, 5.01]
    w[0, 64:68] = [np.nan, np.inf, -np.inf, 2.0 ** -10]
    codes, b, bad = R.quantize(w)
    assert b[0].tolist() == [127, 0, 127 - 12] and bad == 3
    assert R.VALUES[codes[0, :12]].tolist() == [6, -6, 0, 1, 1, 2, 2, 4, 4, 0, 0.5, 6]
    assert R.VALUES[codes[0, 64:68]].tolist() == [0, 6, -6, 4]
    packed = R.pack(codes)
    assert packed[0, 0] == 0xF7 and packed.shape == (1, 48)
    assert R.scale_index(130, 160)[129, 4] == (1 * 2 + 1) * 512 + 16 * 1 + 4 * 0 + 0
