"""The product around the numbers of clusters that the device holds at once
(at two CTAs per SM 71 of four and 33 of eight, at one 33 and 15): units that
fill them, one more, and several rounds; long K, so that the units are split."""
import numpy as np
import pytest
import torch

from decode_gemv_tb_b200 import tb
from tests import mx4_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("M,units,K", [(1, 71, 4096), (1, 72, 4096), (16, 74, 4096), (1, 33, 8192), (1, 34, 8192),
                                       (40, 15, 5120), (40, 16, 5120), (61, 16, 17408), (33, 33, 5120), (33, 34, 5120),
                                       (100, 15, 8192), (100, 16, 8192), (128, 34, 8192), (20, 37, 5120), (2, 150, 2304)])
def test_units_around_the_clusters_held(M, units, K):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    N = units * 128 - 5
    rng = np.random.default_rng(M * units)
    w, ws = R.random_mx4(N, K, rng)
    x, xs = R.random_mx4(M, K, rng)
    wd, xd = R.to_gpu(w, ws), R.to_gpu(x, xs)
    Y = torch.full((M, N + 3), 7.0, device=DEV)
    tb.tb_mx4_gemm(*wd, *xd, M, N, K, Y=Y[:, :N])
    assert tb.sync_status() == 0 and torch.all(Y[:, N:] == 7.0)
    W, X = torch.from_numpy(R.values(w, ws)).to(DEV), torch.from_numpy(R.values(x, xs)).to(DEV)
    ref, mag = X @ W.T, X.abs() @ W.abs().T
    assert torch.all((Y[:, :N].double() - ref).abs() <= (K / 64 + 12) * 2.0 ** -23 * mag)
    assert torch.equal(Y[:, :N], tb.tb_mx4_gemm(*wd, *xd, M, N, K))
