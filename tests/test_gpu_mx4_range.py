"""4-bit products and expert layers at both ends of fp32's range: the bounds
of include/tb.h with their absolute terms, the largest scale byte that the
quantiser writes, and where sums pass the range."""
import numpy as np
import pytest
import torch

from decode_gemv_tb_b200 import tb
from tests import mx4_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tb.load()


@pytest.mark.parametrize("M,N,K", [(1, 130, 64), (3, 300, 2048), (40, 257, 512), (300, 9472, 288)])
@pytest.mark.parametrize("lo,hi", [(20, 70), (45, 60), (0, 55)])
def test_products_below_the_normal_range(M, N, K, lo, hi):
    """Scales so small that products, or sums, fall below 2^-126 and 2^-149: a product may lose what is below 2^-149."""
    rng = np.random.default_rng(M + lo)
    w, ws = R.random_mx4(N, K, rng, lo, hi)
    x, xs = R.random_mx4(M, K, rng, lo, hi)
    ref = torch.from_numpy(R.values(x, xs)).to(DEV) @ torch.from_numpy(R.values(w, ws)).to(DEV).T
    mag = torch.from_numpy(np.abs(R.values(x, xs))).to(DEV) @ torch.from_numpy(np.abs(R.values(w, ws))).to(DEV).T
    for dt in (torch.float32, torch.bfloat16):
        Y = tb.tb_mx4_gemm(*R.to_gpu(w, ws), *R.to_gpu(x, xs), M, N, K, out_dtype=dt)
        tol = (K / 64 + 12) * 2.0 ** -23 * mag + K * 2.0 ** -149
        if dt == torch.bfloat16:
            tol = tol + 2.0 ** -8 * ref.abs() + 2.0 ** -134
        assert torch.all((Y.double() - ref).abs() <= tol), (((Y.double() - ref).abs() - tol).max() / 2.0 ** -149).item()


def test_products_near_and_past_the_range():
    """sum |x w| just below 2^127 keeps its bound; past the range the sign is right; zeros stay zeros."""
    N, M, K = 130, 5, 256
    w, x = np.full((N, K), 2), np.full((M, K), 2)  # 1.0 everywhere
    x[1] = 10  # -1.0
    x[2] = 0
    for e, finite in ((126, True), (128, False), (250, False)):
        total = e - 8 + 254  # K = 2^8 products of 2^(total - 254)
        a = total // 2
        ws, xs = np.full((N, K // 32), a, np.uint8), np.full((M, K // 32), total - a, np.uint8)
        Y = tb.tb_mx4_gemm(*R.to_gpu(w, ws), *R.to_gpu(x, xs), M, N, K).double().cpu()
        want = 2.0 ** e if finite else float("inf")
        assert torch.all(Y[0] == want) and torch.all(Y[1] == -want) and torch.all(Y[2] == 0.0) and torch.all(Y[3:] == want)


def layer_of(H, I, E, bytes_, rng):
    """MX4 matrices with scale bytes in the given ranges; (values of gate, up, down), layer."""
    mats, parts = [], []
    for (rows, cols), (lo, hi) in zip(((E * I, H), (E * I, H), (E * H, I)), bytes_):
        c, b = R.random_mx4(rows, cols, rng, lo, hi + 1)
        mats.append(torch.from_numpy(R.values(c, b)).to(DEV))
        parts.append((*R.to_gpu(c, b), R.MX4))
    return mats, tb.moe_layer(*parts, E, H, I)


def bound(wg, wu, wd, E, x, ids, weights):
    """(y, bound) of include/tb.h with its absolute terms, in float64"""
    T, H = x.shape
    I, k, u, tiny = wd.shape[1], ids.shape[1], 2.0 ** -24, 2.0 ** -126
    x, weights = x.double(), weights.double()
    y, tol = torch.zeros_like(x), torch.full_like(x, tiny)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            G, U, D = wg[e * I:(e + 1) * I], wu[e * I:(e + 1) * I], wd[e * H:(e + 1) * H]
            g, up = G @ x[t], U @ x[t]
            dg, du = ((H / 8 + 16) * u * (m.abs() @ x[t].abs()) + tiny for m in (G, U))
            s = g * torch.sigmoid(g)
            h = s * up
            dh = 1.1 * dg * (up.abs() + du) + s.abs() * du + 2.0 ** -8 * h.abs() + tiny
            y[t] += weights[t, j] * (D @ h)
            tol[t] += weights[t, j].abs() * (D.abs() @ dh + (I / 8 + k + 24) * u * (D.abs() @ (h.abs() + dh)) + tiny)
    return y, tol


@pytest.mark.parametrize("name,exps,bytes_", [
    # every scale at the quantiser's largest, activations that bring the sums back; down's on h of about 2^-60
    ("gate and up at 252", -126, ((248, 252), (248, 252), (118, 123))),
    ("down at 252", -30, ((118, 123), (118, 123), (245, 252))),
    # everything small: products and h below the normal range
    ("small", -50, ((40, 127), (40, 127), (60, 127))),
    ("h below the normal range, brought back", -12, ((66, 72), (66, 72), (240, 250))),
    ("smallest", -120, ((0, 30), (0, 30), (0, 252))),
])
@pytest.mark.parametrize("T", [2, 24])
def test_layers_at_the_ends_of_the_range(name, exps, bytes_, T):
    E, H, I, k = 2, 256, 128, 2
    rng = np.random.default_rng(T)
    mats, layer = layer_of(H, I, E, bytes_, rng)
    g = torch.Generator().manual_seed(T)
    x = (torch.randn((T, H), generator=g) * 2.0 ** exps).to(torch.bfloat16).to(DEV)
    x[1] = 0.0  # decoded values that were infinite would make this row NaN
    ids = torch.tensor([[0, 1], [1, 0]] * (T // 2), dtype=torch.int32)
    w = torch.rand((T, k), generator=g).to(DEV)
    y = tb.tb_moe(layer, x, ids.to(DEV), w).double()
    ref, tol = bound(*mats, E, x, ids, w)
    assert torch.all(y[1] == 0.0)
    assert torch.isfinite(ref).all() and ref.abs().max() < 2.0 ** 127
    assert torch.all((y - ref).abs() <= tol), name


def test_quantiser_never_writes_a_larger_scale():
    w = torch.full((4, 64), torch.finfo(torch.float32).max, device=DEV)
    w[1, :32], w[2] = -torch.finfo(torch.float32).max, float("inf")
    _, s = tb.tb_mx4_quantize(w)
    idx = torch.from_numpy(R.scale_index(4, 64)[:, :2].reshape(-1)).to(DEV)
    assert s[idx].max().item() == 252
