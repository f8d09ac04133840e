"""The 4-bit format on the GPU against 64-bit implementations of its
definition: quantisation bit for bit, its inverse exactly, the product
within its bound
    |y - y_exact| <= (K/64 + 12) 2^-23 sum_k |x_k w_k|  (+ 2^-8 |y|, bf16):
products of 4-bit values and powers of two are exact; an MMA adds 64 of them
to the running fp32 sum, a step that loses at most one unit in the last place
(2^-23) of a sum no larger than sum |x w|; a chunk split over up to eight
CTAs adds at most eight more such roundings, alignment inside the steps and
the final one the rest."""
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


def wide(t, extra):
    """t's values in rows of a wider buffer."""
    buf = torch.full((t.shape[0], t.shape[1] + extra), 7.0, dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


def check_quantize(w, extra=0):
    N, K = w.shape
    ref_codes, ref_bytes, ref_bad = R.quantize(w.double().numpy())
    W = wide(w.to(DEV), extra)
    scales = torch.full((tb.mx4_scale_bytes(N, K),), 0xAB, dtype=torch.uint8, device=DEV)
    bad = torch.full((1,), -5, dtype=torch.int32, device=DEV)
    codes, scales = tb.tb_mx4_quantize(W, scales=scales, bad_count=bad)
    assert np.array_equal(codes.cpu().numpy(), R.pack(ref_codes))
    want = np.full(scales.numel(), 0xAB, dtype=np.uint8)  # rows past N stay as they were
    idx = R.scale_index(N, K)
    want[idx] = 0
    want[idx[:, : K // 32]] = ref_bytes
    assert np.array_equal(scales.cpu().numpy(), want)
    assert bad.item() == ref_bad
    values = R.values(ref_codes, ref_bytes)
    for dt in (torch.float32, torch.bfloat16):
        out = torch.full((N, K + 8), 3.0, dtype=dt, device=DEV)
        tb.tb_mx4_dequantize(codes, scales, N, K, W=out[:, :K])
        assert torch.equal(out[:, :K].double().cpu(), torch.from_numpy(values).to(dt).double())
        assert torch.all(out[:, K:] == 3.0)


@pytest.mark.parametrize("N,K", [(1, 32), (1, 96), (1, 4096), (3, 160), (31, 544), (130, 288), (128, 128), (517, 5120)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("extra", [0, 8])
def test_quantize(N, K, dtype, extra):
    g = torch.Generator().manual_seed(N * 7 + K)
    w = torch.randn((N, K), generator=g) * torch.exp(torch.randn((N, 1), generator=g))
    check_quantize(w.to(dtype), extra)


def test_quantize_special_values():
    """Ties of every kind, exact powers of two, zeros of both signs, subnormals, the largest floats, NaN and
    infinities alone and among others."""
    grid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.99, 4.0, 0.2500001, 0.7499999, 1e-30, 0.0, -0.0])
    rows = [torch.cat([grid, -grid]) * 2.0 ** e for e in (-140, -130, -127, -126, -124, -20, 0, 13, 120, 125)]
    top = torch.zeros(32)
    top[:4] = torch.tensor([3.4028234e38, -3.4028234e38, 1e38, 1e-45])
    tiny = torch.zeros(32)
    tiny[:3] = torch.tensor([1e-45, -3e-45, 1.1754944e-38])
    mixed = torch.linspace(-3, 3, 32)
    mixed[5], mixed[6], mixed[7] = float("nan"), float("inf"), -float("inf")
    only = torch.full((32,), float("nan"))
    only[1::2] = float("inf")
    only[3] = -float("inf")
    rows += [top, tiny, mixed, only, torch.zeros(32), -torch.zeros(32)]
    w = torch.stack(rows)
    check_quantize(w)
    check_quantize(w.reshape(4, -1))
    check_quantize(w.to(torch.bfloat16))


def test_dequantize_extreme_scales():
    """Every scale byte: below the normal range, above fp32's (infinite), 255 (NaN)."""
    codes = np.tile(np.arange(32) % 16, (256, 1))
    b = np.arange(256, dtype=np.uint8)[:, None]
    c, s = R.to_gpu(codes, b)
    with np.errstate(over="ignore"):
        want = torch.from_numpy(R.values(codes, b))
    for dt in (torch.float32, torch.bfloat16):
        got = tb.tb_mx4_dequantize(c, s, 256, 32, out_dtype=dt).double().cpu()
        assert torch.equal(torch.nan_to_num(got, nan=-1e300), torch.nan_to_num(want.to(dt).double(), nan=-1e300))


def check_gemm(w, ws, x, xs, dt=torch.float32, extra=0, what=""):
    N, K = w.shape
    M = x.shape[0]
    Y = torch.full((M, N + extra), 7.0, dtype=dt, device=DEV)
    tb.tb_mx4_gemm(*R.to_gpu(w, ws), *R.to_gpu(x, xs), M, N, K, Y=Y[:, :N])
    assert tb.sync_status() == 0
    assert torch.all(Y[:, N:] == 7.0)
    W, X = torch.from_numpy(R.values(w, ws)).to(DEV), torch.from_numpy(R.values(x, xs)).to(DEV)
    ref, mag = X @ W.T, X.abs() @ W.abs().T
    tol = (K / 64 + 12) * 2.0 ** -23 * mag + (2.0 ** -8 * ref.abs() if dt == torch.bfloat16 else 0)
    err = (Y[:, :N].double() - ref).abs()
    assert torch.all(err <= tol), (what, M, N, K, (err - tol).max().item())
    return Y


SHAPES = [(1, 1, 32), (1, 128, 64), (1, 130, 96), (1, 4096, 4096), (2, 7, 288), (15, 129, 160), (16, 300, 512),
          (17, 128, 2048), (32, 100, 1056), (33, 257, 256), (61, 1000, 5120), (64, 128, 17408), (65, 130, 128),
          (127, 2048, 224), (128, 64, 4096), (129, 300, 544), (255, 128, 1024), (257, 1000, 96), (300, 20000, 256),
          (517, 9600, 320)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_gemm(M, N, K, dt):
    rng = np.random.default_rng(M * 131 + N * 7 + K)
    w, ws = R.random_mx4(N, K, rng)
    x, xs = R.random_mx4(M, K, rng)
    check_gemm(w, ws, x, xs, dt, extra=3 if N % 2 else 0)


@pytest.mark.parametrize("M,N,K,extra", [(200, 6000, 288, 0), (200, 6000, 288, 8), (385, 5001, 1088, 7), (385, 5001, 1088, 8),
                                         (1000, 4500, 96, 4), (300, 20000, 544, 4), (300, 20000, 544, 5)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_gemm_prefill_tiles(M, N, K, extra, dt):
    """Tiles of 128 and of 256 rows of W, ragged in every direction; row lengths that are multiples of 16 bytes and
    ones that are not."""
    rng = np.random.default_rng(M + N + K)
    w, ws = R.random_mx4(N, K, rng)
    x, xs = R.random_mx4(M, K, rng)
    check_gemm(w, ws, x, xs, dt, extra)


def test_gemm_persistent_units():
    """More units than the GPU holds at once: every CTA takes several."""
    rng = np.random.default_rng(5)
    w, ws = R.random_mx4(6000, 288, rng)
    x, xs = R.random_mx4(3000, 288, rng)
    check_gemm(w, ws, x, xs, torch.bfloat16)


def test_gemm_is_exact_on_small_sums():
    """Scales of one, K = 64: every sum is a multiple of 1/4 below 2^24/4, so the result is exact."""
    rng = np.random.default_rng(6)
    w, x = rng.integers(0, 16, (200, 64)), rng.integers(0, 16, (70, 64))
    ws, xs = np.full((200, 2), 127, np.uint8), np.full((70, 2), 127, np.uint8)
    Y = tb.tb_mx4_gemm(*R.to_gpu(w, ws), *R.to_gpu(x, xs), 70, 200, 64)
    ref = R.values(x, xs) @ R.values(w, ws).T
    assert np.array_equal(Y.cpu().numpy().astype(np.float64), ref)


def test_gemm_nan_scale_stays_in_its_row():
    """A NaN scale makes its row's outputs NaN and no others; bytes of rows past the last are never used."""
    rng = np.random.default_rng(7)
    w, ws = R.random_mx4(130, 160, rng)
    x, xs = R.random_mx4(20, 160, rng)
    ws[129, 4] = 255
    xs[3, 0] = 255
    wc, wt = R.to_gpu(w, ws)
    xc, xt = R.to_gpu(x, xs)
    for t, n in ((wt, 130), (xt, 20)):  # the rows past the last hold NaN scales
        keep = torch.zeros(t.numel(), dtype=torch.bool)
        keep[torch.from_numpy(R.scale_index(n, 160).reshape(-1))] = True
        t[~keep.to(DEV)] = 255
    Y = tb.tb_mx4_gemm(wc, wt, xc, xt, 20, 130, 160)
    nan = torch.isnan(Y).cpu()
    want = torch.zeros(20, 130, dtype=torch.bool)
    want[3, :] = True
    want[:, 129] = True
    assert torch.equal(nan, want)


def test_gemm_repeats_bitwise_and_in_a_graph():
    rng = np.random.default_rng(8)
    w, ws = R.random_mx4(4096, 2048, rng)
    x, xs = R.random_mx4(5, 2048, rng)
    args = (*R.to_gpu(w, ws), *R.to_gpu(x, xs), 5, 4096, 2048)
    first = tb.tb_mx4_gemm(*args)
    for _ in range(3):
        assert torch.equal(first, tb.tb_mx4_gemm(*args))
    Y = torch.zeros_like(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tb.tb_mx4_gemm(*args, Y=Y)  # a stream of its own
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, Y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tb.tb_mx4_gemm(*args, Y=Y)
    Y.zero_()
    for _ in range(2):
        g.replay()
    assert torch.equal(first, Y) and tb.sync_status() == 0


def test_quantized_linear_run():
    """Quantise weights and a batch, multiply, against the 64-bit product of the quantised values."""
    g = torch.Generator().manual_seed(9)
    W = torch.randn((300, 512), generator=g).mul_(0.02)
    X = torch.randn((9, 512), generator=g).to(torch.bfloat16)
    wc, ws = tb.tb_mx4_quantize(W.to(DEV))
    xc, xs = tb.tb_mx4_quantize(X.to(DEV))
    Y = tb.tb_mx4_gemm(wc, ws, xc, xs, 9, 300, 512)
    w = R.values(*R.quantize(W.double().numpy())[:2])
    x = R.values(*R.quantize(X.double().numpy())[:2])
    err = np.abs(Y.double().cpu().numpy() - x @ w.T)
    assert np.all(err <= (512 / 64 + 12) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T))


def test_gemm_waits_that_give_up_are_reported():
    """The copies are never issued: every wait gives up after about 10 ms, the outputs are NaN, the status says
    so, and the next call is correct."""
    rng = np.random.default_rng(10)
    for M, N in ((3, 256), (200, 19200)):  # a cluster's split and a persistent grid
        w, ws = R.random_mx4(N, 512, rng)
        x, xs = R.random_mx4(M, 512, rng)
        Y = torch.zeros((M, N), device=DEV)
        tb.tb_mx4_gemm(*R.to_gpu(w, ws), *R.to_gpu(x, xs), M, N, 512, Y=Y, flags=tb.FLAG_TEST_STALL)
        assert tb.sync_status() == 6
        assert torch.isnan(Y).all()
        check_gemm(w, ws, x, xs)


def test_calls_at_once_on_two_streams():
    """Split and persistent products of two streams at the same time, beside the scalar grids' product, which takes
    tensor memory too."""
    rng = np.random.default_rng(11)
    shapes = [(5, 4096, 2048), (40, 6000, 1056), (100, 2048, 2048), (300, 9000, 512)]
    args = []
    for M, N, K in shapes:
        w, ws = R.random_mx4(N, K, rng)
        x, xs = R.random_mx4(M, K, rng)
        args.append((*R.to_gpu(w, ws), *R.to_gpu(x, xs), M, N, K))
    want = [tb.tb_mx4_gemm(*a) for a in args]
    wd, dense = R.random_matrix(4096, 2048, R.INT3, rng)
    X = torch.from_numpy(rng.standard_normal((64, 2048))).to(torch.bfloat16).to(DEV)
    y0 = tb.tb_gemm(dense[0], dense[2], dense[1], X, 4096, 2048)
    wsp = tb.workspace(tb.workspace_bytes(64, 4096, 2048), DEV)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    out, dout = [[], []], []
    for i in range(6):
        for s in range(2):
            with torch.cuda.stream(streams[s]):
                for j in range(4):
                    out[s].append(tb.tb_mx4_gemm(*args[(j + 2 * s) % 4]))
        with torch.cuda.stream(streams[2]):
            dout.append(tb.tb_gemm(dense[0], dense[2], dense[1], X, 4096, 2048, ws=wsp))
    torch.cuda.synchronize()
    for s in range(2):
        for i, y in enumerate(out[s]):
            assert torch.equal(y, want[(i % 4 + 2 * s) % 4])
    assert all(torch.equal(y, y0) for y in dout) and tb.sync_status() == 0


def test_quantize_replays_with_its_count():
    """The count is set anew by every replay, beside whatever it held."""
    W = torch.randn((600, 1024), generator=torch.Generator().manual_seed(12)).to(DEV)
    W[3, 5], W[599, 1000], W[100, 0] = float("nan"), float("inf"), float("-inf")
    bad = torch.full((1,), 77, dtype=torch.int32, device=DEV)
    codes, scales = tb.tb_mx4_quantize(W)
    c2, s2 = torch.zeros_like(codes), torch.zeros_like(scales)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tb.tb_mx4_quantize(W, codes=c2, scales=s2, bad_count=bad)
    idx = torch.from_numpy(R.scale_index(600, 1024).reshape(-1)).to(DEV)
    for n in (3, 3, 2):
        if n == 2:
            W[3, 5] = 0.0  # (a NaN's code is that of 0)
        graph.replay()
        assert bad.item() == n
        assert torch.equal(codes, c2) and torch.equal(scales[idx], s2[idx])


def test_single_rows_of_wider_buffers():
    """One row's stride reaches nothing, whatever it is."""
    W = torch.zeros((1, 163), device=DEV)
    W[:, :160] = torch.randn((1, 160), generator=torch.Generator().manual_seed(13))
    c, s = tb.tb_mx4_quantize(W[:, :160])
    c2, s2 = tb.tb_mx4_quantize(W[:, :160].contiguous())
    assert torch.equal(c, c2)
    idx = torch.from_numpy(R.scale_index(1, 160).reshape(-1)).to(DEV)
    assert torch.equal(s[idx], s2[idx])
    out = torch.full((1, 163), 3.0, device=DEV)
    tb.tb_mx4_dequantize(c, s, 1, 160, W=out[:, :160])
    assert torch.all(out[:, 160:] == 3.0)


def test_tensors_past_four_gigabytes():
    """Values, codes and outputs whose offsets pass 32 bits."""
    N, K, n = 270000, 32768, 200
    g = torch.Generator().manual_seed(14)
    tail = torch.randn((n, K), generator=g).to(torch.bfloat16).to(DEV)
    W = torch.zeros((N, K), dtype=torch.bfloat16, device=DEV)
    W[-n:] = tail
    bad = torch.empty(1, dtype=torch.int32, device=DEV)
    codes, scales = tb.tb_mx4_quantize(W, bad_count=bad)
    small = tb.tb_mx4_quantize(tail)
    assert bad.item() == 0 and codes.numel() > 1 << 32
    assert torch.equal(codes[-n:], small[0]) and not codes[:-n].any()
    back = tb.tb_mx4_dequantize(codes, scales, N, K, W=W)
    assert torch.equal(back[-n:], tb.tb_mx4_dequantize(*small, n, K)) and not back[:-n].any()
    del back, W
    X = torch.randn((3, K), generator=g).to(torch.bfloat16).to(DEV)
    x = tb.tb_mx4_quantize(X)
    Y = tb.tb_mx4_gemm(codes, scales, *x, 3, N, K)
    a, b = (R.values(*R.quantize(t.double().cpu().numpy())[:2]) for t in (X, tail))
    err = np.abs(Y[:, -n:].double().cpu().numpy() - a @ b.T)
    assert np.all(err <= (K / 64 + 12) * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)) and not Y[:, :-n].any()


def test_gemm_outputs_past_four_gigabytes():
    rng = np.random.default_rng(15)
    M, N, K, n = 65536, 65600, 32, 300
    w, ws = R.random_mx4(N, K, rng)
    x, xs = R.random_mx4(M, K, rng)
    Y = tb.tb_mx4_gemm(*R.to_gpu(w, ws), *R.to_gpu(x, xs), M, N, K, out_dtype=torch.bfloat16)
    assert M * N > 1 << 32
    a, b = R.values(x, xs), R.values(w, ws)
    for r in (slice(0, n), slice(M // 2, M // 2 + n), slice(M - n, M)):
        for c in (slice(0, n), slice(N - n, N)):
            ref = a[r] @ b[c].T
            tol = (K / 64 + 12) * 2.0 ** -23 * (np.abs(a[r]) @ np.abs(b[c]).T) + 2.0 ** -8 * np.abs(ref)
            assert np.all(np.abs(Y[r, c].double().cpu().numpy() - ref) <= tol)


@pytest.mark.parametrize("M,N,K", [(5, 5120, 8704), (61, 5120, 8704), (64, 9600, 2272), (40, 19200, 544), (33, 128, 17408)])
def test_gemm_rings_and_splits(M, N, K):
    """Long K: rings that go round several times, in units of an SM each and of two to an SM, whole and split."""
    rng = np.random.default_rng(M + N)
    w, ws = R.random_mx4(N, K, rng)
    x, xs = R.random_mx4(M, K, rng)
    check_gemm(w, ws, x, xs)


def test_chains_without_waits():
    """Calls that begin while the one before still runs: activations quantised into one buffer again and again, each
    batch multiplied and restored before the next overwrites it; eagerly and in a graph, the same bits as one by one."""
    g = torch.Generator().manual_seed(16)
    N, K, n = 2048, 2048, 12
    wc, ws = tb.tb_mx4_quantize(torch.randn((N, K), generator=g).to(DEV))
    for M in (1, 40, 300):
        X = torch.randn((n, M, K), generator=g).to(torch.bfloat16).to(DEV)
        want, back = [], []
        for i in range(n):
            xc, xs = tb.tb_mx4_quantize(X[i])
            want.append(tb.tb_mx4_gemm(wc, ws, xc, xs, M, N, K))
            back.append(tb.tb_mx4_dequantize(xc, xs, M, K))
            torch.cuda.synchronize()
        xc, xs = torch.empty_like(xc), torch.empty_like(xs)
        bad = torch.empty(1, dtype=torch.int32, device=DEV)
        Y, B = torch.empty((n, M, N), device=DEV), torch.empty((n, M, K), dtype=torch.bfloat16, device=DEV)

        def run():
            for i in range(n):
                tb.tb_mx4_quantize(X[i], codes=xc, scales=xs, bad_count=bad)
                tb.tb_mx4_gemm(wc, ws, xc, xs, M, N, K, Y=Y[i])
                tb.tb_mx4_dequantize(xc, xs, M, K, W=B[i])

        def check():
            assert all(torch.equal(Y[i], want[i]) and torch.equal(B[i], back[i]) for i in range(n))

        for _ in range(4):
            Y.fill_(-1), B.fill_(-1)
            run()
            check()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        for _ in range(4):
            Y.fill_(-1), B.fill_(-1)
            graph.replay()
            check()
    assert tb.sync_status() == 0
