"""The router and the expert layer on the GPU against 64-bit
implementations (tests/mx4_ref.py).  Expert ids have to be equal; weights
within (E + 16) 2^-22 of their value (E terms of fp32 sums and an
exponential); layer outputs within the bound of include/tb.h, which the
reference computes from its own 64-bit values."""
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


# ---- router -----------------------------------------------------------------------------
def check_route(x, router, k, renorm, extra=0):
    T, H = x.shape
    E = router.shape[0]
    xb = torch.full((T, H + extra), 5.0, dtype=torch.bfloat16, device=DEV)
    xb[:, :H] = x
    ids, w = tb.tb_moe_route(xb[:, :H], router.to(DEV), k, renormalize=renorm)
    rid, rw, _ = R.route(x.to(DEV), router.to(DEV), k, renorm)
    assert torch.equal(ids.long(), rid), (T, E, H, k)
    # (below 2^-126 fp32 values are 2^-149 apart: the exponential's result and the quotient round there by that much)
    assert torch.all((w.double() - rw).abs() <= (E + 16) * 2.0 ** -22 * rw + 3 * 2.0 ** -149)
    return ids, w


@pytest.mark.parametrize("T,E,H,k", [(1, 1, 8, 1), (1, 128, 2048, 8), (5, 60, 1000, 4), (16, 8, 64, 8), (17, 200, 264, 3),
                                     (32, 512, 512, 16), (33, 16, 4096, 2), (64, 256, 4096, 8), (101, 33, 128, 16),
                                     (3, 130, 56000, 5)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(T, E, H, k, renorm):
    g = torch.Generator().manual_seed(T * 1000 + E)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16)
    r = (torch.randn((E, H), generator=g) / H ** 0.5).to(torch.bfloat16)
    check_route(x, r, k, renorm, extra=8 if T % 2 else 0)


def test_route_ties_take_the_lower_index():
    g = torch.Generator().manual_seed(1)
    x = torch.randn((7, 256), generator=g).to(torch.bfloat16)
    base = torch.randn((5, 256), generator=g).to(torch.bfloat16)
    r = base[torch.tensor([4, 1, 1, 0, 3, 4, 2, 0, 1, 3, 2, 2])]
    check_route(x, r, 9, True)
    ids, w = check_route(x, torch.zeros(300, 256, dtype=torch.bfloat16), 4, True)  # every logit is 0
    assert torch.equal(ids.cpu(), torch.arange(4, dtype=torch.int32).repeat(7, 1)) and torch.all(w == 0.25)
    signs = torch.zeros(4, 256, dtype=torch.bfloat16)
    signs[0], signs[2] = -0.0, -0.0  # zeros of both signs are equal
    ids, _ = check_route(x.abs(), signs, 4, False)
    assert torch.equal(ids.cpu(), torch.arange(4, dtype=torch.int32).repeat(7, 1))


def test_route_order_beyond_fp32():
    """Logits that agree in fp32 and differ in their 30th bit; subnormal weights decide among equals."""
    H = 64
    r = torch.zeros(6, H)
    r[:, 0] = 1024.0
    for e, v in enumerate((0.0, 1.0, -1.0, 3.0, 2.0, 0.5)):
        r[e, 1] = v * 2.0 ** -20
    r = r.to(torch.bfloat16)
    x = torch.zeros(2, H)
    x[:, 0], x[:, 1] = 1.0, 1.0
    ids, _ = check_route(x.to(torch.bfloat16), r, 6, True)
    assert ids[0].tolist() == [3, 4, 1, 5, 0, 2]
    tiny = torch.zeros(4, H)
    for e, v in enumerate((1, 3, 0, 2)):
        tiny[e, 5] = v * 2.0 ** -133
    x2 = torch.full((1, H), 2.0)
    ids, _ = check_route(x2.to(torch.bfloat16), tiny.to(torch.bfloat16), 4, False)
    assert ids[0].tolist() == [1, 3, 0, 2]


def test_route_non_finite_token_stays_in_its_row():
    g = torch.Generator().manual_seed(3)
    x = torch.randn((6, 128), generator=g).to(torch.bfloat16)
    r = torch.randn((20, 128), generator=g).to(torch.bfloat16)
    want, ww = tb.tb_moe_route(x.to(DEV), r.to(DEV), 4)
    x[2, 7] = float("nan")
    ids, w = tb.tb_moe_route(x.to(DEV), r.to(DEV), 4)
    keep = torch.tensor([0, 1, 3, 4, 5], device=DEV)
    assert torch.equal(ids[keep], want[keep]) and torch.equal(w[keep], ww[keep])
    assert ids[2].tolist() == [0, 1, 2, 3] and torch.isnan(w[2]).all()


# ---- experts ------------------------------------------------------------------------------
def make_layer(E, H, I, grids, seed):
    rng = np.random.default_rng(seed)
    wg, g = R.random_matrix(E * I, H, grids[0], rng)
    wu, u = R.random_matrix(E * I, H, grids[1], rng)
    wd, d = R.random_matrix(E * H, I, grids[2], rng)
    return (wg, wu, wd), tb.moe_layer(g, u, d, E, H, I)


def check_moe(mats, layer, x, ids, weights, dt=torch.float32, extra=0, ws=None):
    T, H = x.shape
    E = layer.desc.E
    xb = torch.full((T, H + 8 * extra), 5.0, dtype=torch.bfloat16, device=DEV)
    xb[:, :H] = x
    y = torch.full((T, H + extra), 7.0, dtype=dt, device=DEV)
    tb.tb_moe(layer, xb[:, :H], ids.to(DEV), weights.to(DEV), y=y[:, :H], ws=ws)
    torch.cuda.synchronize()
    assert torch.all(y[:, H:] == 7.0)
    ref, tol = R.moe(*mats, E, x.to(DEV), ids, weights.to(DEV))
    if dt == torch.bfloat16:
        tol = tol + 2.0 ** -8 * ref.abs()
    err = (y[:, :H].double() - ref).abs()
    assert torch.all(err <= tol), (T, E, (err / tol.clamp(min=1e-300)).max().item())
    return y


def draw_ids(T, k, E, g):
    return torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)


GRIDS = [(0, 0, 0), (2, 2, 2), (4, 4, 4), (1, 2, 4), (4, 0, 2), (2, 4, 1)]


@pytest.mark.parametrize("grids", GRIDS)
@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 256, 128), (1, 4, 4, 128, 640), (3, 16, 8, 384, 256), (13, 5, 3, 512, 384),
                                       (64, 6, 2, 128, 128)])
def test_moe(T, E, k, H, I, grids):
    g = torch.Generator().manual_seed(T + E)
    mats, layer = make_layer(E, H, I, grids, T * 100 + E)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16)
    ids = draw_ids(T, k, E, g)
    w = torch.rand((T, k), generator=g)
    check_moe(mats, layer, x, ids, w, torch.bfloat16 if T == 3 else torch.float32, extra=T % 2)


@pytest.mark.parametrize("T", [1, 4, 5, 8, 9, 16, 17, 63, 64])
def test_moe_one_expert_takes_every_token(T):
    """Blocks of up to four, of up to eight and several blocks of one expert."""
    g = torch.Generator().manual_seed(T)
    mats, layer = make_layer(1, 256, 256, (0, 4, 2), 7)
    x = torch.randn((T, 256), generator=g).to(torch.bfloat16)
    check_moe(mats, layer, x, torch.zeros(T, 1, dtype=torch.int32), torch.randn((T, 1), generator=g))


def test_moe_empty_and_odd_ids():
    """Tokens without experts give 0; ids outside the range are skipped; a repeated id counts every time."""
    g = torch.Generator().manual_seed(4)
    mats, layer = make_layer(6, 256, 128, (1, 1, 1), 8)
    x = torch.randn((7, 256), generator=g).to(torch.bfloat16)
    ids = draw_ids(7, 4, 6, g)
    ids[0] = -1
    ids[1] = torch.tensor([6, 2 ** 31 - 1, -(2 ** 31), 512])
    ids[2] = torch.tensor([3, 3, 3, 3])
    ids[3] = torch.tensor([2, -1, 2, 5])
    ids[6, 1:] = -1
    w = torch.rand((7, 4), generator=g)
    y = check_moe(mats, layer, x, ids, w)
    assert torch.all(y[:2] == 0)
    y = check_moe(mats, layer, x, torch.full_like(ids, -1), w, torch.bfloat16)
    assert torch.all(y == 0)


def test_moe_many_experts_and_the_largest_batch():
    g = torch.Generator().manual_seed(5)
    mats, layer = make_layer(512, 128, 128, (0, 1, 4), 9)
    x = torch.randn((64, 128), generator=g).to(torch.bfloat16)
    check_moe(mats, layer, x, draw_ids(64, 16, 512, g), torch.rand((64, 16), generator=g))


@pytest.mark.parametrize("grids", [(0, 2, 4), (4, 4, 2)])
def test_moe_decode_sizes(grids):
    """Long rows (K split between the warps of a CTA at one token, and not at many)."""
    g = torch.Generator().manual_seed(6)
    mats, layer = make_layer(8, 2048, 1408, grids, 10)
    for T, k in ((1, 2), (2, 8), (24, 4)):
        x = torch.randn((T, 2048), generator=g).to(torch.bfloat16)
        check_moe(mats, layer, x, draw_ids(T, k, 8, g), torch.rand((T, k), generator=g))


def test_moe_outlier_activations():
    g = torch.Generator().manual_seed(7)
    mats, layer = make_layer(4, 256, 128, (2, 2, 2), 11)
    x = torch.randn((3, 256), generator=g)
    x[:, 17], x[1, 90] = 2.0 ** 12, -2.0 ** 14
    check_moe(mats, layer, x.to(torch.bfloat16), draw_ids(3, 2, 4, g), torch.rand((3, 2), generator=g))


def test_moe_repeats_bitwise_shares_a_workspace_and_replays():
    """Same bits from call to call, on another stream and in a graph; a workspace shared with a dense product keeps
    that product's control words zero."""
    g = torch.Generator().manual_seed(8)
    mats, layer = make_layer(16, 512, 256, (0, 1, 2), 12)
    x = torch.randn((9, 512), generator=g).to(torch.bfloat16).to(DEV)
    ids, w = draw_ids(9, 4, 16, g).to(DEV), torch.rand((9, 4), generator=g).to(DEV)
    wd, dense = R.random_matrix(8192, 4096, R.INT2, np.random.default_rng(13))
    xd = torch.randn(4096, generator=g).to(torch.bfloat16).to(DEV)
    ws = tb.workspace(max(tb.moe_workspace_bytes(layer, 9, 4), tb.workspace_bytes(1, 8192, 4096)), DEV)
    y0 = tb.tb_gemv(dense[0], dense[2], dense[1], xd, 8192, 4096, ws=ws)
    first = tb.tb_moe(layer, x, ids, w, ws=ws)
    for _ in range(3):
        assert torch.equal(first, tb.tb_moe(layer, x, ids, w, ws=ws))
        assert torch.equal(y0, tb.tb_gemv(dense[0], dense[2], dense[1], xd, 8192, 4096, ws=ws))
    assert tb.sync_status() == 0
    y = torch.zeros_like(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tb.tb_moe(layer, x, ids, w, y=y, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tb.tb_moe(layer, x, ids, w, y=y, ws=ws)
    other = ids.clone()
    y.zero_()
    graph.replay()
    assert torch.equal(first, y)
    ids[0] = -1  # a replay reads the ids of its own time
    graph.replay()
    assert torch.all(y[0] == 0) and torch.equal(first[1:], y[1:])
    ids.copy_(other)
    graph.replay()
    assert torch.equal(first, y)


def test_moe_batch_rows_are_independent():
    """A token's result does not depend on its neighbours beyond rounding; with the same grouping it is the same."""
    g = torch.Generator().manual_seed(9)
    mats, layer = make_layer(8, 256, 256, (0, 2, 4), 14)
    x = torch.randn((6, 256), generator=g).to(torch.bfloat16)
    ids, w = draw_ids(6, 3, 8, g), torch.rand((6, 3), generator=g)
    x2 = x.clone()
    x2[3] = float("nan")
    y = check_moe(mats, layer, x, ids, w)
    y2 = tb.tb_moe(layer, x2.to(DEV), ids.to(DEV), w.to(DEV))
    keep = torch.tensor([0, 1, 2, 4, 5], device=DEV)
    assert torch.equal(y[keep, :256], y2[keep]) and torch.isnan(y2[3]).all()


def test_moe_long_rows():
    """Rows of more 128-groups than their scales are copied whole for."""
    g = torch.Generator().manual_seed(16)
    for grids, H, I in (((0, 2, 1), 128 * 67, 128), ((2, 4, 2), 256, 128 * 65), ((1, 0, 4), 128 * 65, 128 * 3)):
        mats, layer = make_layer(2, H, I, grids, H + I)
        x = torch.randn((3, H), generator=g).to(torch.bfloat16)
        check_moe(mats, layer, x, draw_ids(3, 2, 2, g), torch.rand((3, 2), generator=g))


def test_moe_waits_that_give_up_are_reported():
    """The copies are never issued: every wait gives up after about 10 ms, the outputs of tokens with experts are NaN,
    the status says so, and the next call is correct."""
    g = torch.Generator().manual_seed(17)
    for grids, T in (((0, 2, 4), 1), ((4, 1, 2), 20)):
        mats, layer = make_layer(4, 256, 256, grids, 18)
        x = torch.randn((T, 256), generator=g).to(torch.bfloat16)
        ids, w = draw_ids(T, 2, 4, g), torch.rand((T, 2), generator=g) + 0.1
        y = tb.tb_moe(layer, x.to(DEV), ids.to(DEV), w.to(DEV), flags=tb.FLAG_TEST_STALL)
        assert tb.sync_status() == 6 and torch.isnan(y).all()
        check_moe(mats, layer, x, ids, w)
        assert tb.sync_status() == 0


def test_moe_large_scales():
    """4-bit scales across their range: below 2^1 (one factor), above it (two), 255 (no number, in its row only)."""
    rng = np.random.default_rng(19)
    H = I = 128
    wg, g = R.random_matrix(2 * I, H, R.INT2, rng)
    wu, u = R.random_matrix(2 * I, H, R.INT2, rng)
    c, b = R.random_mx4(2 * H, I, rng)
    b[:, 0], b[5, 1], b[6, 2], b[7, 3] = 127, 129, 200, 240
    b[130, 1], b[131, 1], b[132, 1] = 128, 1, 0
    p, s = R.to_gpu(c, b)
    layer = tb.moe_layer(g, u, (p, s, R.MX4), 2, H, I)
    gen = torch.Generator().manual_seed(19)
    x = torch.randn((2, H), generator=gen).to(torch.bfloat16)
    ids, w = torch.tensor([[0, 1], [1, -1]], dtype=torch.int32), torch.rand((2, 2), generator=gen)
    check_moe((wg, wu, torch.from_numpy(R.values(c, b)).to(DEV)), layer, x, ids, w)
    b[9, 2] = 255
    p, s = R.to_gpu(c, b)
    layer = tb.moe_layer(g, u, (p, s, R.MX4), 2, H, I)
    y = tb.tb_moe(layer, x.to(DEV), ids.to(DEV), w.to(DEV))
    want = torch.zeros(2, H, dtype=torch.bool)
    want[0, 9] = True
    assert torch.equal(torch.isnan(y).cpu(), want)


def test_routed_layer_run():
    """The operators as a decoder uses them: weights quantised and packed by the library (scalar grid for gate and up,
    4-bit floats for down), tokens routed, experts applied -- in one stream, captured and replayed."""
    E, H, I, T, k = 12, 512, 384, 10, 3
    g = torch.Generator().manual_seed(15)
    wg, wu = (torch.randn((E * I, H), generator=g).mul_(0.05).to(torch.bfloat16).to(DEV) for _ in range(2))
    wd = torch.randn((E * H, I), generator=g).mul_(0.05).to(torch.bfloat16).to(DEV)
    sg, su = tb.tb_scales_absmax(wg, tb.INT3), tb.tb_scales_absmax(wu, tb.INT2)
    pg, pu = tb.tb_pack(wg, tb.INT3, sg), tb.tb_pack(wu, tb.INT2, su)
    cd, td = tb.tb_mx4_quantize(wd)
    layer = tb.moe_layer((pg, sg, tb.INT3), (pu, su, tb.INT2), (cd, td, tb.MX4), E, H, I)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16).to(DEV)
    r = torch.randn((E, H), generator=g).mul_(H ** -0.5).to(torch.bfloat16).to(DEV)
    ws = tb.workspace(tb.moe_workspace_bytes(layer, T, k), DEV)
    ids, w = torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty((T, k), device=DEV)
    y = torch.empty((T, H), device=DEV)

    def step():
        tb.tb_moe_route(x, r, k, ids=ids, weights=w)
        tb.tb_moe(layer, x, ids, w, y=y, ws=ws)
    step()
    first = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        graph.replay()
    assert torch.equal(first, y) and tb.sync_status() == 0
    G = tb.tb_unpack(pg, tb.INT3, E * I, H).double() * sg.double().repeat_interleave(128, 1)
    U = tb.tb_unpack(pu, tb.INT2, E * I, H).double() * su.double().repeat_interleave(128, 1)
    D = tb.tb_mx4_dequantize(cd, td, E * H, I, out_dtype=torch.float32).double()
    rid, rw, _ = R.route(x, r, k, True)
    assert torch.equal(ids.long(), rid)
    ref, tol = R.moe(G, U, D, E, x, ids, w)
    assert torch.all((y.double() - ref).abs() <= tol)


# ---- calls beside one another, padded batches --------------------------------------------
def test_moe_layers_in_a_row_hand_over_their_activations():
    """Layers that read what the layer before wrote, through two buffers in turn and without a wait between them: the
    same bits as one by one with fresh buffers, eagerly and in a graph."""
    g = torch.Generator().manual_seed(21)
    T, E, k, H, I, depth = 3, 8, 2, 512, 128, 12
    mats, layer = make_layer(E, H, I, (2, 1, 4), 22)
    x0 = torch.randn((T, H), generator=g).to(torch.bfloat16).to(DEV)
    ids = [draw_ids(T, k, E, g).to(DEV) for _ in range(depth)]
    w = torch.rand((T, k), generator=g).to(DEV)
    # weights that keep the activations near one from layer to layer
    scale, want = [], x0
    for i in range(depth):
        f = 1.0 / tb.tb_moe(layer, want, ids[i], w).abs().mean().item()
        scale.append((w * f).contiguous())
        want = tb.tb_moe(layer, want, ids[i], scale[i], out_dtype=torch.bfloat16)
        torch.cuda.synchronize()
    assert torch.isfinite(want).all() and want.abs().max() > 0
    ws = tb.workspace(tb.moe_workspace_bytes(layer, T, k), DEV)
    buf = [x0.clone(), torch.empty_like(x0)]

    def run():
        for i in range(depth):
            tb.tb_moe(layer, buf[i & 1], ids[i], scale[i], y=buf[~i & 1], ws=ws)

    for _ in range(5):
        buf[0].copy_(x0)
        run()
        assert torch.equal(buf[depth & 1], want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(5):
        buf[0].copy_(x0)
        graph.replay()
        assert torch.equal(buf[depth & 1], want)
    assert tb.sync_status() == 0


def test_calls_at_once_on_two_streams():
    """Two streams, each with its own workspace, route and apply experts at the same time."""
    g = torch.Generator().manual_seed(23)
    T, E, k, H, I = 24, 16, 4, 512, 256
    mats, layer = make_layer(E, H, I, (0, 2, 4), 24)
    r = torch.randn((E, H), generator=g).to(torch.bfloat16).to(DEV)
    xs = [torch.randn((T, H), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2)]
    want = []
    for x in xs:
        ids, w = tb.tb_moe_route(x, r, k)
        want.append(tb.tb_moe(layer, x, ids, w))
    ws = [tb.workspace(tb.moe_workspace_bytes(layer, T, k), DEV) for _ in range(2)]
    ids = [torch.empty((T, k), dtype=torch.int32, device=DEV) for _ in range(2)]
    w = [torch.empty((T, k), device=DEV) for _ in range(2)]
    ys = [[torch.zeros((T, H), device=DEV) for _ in range(10)] for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(10):
        for s in range(2):
            with torch.cuda.stream(streams[s]):
                tb.tb_moe_route(xs[s], r, k, ids=ids[s], weights=w[s])
                tb.tb_moe(layer, xs[s], ids[s], w[s], y=ys[s][i], ws=ws[s])
    torch.cuda.synchronize()
    for s in range(2):
        for y in ys[s]:
            assert torch.equal(y, want[s])
    assert tb.sync_status() == 0


def test_moe_padded_batch():
    """Padding rows (no expert; activations and weights that are no numbers) give 0 and change nothing."""
    g = torch.Generator().manual_seed(25)
    mats, layer = make_layer(6, 256, 128, (2, 0, 4), 26)
    x = torch.randn((11, 256), generator=g).to(torch.bfloat16)
    ids, w = draw_ids(11, 3, 6, g), torch.rand((11, 3), generator=g)
    want = check_moe(mats, layer, x, ids, w)[:, :256]
    xp = torch.full((64, 256), float("nan"), dtype=torch.bfloat16)
    ip, wp = torch.full((64, 3), -1, dtype=torch.int32), torch.full((64, 3), float("nan"))
    xp[:11], ip[:11], wp[:11] = x, ids, w
    y = tb.tb_moe(layer, xp.to(DEV), ip.to(DEV), wp.to(DEV))
    ref, tol = R.moe(*mats, 6, x.to(DEV), ids, w.to(DEV))  # (another grouping may be taken: within the bound)
    assert torch.all((y[:11].double() - ref).abs() <= tol) and torch.all(y[11:] == 0)
    assert torch.all((want.double() - ref).abs() <= tol)


def test_single_rows_of_wider_buffers():
    """One row's stride reaches nothing, whatever it is."""
    g = torch.Generator().manual_seed(27)
    mats, layer = make_layer(4, 256, 128, (2, 2, 4), 28)
    wide = torch.zeros((1, 259), dtype=torch.bfloat16, device=DEV)
    wide[:, :256] = torch.randn((1, 256), generator=g)
    x, r = wide[:, :256], torch.randn((4, 256), generator=g).to(torch.bfloat16).to(DEV)
    ids, w = tb.tb_moe_route(x, r, 2)
    ids2, w2 = tb.tb_moe_route(x.contiguous(), r, 2)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    assert torch.equal(tb.tb_moe(layer, x, ids, w), tb.tb_moe(layer, x.contiguous(), ids, w))


def test_route_long_batch():
    """More clusters than the GPU holds at once, the last of them not full."""
    g = torch.Generator().manual_seed(29)
    x = torch.randn((1501, 96), generator=g).to(torch.bfloat16)
    check_route(x, torch.randn((33, 96), generator=g).to(torch.bfloat16), 5, True)


def test_moe_experts_past_four_gigabytes():
    """The last of so many experts that its codes begin past 2^32 bytes."""
    E, H, I = 172, 8192, 8192
    rng = np.random.default_rng(30)
    mats, parts = [], []
    for rows, cols, grid in ((I, H, R.MX4), (I, H, R.INT3), (H, I, R.MX4)):
        m, (packed, scales, _) = R.random_matrix(rows, cols, grid, rng)
        packed, scales = packed.reshape(-1), scales.reshape(-1)
        assert (E - 1) * packed.numel() * packed.element_size() > 1 << 32
        P = torch.zeros(E * packed.numel(), dtype=packed.dtype, device=DEV)
        S = torch.zeros(E * scales.numel(), dtype=scales.dtype, device=DEV)
        P[-packed.numel():], S[-scales.numel():] = packed, scales
        mats.append(m)
        parts.append((P, S, grid))
    layer = tb.moe_layer(*parts, E, H, I)
    g = torch.Generator().manual_seed(31)
    x = torch.randn((2, H), generator=g).to(torch.bfloat16).to(DEV)
    w = torch.rand((2, 2), generator=g).to(DEV)
    y = tb.tb_moe(layer, x, torch.tensor([[E - 1, -1], [0, E - 1]], dtype=torch.int32, device=DEV), w)
    # every other expert is 0: the rest of the layer does not count
    ref, tol = R.moe(*mats, 1, x, torch.tensor([[0, -1], [-1, 0]], dtype=torch.int32), w)
    assert torch.all((y.double() - ref).abs() <= tol) and ref.abs().max() > 0


def test_experts_requantised_between_calls():
    """Layers whose 4-bit experts are quantised into the same buffers right before each call, and whose router reads
    what the layer before wrote: nothing is read before it is final."""
    g = torch.Generator().manual_seed(32)
    T, E, k, H, I, depth = 5, 6, 2, 256, 128, 6
    W = [[torch.randn((E * r, c), generator=g).mul_(0.1).to(torch.bfloat16).to(DEV) for r, c in ((I, H), (I, H), (H, I))]
         for _ in range(depth)]
    R_ = torch.randn((depth, E, H), generator=g).to(torch.bfloat16).to(DEV)
    x0 = torch.randn((T, H), generator=g).to(torch.bfloat16).to(DEV)
    x = x0
    for i in range(depth):  # one by one
        layer = tb.moe_layer(*((*tb.tb_mx4_quantize(w), tb.MX4) for w in W[i]), E, H, I)
        x = tb.tb_moe(layer, x, *tb.tb_moe_route(x, R_[i], k), out_dtype=torch.bfloat16)
        torch.cuda.synchronize()
    assert torch.isfinite(x).all() and x.abs().max() > 0
    codes = [tb.tb_mx4_quantize(w) for w in W[0]]
    layer = tb.moe_layer(*((*c, tb.MX4) for c in codes), E, H, I)
    ws = tb.workspace(tb.moe_workspace_bytes(layer, T, k), DEV)
    ids, wt = torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty((T, k), device=DEV)
    buf = [x0.clone(), torch.empty_like(x0)]

    def run():
        for i in range(depth):
            for w, (c, s) in zip(W[i], codes):
                tb.tb_mx4_quantize(w, codes=c, scales=s)
            tb.tb_moe_route(buf[i & 1], R_[i], k, ids=ids, weights=wt)
            tb.tb_moe(layer, buf[i & 1], ids, wt, y=buf[~i & 1], ws=ws)

    for _ in range(4):
        buf[0].copy_(x0)
        run()
        assert torch.equal(buf[depth & 1], x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(4):
        buf[0].copy_(x0)
        graph.replay()
        assert torch.equal(buf[depth & 1], x)


def test_calls_on_a_given_stream_allocate_there():
    """A stream's address instead of the current stream: outputs and workspace that the call allocates are that stream's,
    while the current one is busy with memory it has just freed."""
    g = torch.Generator().manual_seed(33)
    T, E, k, H, I = 6, 8, 2, 512, 256
    mats, layer = make_layer(E, H, I, (2, 0, 4), 34)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16).to(DEV)
    r = torch.randn((E, H), generator=g).to(torch.bfloat16).to(DEV)
    want = tb.tb_moe(layer, x, *tb.tb_moe_route(x, r, k))
    wc, ws = tb.tb_mx4_quantize(x)
    wy, wv = tb.tb_mx4_gemm(wc, ws, wc, ws, T, T, H), tb.tb_mx4_dequantize(wc, ws, T, H)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    n = tb.moe_workspace_bytes(layer, T, k)
    for _ in range(5):
        busy = torch.empty(1 << 26, device=DEV)
        for _ in range(4):
            busy.fill_(1.0)  # the current stream is behind ...
        for size in (n, T * H * 4, T * k * 4, 512 * 4, T * H // 2):
            torch.empty(size, dtype=torch.uint8, device=DEV).fill_(255)  # ... with blocks that are free to allocate
        s = side.cuda_stream
        ids, w = tb.tb_moe_route(x, r, k, stream=s)
        y = tb.tb_moe(layer, x, ids, w, stream=s)
        c, t = tb.tb_mx4_quantize(x, stream=s)
        Y, v = tb.tb_mx4_gemm(c, t, c, t, T, T, H, stream=s), tb.tb_mx4_dequantize(c, t, T, H, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(Y, wy) and torch.equal(v, wv) and torch.equal(c, wc)


@pytest.mark.parametrize("T,E,H,k", [(16, 256, 4096, 8), (32, 64, 2048, 4), (40, 512, 4096, 8), (63, 256, 4096, 8),
                                     (130, 40, 1032, 3), (9, 300, 2056, 16)])
def test_route_batches(T, E, H, k):
    """One, two and four tokens to a cluster of four or eight, the last cluster full or not."""
    g = torch.Generator().manual_seed(T * E)
    check_route(torch.randn((T, H), generator=g).to(torch.bfloat16), torch.randn((E, H), generator=g).to(torch.bfloat16), k,
                T % 2 == 0, extra=8)
