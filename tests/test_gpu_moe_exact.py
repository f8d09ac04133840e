"""Expert layers whose results are exact, so that one lost, doubled or
misplaced value shows, and every kernel of the layer at both numbers of
column sets.

Rows of gate give g in [20, 30], a multiple of 1/2; rows of up give u in
{0, +-1/2, +-1, +-2}; a token's activations are one vector of +-1 times 2^p,
p in {0, 1, 2}.  Then silu(g) u differs from g u by less than e^-20 + 2^-20 of
it, and g u 4^p has at most six significant bits: its rounding to bf16 is g u 4^p
itself.  down's weights are multiples of 1/4, the routing weights powers of
two, and every partial sum is a multiple of a power of two that fits 24
bits (checked on the sums of absolute values): y has no rounding at all."""
import numpy as np
import pytest
import torch

from decode_gemv_tb_b200 import tb
from tests import mx4_ref as R

GRIDS = [(g, u) for g in (R.INT2, R.INT3, R.MX4) for u in (R.INT2, R.INT3, R.MX4)]
VALUES = {R.TERNARY: [-1, 0, 1], R.INT2: [-2, -1, 0, 1], R.INT3: [-4, -3, -2, -1, 0, 1, 2, 3],
          R.MX4: [-3, -2, -1.5, -1, -.5, 0, .5, 1, 1.5, 2, 3]}


def exact_rows(rows, K, grid, x, targets, rng):
    """(values c [rows][K], scale exponents [rows][K / block]): a random matrix with (c 2^e) x = targets.  Its values are
    moved, in random order, until the row's sum is right; the first block has the finest scale."""
    block = 32 if grid == R.MX4 else 128
    vals = np.array(VALUES[grid])
    c = rng.choice(vals, (rows, K)).astype(np.float64)
    e = rng.integers(-1, 2, (rows, K // block))
    e[:, 0] = -1
    unit = np.exp2(e).repeat(block, 1)
    order, r = rng.permuted(np.tile(np.arange(K), (rows, 1)), axis=1), np.arange(rows)
    left = targets - (c * unit) @ x
    for i in range(3 * K):
        k = order[:, i % K]
        f = x[k] * unit[r, k]  # what one more in c adds to the sum
        room = (vals[None, :] - c[r, k][:, None]) * f[:, None]
        move = np.where((room * left[:, None] > 0) & (np.abs(room) <= np.abs(left)[:, None]), room, 0)
        move = move[r, np.abs(move).argmax(1)]
        c[r, k] += move / f
        left -= move
    assert np.all(left == 0) and np.all(np.isin(c, vals))
    return c, e


def pack_rows(c, e, grid, dev):
    N, K = c.shape
    if grid == R.MX4:
        codes = np.searchsorted(R.VALUES[:8], np.abs(c))
        codes = codes + 8 * (c < 0)
        return (*R.to_gpu(codes, (e + 127).astype(np.uint8), dev), grid)
    s = torch.from_numpy(np.exp2(e.astype(np.float64))).to(torch.bfloat16).to(dev)
    return torch.from_numpy(R.pack_codes(c.astype(np.int64), grid).view(np.uint8).reshape(-1)).to(dev), s, grid


def exact_layer(E, H, I, grids, seed, dev):
    """(layer parts, x0, g [E*I], u [E*I], down [E*H][I] in float64)"""
    rng = np.random.default_rng(seed)
    x0 = rng.choice([-1.0, 1.0], H)
    g = rng.integers(40, 61, E * I) / 2
    u = rng.choice([0, .5, -.5, 1, -1, 2, -2], E * I)
    gc, ge = exact_rows(E * I, H, grids[0], x0, g, rng)
    uc, ue = exact_rows(E * I, H, grids[1], x0, u, rng)
    dc = rng.choice(np.array(VALUES[grids[2]]), (E * H, I))
    de = rng.integers(-1, 2, (E * H, I // (32 if grids[2] == R.MX4 else 128)))
    d = dc * np.exp2(de).repeat(I // de.shape[1], 1)
    return [pack_rows(c, e, q, dev) for c, e, q in ((gc, ge, grids[0]), (uc, ue, grids[1]), (dc, de, grids[2]))], x0, g, u, d


def batch(T, k, E, x0, rng):
    """x [T][H], p [T], ids [T][k], weights [T][k]: -1 among the ids, weights of powers of two"""
    p = rng.integers(0, 3, T)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    ids[rng.random((T, k)) < .1] = -1
    return x0[None, :] * np.exp2(p)[:, None], p, ids, np.exp2(rng.integers(-2, 1, (T, k)))


def expected(E, I, H, p, ids, w, g, u, d):
    T, k = ids.shape
    y, size = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if e >= 0:
                h = (g * u)[e * I:(e + 1) * I] * 4.0 ** p[t]
                D = d[e * H:(e + 1) * H]
                y[t] += w[t, j] * (D @ h)
                size[t] += w[t, j] * (np.abs(D) @ np.abs(h))
    # multiples of 1/4 (g u) 4^p times 1/4 (down) times 1/4 (weights)
    assert np.all(size * 64 / 4.0 ** p[:, None] < 2 ** 24)
    return y


def check(E, H, I, T, k, grids, seed, dev):
    parts, x0, g, u, d = exact_layer(E, H, I, grids, seed, dev)
    x, p, ids, w = batch(T, k, E, x0, np.random.default_rng(seed + 1))
    want = expected(E, I, H, p, ids, w, g, u, d)
    layer = tb.moe_layer(*parts, E, H, I)
    y = tb.tb_moe(layer, torch.from_numpy(x).to(torch.bfloat16).to(dev), torch.from_numpy(ids).to(torch.int32).to(dev),
                  torch.from_numpy(w).float().to(dev))
    got = y.double().cpu().numpy()
    assert np.array_equal(got, want), (np.abs(got - want).max(), np.argwhere(got != want)[:5].tolist())


def test_the_construction_on_the_host():
    """The rows' sums, the exactness of h, and that one lost column of any matrix changes nearly every result."""
    for grid in (R.TERNARY, R.INT2, R.INT3, R.MX4):
        rng = np.random.default_rng(grid)
        x0, t = rng.choice([-1.0, 1.0], 384), rng.integers(40, 61, 64) / 2
        c, e = exact_rows(64, 384, grid, x0, t, rng)
        w = c * np.exp2(e).repeat(384 // e.shape[1], 1)
        assert np.array_equal(w @ x0, t)
        assert np.mean(w[:, 5] != 0) > .5 and np.mean(w[:, 380] != 0) > .5
    for g in np.arange(20, 30.5, .5):
        for u in (.5, 1.0, -2.0):
            for p in range(3):
                v = g * 2.0 ** p
                silu = v / (1 + np.exp(-v))
                for err in (1 - 2.0 ** -20, 1.0, 1 + 2.0 ** -20):
                    assert torch.tensor(silu * u * 2.0 ** p * err).to(torch.bfloat16).item() == g * u * 4.0 ** p


@pytest.fixture
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tb.load()
    return "cuda:0"


@pytest.mark.gpu
@pytest.mark.parametrize("gate,up", GRIDS)
@pytest.mark.parametrize("T,E,k", [(1, 8, 4), (20, 6, 3), (64, 4, 3)])
def test_exact(dev, gate, up, T, E, k):
    """One token; one set of columns in several blocks; two sets.  Every pair of formats of gate and up, each of them
    with a format of down in turn; odd numbers of 128-groups."""
    down = (R.INT2, R.INT3, R.MX4)[(GRIDS.index((gate, up)) + T) % 3]
    assert (T * k > 10 * E) == (T == 64)
    check(E, 384, 128, T, k, (gate, up, down), 7 * T + gate, dev)


@pytest.mark.gpu
@pytest.mark.parametrize("down", [R.TERNARY, R.INT2, R.INT3, R.MX4])
@pytest.mark.parametrize("T,E,k", [(2, 3, 2), (40, 3, 2)])
def test_exact_down(dev, down, T, E, k):
    """The second product alone at odd sizes: rows of 384, split in slices where there are few pairs."""
    check(E, 640, 384, T, k, (R.INT3, R.TERNARY, down), down + T, dev)


@pytest.mark.gpu
@pytest.mark.parametrize("gate,up", GRIDS)
@pytest.mark.parametrize("T", [10, 11])
def test_both_sides_of_the_second_column_set(dev, gate, up, T):
    """Ten pairs per expert, then more: one set of columns, then two, on random layers against the bound."""
    E, k, H, I = 2, 2, 512, 256
    rng = np.random.default_rng(gate * 8 + up)
    down = (R.MX4, R.INT2, R.INT3)[(gate + up + T) % 3]
    (wg, a), (wu, b), (wd, c) = (R.random_matrix(n, m, q, rng, dev) for n, m, q in
                                 ((E * I, H, gate), (E * I, H, up), (E * H, I, down)))
    layer = tb.moe_layer(a, b, c, E, H, I)
    gen = torch.Generator().manual_seed(T)
    x = torch.randn((T, H), generator=gen).to(torch.bfloat16).to(dev)
    ids = torch.stack([torch.randperm(E, generator=gen)[:k] for _ in range(T)]).to(torch.int32)
    w = torch.rand((T, k), generator=gen).to(dev)
    y = tb.tb_moe(layer, x, ids.to(dev), w)
    ref, tol = R.moe(wg, wu, wd, E, x, ids, w)
    assert torch.all((y.double() - ref).abs() <= tol)
