"""Plain implementations of the 4-bit format and of the expert layer in 64
bits (numpy), written from the definitions in include/tb.h.  Test support
only; nothing here comes from the library."""
import numpy as np
import torch

VALUES = np.array([0, .5, 1, 1.5, 2, 3, 4, 6] + [-0.0, -.5, -1, -1.5, -2, -3, -4, -6])


def scale_index(N, K):
    """Byte index in the scale tiles of every (row, block), and of the blocks past K: [N][4 ceil(K/128)]."""
    kt = -(-K // 128)
    n, b = np.arange(N)[:, None], np.arange(4 * kt)[None, :]
    return ((n // 128) * kt + b // 4) * 512 + 16 * (n % 32) + 4 * (n % 128 // 32) + b % 4


def quantize(w):
    """w [N][K] float64 (exact copies of the inputs) -> (codes [N][K] 0..15, bytes [N][K/32], bad)."""
    N, K = w.shape
    b = w.reshape(N, K // 32, 32)
    fine = np.isfinite(b)
    amax = np.where(fine, np.abs(b), 0).max(-1)
    floor_log2 = np.frexp(amax)[1] - 1
    e = np.where(amax > 0, np.clip(floor_log2 - 2, -127, 127), -127)
    with np.errstate(invalid="ignore", over="ignore"):
        q = np.abs(b) * np.exp2(-e.astype(np.float64))[..., None]
        q = np.where(np.isnan(q), 0, np.minimum(q, 6.0))
    # nearest value; of two equally near the one with the even code
    d = np.abs(q[..., None] - VALUES[:8])
    near = d == d.min(-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    code = np.where(np.signbit(b) & ~np.isnan(b), code + 8, code)
    return code.reshape(N, K), (e + 127).astype(np.uint8), int((~fine).sum())


def pack(codes):
    c = codes.astype(np.uint8)
    return c[:, 0::2] | (c[:, 1::2] << 4)


def tiles(scale_bytes, N, K):
    out = np.zeros(512 * -(-N // 128) * -(-K // 128), dtype=np.uint8)
    out[scale_index(N, K)[:, : K // 32]] = scale_bytes
    return out


def values(codes, scale_bytes):
    """float64 values of codes [N][K] under bytes [N][K/32]."""
    N, K = codes.shape
    s = np.where(scale_bytes == 255, np.nan, np.exp2(scale_bytes.astype(np.float64) - 127))
    return (VALUES[codes].reshape(N, K // 32, 32) * s[..., None]).reshape(N, K)


def random_mx4(N, K, rng, lo=110, hi=130):
    """Random codes and scale bytes."""
    return rng.integers(0, 16, (N, K)), rng.integers(lo, hi, (N, K // 32)).astype(np.uint8)


def to_gpu(codes, scale_bytes, dev="cuda:0"):
    N, K = codes.shape
    return (torch.from_numpy(pack(codes)).to(dev), torch.from_numpy(tiles(scale_bytes, N, K)).to(dev))


# ---- the expert layer -----------------------------------------------------------------
TERNARY, INT2, INT3, MX4 = 0, 1, 2, 4


def pack_codes(codes, grid):
    """Codewords [N][K] -> the packed bytes of the scalar grids."""
    N, K = codes.shape
    if grid == INT3:
        u = (codes + 4).astype(np.uint32).reshape(N, K // 32, 16, 2)
        m = np.arange(16, dtype=np.uint32)
        planes = [(((u[..., 0] >> p) & 1) << m | ((u[..., 1] >> p) & 1) << (m + 16)).sum(-1, dtype=np.uint32)
                  for p in range(3)]
        return np.stack(planes, -1).reshape(N, -1)
    u = (codes + 2).astype(np.uint32).reshape(N, K // 16, 8, 2)
    m = 2 * np.arange(8, dtype=np.uint32)
    return (u[..., 0] << m | u[..., 1] << (m + 16)).sum(-1, dtype=np.uint32)


def random_matrix(N, K, grid, rng, dev="cuda:0", std=0.02):
    """(float64 weights on `dev`, (packed, scales, grid) for the library)."""
    if grid == MX4:
        c, b = random_mx4(N, K, rng, 118, 123)
        p, s = to_gpu(c, b, dev)
        return torch.from_numpy(values(c, b)).to(dev), (p, s, grid)
    lo, hi = {TERNARY: (-1, 1), INT2: (-2, 1), INT3: (-4, 3)}[grid]
    c = rng.integers(lo, hi + 1, (N, K))
    s = torch.from_numpy(np.abs(rng.standard_normal((N, K // 128))) * std + 1e-3).to(torch.bfloat16).to(dev)
    p = torch.from_numpy(pack_codes(c, grid).view(np.uint8).reshape(-1)).to(dev)
    w = torch.from_numpy(c).to(dev).double() * s.double().repeat_interleave(128, 1)
    return w, (p, s, grid)


def moe(wg, wu, wd, E, x, ids, weights):
    """(y, bound) in float64: wg, wu [E*I][H], wd [E*H][I], x [T][H], ids / weights [T][k]; the bound is that of
    include/tb.h for fp32 outputs."""
    T, H = x.shape
    I, k, u = wd.shape[1], ids.shape[1], 2.0 ** -24
    x, weights = x.double(), weights.double()
    y, tol = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if not 0 <= e < E:
                continue
            G, U, D = wg[e * I:(e + 1) * I], wu[e * I:(e + 1) * I], wd[e * H:(e + 1) * H]
            g, up = G @ x[t], U @ x[t]
            dg, du = ((H / 8 + 16) * u * (m.abs() @ x[t].abs()) for m in (G, U))
            s = g / (1 + torch.exp(-g))
            h = s * up
            dh = 1.1 * dg * (up.abs() + du) + s.abs() * du + 2.0 ** -8 * h.abs()
            y[t] += weights[t, j] * (D @ h)
            tol[t] += weights[t, j].abs() * (D.abs() @ dh + (I / 8 + k + 24) * u * (D.abs() @ (h.abs() + dh)))
    return y, tol


def route(x, router, k, renorm):
    """(ids, weights, all logits) in float64."""
    l = x.double() @ router.double().T
    key = torch.nan_to_num(l, nan=-np.inf, posinf=np.inf, neginf=-np.inf)
    ids = torch.sort(key, dim=-1, descending=True, stable=True)[1][:, :k]
    top = l.gather(1, ids)
    p = torch.exp(top - top[:, :1])
    z = p.sum(-1, keepdim=True) if renorm else torch.exp(l - top[:, :1]).sum(-1, keepdim=True)
    return ids, p / z, l
