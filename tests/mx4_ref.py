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
