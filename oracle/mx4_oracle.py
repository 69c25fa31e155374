"""4-bit codes in plain NumPy, fp64: the definition of include/fgmm.h (OCP Microscaling Formats
v1.0, MXFP4), one block at a time.  Test infrastructure only."""
import numpy as np

BLOCK = 32
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def encode(x):
    """Codes [N, blocks * 32] (one per byte) and scale bytes [N, blocks] of x [N, D]."""
    x = np.asarray(x, dtype=np.float64)
    n, d = x.shape
    nb = -(-d // BLOCK)
    p = np.zeros((n, nb * BLOCK))
    p[:, :d] = x
    p = p.reshape(n, nb, BLOCK)
    bad = ~np.isfinite(p).all(2)
    p = np.where(bad[..., None], 0.0, p)
    top = np.abs(p).max(2)
    e = np.where(top > 0, np.frexp(top)[1] - 3, -127)      # floor(log2 top) - 2
    e = np.clip(e, -127, 127)
    a = np.abs(p) / np.ldexp(1.0, e)[..., None]
    dist = np.abs(a[..., None] - GRID)
    near = dist == dist.min(-1, keepdims=True)             # two of them on a tie
    first = near.argmax(-1)
    second = 7 - near[..., ::-1].argmax(-1)
    c = np.where(first % 2 == 0, first, second)            # ties: the even code
    c = c | np.where(np.signbit(p), 8, 0)
    s = np.where(bad, 255, e + 127)
    return np.where(bad[..., None], 0, c).reshape(n, nb * BLOCK).astype(np.uint8), s.astype(np.uint8)


def decode(codes, scales, d):
    n, nb = scales.shape
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    c = codes.reshape(n, nb, BLOCK)
    v = np.where(c & 8, -1.0, 1.0) * GRID[c & 7] * s[..., None]
    return v.reshape(n, nb * BLOCK)[:, :d]


def pack(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def unpack(packed):
    return np.stack([packed & 15, packed >> 4], 2).reshape(packed.shape[0], -1)


def tile_index(n, nb):
    """Byte of the scale tiles that holds row r, block b: [n, nb]."""
    r, b = np.arange(n)[:, None], np.arange(nb)[None]
    return ((r // 128) * (-(-nb // 4)) + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4


def tile_scales(scales):
    n, nb = scales.shape
    out = np.zeros(-(-n // 128) * -(-nb // 4) * 512, dtype=np.uint8)
    out[tile_index(n, nb)] = scales
    return out


def scores(qv, xv, alpha=1.0, bias=None):
    """alpha qv xv^T + bias, and the sum of the terms' magnitudes (for error bounds)."""
    s = alpha * (qv @ xv.T)
    mag = abs(alpha) * (np.abs(qv) @ np.abs(xv).T)
    if bias is not None:
        s, mag = s + bias, mag + np.abs(bias)
    return s, mag
