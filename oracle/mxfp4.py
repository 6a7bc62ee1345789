"""MXFP4 in fp64: quantisation, the packed layout, reading back and the product.

OCP microscaling: blocks of 32 elements along a row share 2^e, elements are
E2M1.  Codes are found by comparing the scaled magnitude with the midpoints
of the grid (nearest) or with the fraction of the way to the next value
(stochastic); nothing here knows how the kernels do it.
"""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _blocked(x):
    rows, k = x.shape
    nb = -(-k // 32)
    out = np.zeros((rows, nb * 32), dtype=x.dtype)
    out[:, :k] = x
    return out.reshape(rows, nb, 32)


def quantize(x, scale="floor", noise=None):
    """Codes [rows, blocks, 32] and scale bytes [rows, blocks] of the rows of x."""
    b = _blocked(np.asarray(x, dtype=np.float64))
    bad = ~np.isfinite(b).all(-1)
    fine = np.where(bad[..., None], 0.0, b)
    amax = np.abs(fine).max(-1)
    mant, ex = np.frexp(amax)  # amax = mant 2^ex, mant in [1/2, 1)
    e = ex - 3
    if scale == "ceil":
        e = e + (amax > 6.0 * np.ldexp(1.0, e))
    e = np.clip(np.where(amax > 0, e, -127), -127, 127)
    v = np.minimum(np.ldexp(np.abs(fine), -e[..., None]), 6.0)
    if noise is None:
        code = np.zeros(v.shape, dtype=np.int64)
        for j in range(7):
            mid = (GRID[j] + GRID[j + 1]) / 2
            code += (v >= mid) if j % 2 else (v > mid)
    else:
        r = _blocked(np.asarray(noise)).astype(np.float64)
        code = np.searchsorted(GRID, v, side="right") - 1
        nxt = np.minimum(code + 1, 7)
        gap = np.where(nxt > code, GRID[nxt] - GRID[code], 1.0)
        code = code + ((v - GRID[code]) / gap * 256 > r + 0.5)
    code = code + 8 * np.signbit(fine)
    return np.where(bad[..., None], 0, code), np.where(bad, 255, e + 127)


def pack(codes, scale_bytes):
    """(data, scales) bytes as include/dmuon.h lays them out."""
    rows, nb, _ = codes.shape
    c = codes.reshape(rows, nb * 16, 2).astype(np.uint8)
    data = c[:, :, 0] | (c[:, :, 1] << 4)
    rt, kt = -(-rows // 128), -(-nb // 4)
    scales = np.zeros(rt * kt * 512, dtype=np.uint8)
    for r in range(rows):
        for j in range(nb):
            scales[((r // 128) * kt + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4] = scale_bytes[r, j]
    return data, scales


def values(codes, scale_bytes, k):
    """What codes and scales stand for, [rows, k]."""
    v = GRID[codes % 8] * np.where(codes >= 8, -1.0, 1.0)
    unit = np.where(scale_bytes == 255, np.nan, np.ldexp(1.0, scale_bytes.astype(np.int64) - 127))
    return (v * unit[..., None]).reshape(codes.shape[0], -1)[:, :k]
