"""MXFP8 in fp64: quantisation, the packed layout and reading back.

OCP microscaling: blocks of 32 elements along a row share 2^e, elements are
E4M3 (largest 448).  Codes are found by comparing the scaled magnitude with the
midpoints of the grid; nothing here knows how the kernels do it.
"""
import numpy as np

from .mxfp4 import _blocked

# The magnitudes of codes 0 .. 126: eight subnormals, then 1.m * 2^(x - 7).
GRID = np.array([m / 512 for m in range(8)] + [(1 + m / 8) * 2.0 ** (x - 7) for x in range(1, 16) for m in range(8)][:119])
MIDDLE = (GRID[1:] + GRID[:-1]) / 2


def quantize(x, scale="floor"):
    """Codes [rows, blocks, 32] and scale bytes [rows, blocks] of the rows of x."""
    b = _blocked(np.asarray(x, dtype=np.float64))
    bad = ~np.isfinite(b).all(-1)
    fine = np.where(bad[..., None], 0.0, b)
    amax = np.abs(fine).max(-1)
    _, ex = np.frexp(amax)  # amax = mant 2^ex, mant in [1/2, 1)
    e = ex - 9
    if scale == "ceil":
        e = e + (amax > 448.0 * np.ldexp(1.0, e))
    e = np.clip(np.where(amax > 0, e, -127), -127, 127)
    v = np.minimum(np.ldexp(np.abs(fine), -e[..., None]), 448.0)
    code = np.searchsorted(MIDDLE, v, side="left")  # a tie goes below ...
    tie = (code < 126) & (v == MIDDLE[np.minimum(code, 125)])
    code = code + (tie & (code % 2 == 1))           # ... and to the even code
    code = code + 128 * np.signbit(fine)
    return np.where(bad[..., None], 0, code), np.where(bad, 255, e + 127)


def pack(codes, scale_bytes):
    """(data, scales) bytes as include/dmuon.h lays them out."""
    rows, nb, _ = codes.shape
    rt, kt = -(-rows // 128), -(-nb // 4)
    scales = np.zeros(rt * kt * 512, dtype=np.uint8)
    r, j = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    scales[((r // 128) * kt + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4] = scale_bytes
    return codes.reshape(rows, nb * 32).astype(np.uint8), scales


def values(codes, scale_bytes, k):
    """What codes and scales stand for, [rows, k]."""
    v = GRID[np.minimum(codes % 128, 126)] * np.where(codes >= 128, -1.0, 1.0)
    unit = np.where(scale_bytes == 255, np.nan, np.ldexp(1.0, scale_bytes.astype(np.int64) - 127))
    return (v * unit[..., None]).reshape(codes.shape[0], -1)[:, :k]
