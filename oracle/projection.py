"""What stands around a projection, in fp64 (formulas in include/dmuon.h):
activations and their slopes, dropout from Philox4x32-10, the residual norm and
its gradients."""
import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[float])
_erfc = np.vectorize(math.erfc, otypes=[float])


def normal_below(z):
    return np.where(z < 0, 0.5 * _erfc(-z / math.sqrt(2)), 0.5 + 0.5 * _erf(z / math.sqrt(2)))


def inner(z, act):
    """u and its slope, where act is z / (1 + exp(-u))."""
    if act == "silu":
        return z, np.ones_like(z)
    c = 2 * math.sqrt(2 / math.pi)
    return c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z * z)


def _sigmoid(u):
    e = np.exp(-np.abs(u))
    return np.where(u < 0, e / (1 + e), 1 / (1 + e))


def activation(z, act):
    if act == "relu":
        return np.maximum(z, 0)
    if act == "gelu":
        return z * normal_below(z)
    if act in ("silu", "gelu_tanh"):
        return z * _sigmoid(inner(z, act)[0])
    return z


def slope(z, act):
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "gelu":
        return normal_below(z) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act in ("silu", "gelu_tanh"):
        u, du = inner(z, act)
        return _sigmoid(u) * (1 + z * du * _sigmoid(-u))
    return np.ones_like(z)


def philox(counter, key):
    """Four words of Philox4x32-10; counter: four integers or arrays, key: two integers."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = list(key)
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return c


def factors(rows, cols, p, seed, offset, first_row=0):
    """What dropout multiplies each element by: 0 or 1 / (1 - p), p in 1 / 65536ths."""
    cut = math.floor(float(np.float32(p)) * 65536 + 0.5)
    out = np.empty((rows, cols))
    r, c = np.meshgrid(np.arange(first_row, first_row + rows), np.arange(cols), indexing="ij")
    words = philox((c // 8, r, np.full_like(r, offset % 2 ** 32), np.full_like(r, offset // 2 ** 32)), (seed % 2 ** 32, seed // 2 ** 32))
    word = np.choose(c % 8 // 2, words).astype(np.int64)
    bits = np.where(c % 2 == 1, word >> 16, word & 0xFFFF)
    out[...] = (bits >= cut) * (65536 / (65536 - cut))
    return out


def add_norm_forward(x, f, w, keep=1.0, eps=1e-6):
    """(y, h, rstd); x may be None, keep as factors() gives it."""
    y = np.where(keep == 0, 0.0, f * keep) + (0.0 if x is None else x)
    r = 1.0 / np.sqrt((y * y).mean(1) + eps)
    return y, y * r[:, None] * w, r


def add_norm_backward(dy, dh, y, w, rstd, keep=1.0):
    """(dx, df, dw) of sum(y * dy) + sum(h * dh)."""
    r = rstd[:, None]
    yn, into = y * r, dh * w
    t = dy + r * (into - yn * (into * yn).mean(1, keepdims=True))
    return t, t * keep, (dh * yn).sum(0)
