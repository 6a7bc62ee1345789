"""The norms after and before a block with its gate and residual scale, and
their gradients, in fp64 (formulas in include/dmuon.h)."""
import numpy as np


def _gate_rows(gate, rows, per):
    return 1.0 if gate is None else gate[np.arange(rows) // per]


def forward(x, f, post_w, pre_w, gate=None, per=None, res=None, eps=1e-6):
    """(y, h, rstd [2, rows])."""
    rows = f.shape[0]
    r1 = 1.0 / np.sqrt((f * f).mean(1, keepdims=True) + eps)
    y = (1.0 if res is None else res) * x + _gate_rows(gate, rows, per) * (f * r1 * post_w)
    r2 = 1.0 / np.sqrt((y * y).mean(1, keepdims=True) + eps)
    return y, y * r2 * pre_w, np.stack((r1[:, 0], r2[:, 0]))


def backward(dy, dh, x, f, y, post_w, pre_w, rstd, gate=None, per=None, res=None):
    """Gradients of sum(y * dy) + sum(h * dh), from the forward's y and rstd."""
    rows = f.shape[0]
    r1, r2 = rstd[0][:, None], rstd[1][:, None]
    yn, fn = y * r2, f * r1
    into = dh * pre_w
    t = dy + r2 * (into - yn * (into * yn).mean(1, keepdims=True))
    g = _gate_rows(gate, rows, per)
    back = g * t * post_w
    out = {"dx": (1.0 if res is None else res) * t, "df": r1 * (back - fn * (back * fn).mean(1, keepdims=True)),
           "d_post_w": (g * t * fn).sum(0), "d_pre_w": (dh * yn).sum(0)}
    if gate is not None:
        out["d_gate"] = np.zeros_like(gate)
        np.add.at(out["d_gate"], np.arange(rows) // per, t * fn * post_w)
    if res is not None:
        out["d_res_scale"] = (t * x).sum(0)
    return out
