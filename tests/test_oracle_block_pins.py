"""The fp64 oracles of the MXFP4 format and of the block norms, pinned by hand
values and by central differences (no GPU)."""
import numpy as np
import pytest

from oracle import block_norm as on
from oracle import mxfp4 as ox


def test_codes_of_hand_values():
    x = np.zeros((1, 32))
    x[0, :16] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -6, -5, -3.5, -2.5, -1.75, -1.25, -0.75, -0.25]
    codes, byte = ox.quantize(x)
    assert byte[0, 0] == 127  # e = floor(log2 6) - 2 = 0
    assert codes[0, 0, :16].tolist() == [7, 6, 6, 4, 4, 2, 2, 0, 15, 14, 14, 12, 12, 10, 10, 8]  # ties to even codes
    assert ox.values(codes, byte, 32)[0, :4].tolist() == [6, 4, 4, 2]


@pytest.mark.parametrize("amax,floor_e,ceil_e", [(4.0, 0, 0), (6.0, 0, 0), (6.01, 0, 1), (7.9, 0, 1), (8.0, 1, 1),
                                                 (2.0 ** -130, -127, -127), (1.0, -2, -2), (0.0, -127, -127)])
def test_block_exponents(amax, floor_e, ceil_e):
    x = np.zeros((1, 32))
    x[0, 5] = -amax
    assert ox.quantize(x, "floor")[1][0, 0] == floor_e + 127
    assert ox.quantize(x, "ceil")[1][0, 0] == ceil_e + 127


def test_stochastic_codes():
    x = np.full((256, 32), 2.5)  # halfway between codes 4 (2) and 5 (3) with amax 4 in the block
    x[:, 0] = 4.0
    codes, _ = ox.quantize(x, "ceil", np.arange(256)[:, None] * np.ones((1, 32), dtype=int))
    assert (codes[:128, 0, 1] == 5).all() and (codes[128:, 0, 1] == 4).all()
    assert (codes[:, 0, 0] == 6).all()


def test_nan_and_inf_blocks():
    x = np.ones((1, 96))
    x[0, 3], x[0, 40] = np.nan, np.inf
    codes, byte = ox.quantize(x)
    assert byte[0].tolist() == [255, 255, 125] and not codes[0, :2].any()
    v = ox.values(codes, byte, 96)
    assert np.isnan(v[0, :64]).all() and (v[0, 64:] == 1).all()


def test_packed_layout():
    codes = np.arange(130 * 5 * 32).reshape(130, 5, 32) % 16
    byte = np.arange(130 * 5).reshape(130, 5) % 251
    data, scales = ox.pack(codes, byte)
    assert data.shape == (130, 80) and scales.size == 2 * 2 * 512
    assert data[7, 3] == codes[7, 0, 6] + 16 * codes[7, 0, 7]
    assert scales[(37 % 32) * 16 + (37 // 32) * 4 + 2] == byte[37, 2]
    assert scales[3 * 512 + 1 * 16] == byte[129, 4]  # second tile row, second tile column
    assert not scales[3 * 512 + 1:3 * 512 + 4].any()


@pytest.mark.parametrize("rows,cols,per,res", [(5, 7, None, False), (6, 9, 4, True), (4, 3, 1, True), (3, 16, 3, False)])
def test_norm_gradients_against_differences(rows, cols, per, res):
    r = np.random.RandomState(rows * 10 + cols)
    x, f, dy, dh = (r.randn(rows, cols) for _ in range(4))
    p = {"post_w": r.randn(cols), "pre_w": r.randn(cols)}
    if per:
        p["gate"] = r.randn(-(-rows // per), cols)
    if res:
        p["res"] = r.randn(cols)

    def loss(x, f, p):
        y, h, _ = on.forward(x, f, p["post_w"], p["pre_w"], p.get("gate"), per, p.get("res"), 1e-3)
        return (y * dy).sum() + (h * dh).sum()

    y, _, rstd = on.forward(x, f, p["post_w"], p["pre_w"], p.get("gate"), per, p.get("res"), 1e-3)
    g = on.backward(dy, dh, x, f, y, p["post_w"], p["pre_w"], rstd, p.get("gate"), per, p.get("res"))
    eps = 1e-6
    for name, grad in g.items():
        key = {"dx": "x", "df": "f"}.get(name, name[2:].replace("res_scale", "res"))
        base = {"x": x, "f": f, **p}[key]
        num = np.zeros_like(base)
        for i in np.ndindex(*base.shape):
            side = []
            for sgn in (1, -1):
                v = base.copy()
                v[i] += sgn * eps
                q = dict(p, **({key: v} if key in p else {}))
                side.append(loss(v if key == "x" else x, v if key == "f" else f, q))
            num[i] = (side[0] - side[1]) / (2 * eps)
        # central differences: eps^2 truncation plus rounding of the loss over eps
        assert np.allclose(num, grad, rtol=1e-6, atol=1e-7), name
