"""The fp64 oracles of MXFP8, of Philox and of what stands around a projection,
pinned by hand values, published vectors and central differences (no GPU)."""
import numpy as np
import pytest

from oracle import mxfp8 as ox
from oracle import projection as op

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def test_grid():
    assert len(ox.GRID) == 127 and ox.GRID[0] == 0 and ox.GRID[1] == 2.0 ** -9 and ox.GRID[8] == 2.0 ** -6 and ox.GRID[-1] == 448
    assert (np.diff(ox.GRID) > 0).all()


def test_codes_of_hand_values():
    x = np.zeros((1, 32))
    x[0, :9] = [256, 448, -448, 500, 1, 1.0625, 1.1875, -0.0, 2.0 ** -10]
    codes, byte = ox.quantize(x)
    assert byte[0, 0] == 127
    assert codes[0, 0, :9].tolist() == [120, 126, 254, 126, 56, 56, 58, 128, 0]  # 1.0625 and 1.1875 are ties
    assert ox.values(codes, byte, 32)[0, :4].tolist() == [256, 448, -448, 448]


@pytest.mark.parametrize("amax,floor_e,ceil_e", [(256.0, 0, 0), (448.0, 0, 0), (448.5, 0, 1), (511.0, 0, 1), (512.0, 1, 1), (1.0, -8, -8),
                                                 (2.0 ** -140, -127, -127), (0.0, -127, -127), (2.0 ** 127 * 1.9, 119, 120)])
def test_block_exponents(amax, floor_e, ceil_e):
    x = np.zeros((1, 32))
    x[0, 5] = -amax
    assert ox.quantize(x, "floor")[1][0, 0] == floor_e + 127
    assert ox.quantize(x, "ceil")[1][0, 0] == ceil_e + 127


def test_nan_blocks_and_layout():
    x = np.ones((130, 160))
    x[7, 33] = np.inf
    x[129, 159] = np.nan
    codes, byte = ox.quantize(x)
    assert byte[7].tolist() == [119, 255, 119, 119, 119] and not codes[7, 1].any() and byte[129, 4] == 255
    data, scales = ox.pack(codes, byte)
    assert data.shape == (130, 160) and scales.size == 2 * 2 * 512
    assert scales[7 * 16 + 1] == 255 and scales[3 * 512 + 1 * 16] == 255 and not scales[3 * 512 + 1 * 16 + 1:3 * 512 + 2 * 16].any()
    assert np.isnan(ox.values(codes, byte, 160)[7, 32:64]).all()


@pytest.mark.parametrize("counter,key,want", [  # the method's published known answers
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0), (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_philox(counter, key, want):
    assert tuple(int(v) for v in op.philox(counter, key)) == want


@pytest.mark.parametrize("p,share", [(0.0, 1.0), (0.1, 58982 / 65536), (0.5, 0.5)])
def test_factors(p, share):
    m = op.factors(300, 517, p, 123456789012345, 2 ** 40 + 5)
    kept = m > 0
    assert abs(kept.mean() - share) <= 6 * (share * (1 - share) / m.size) ** 0.5
    assert np.all(m[kept] == 1 / share)


@pytest.mark.parametrize("act", ACTS)
def test_slopes_against_differences(act):
    z = np.linspace(-6, 6, 97) + 0.003
    d = 1e-5
    want = (op.activation(z + d, act) - op.activation(z - d, act)) / (2 * d)
    assert np.abs(op.slope(z, act) - want).max() < 1e-8
    assert op.activation(np.array([-50.0]), act)[0] == pytest.approx(-50.0 if act == "none" else 0.0, abs=1e-19)


def test_add_norm_gradients_against_differences():
    r = np.random.RandomState(3)
    x, f, dy, dh = (r.randn(5, 7) for _ in range(4))
    w = r.randn(7)
    keep = op.factors(5, 7, 0.3, 11, 4)

    def total(x, f, w):
        y, h, _ = op.add_norm_forward(x, f, w, keep)
        return (y * dy).sum() + (h * dh).sum()
    y, _, rstd = op.add_norm_forward(x, f, w, keep)
    got = op.add_norm_backward(dy, dh, y, w, rstd, keep)
    for k, g in zip(range(3), got):
        v = [x, f, w][k]
        for i in np.ndindex(v.shape):
            a, b = ([t.copy() for t in (x, f, w)] for _ in range(2))
            a[k][i] += 1e-6
            b[k][i] -= 1e-6
            assert abs((total(*a) - total(*b)) / 2e-6 - g[i]) < 1e-6
