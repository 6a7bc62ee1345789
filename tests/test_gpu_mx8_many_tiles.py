"""The 8-bit tiles where a CTA goes down several of them, so that every slot of a
warp's ring is fetched again: dz and the column sums against fp64 on the device, codes
of rows and columns drawn from all tiles, and of the last ones, against the oracle.
Bars as in test_gpu_act_backward.py.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402
from oracle import mxfp8 as ox  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
ROWS, COLS = 16300, 6200  # 128 x 49 tiles, three down a CTA of 152 SMs or fewer


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    h = dm.Handle(0)
    yield h
    h.close()


def slope_and_bar(z, act):
    if act == "none":
        return torch.ones_like(z), torch.zeros_like(z)
    if act == "relu":
        return (z > 0).double(), torch.zeros_like(z)
    if act == "gelu":
        s, bell = 0.5 * torch.special.erfc(-z / math.sqrt(2)), torch.exp(-z * z / 2)
        return (s + z * bell / math.sqrt(2 * math.pi),
                2.0 ** -20 * (2 + z * z / 2) * (s + z.abs() * bell * 0.4) + 2.0 ** -22 * s)
    c = 2 * math.sqrt(2 / math.pi)
    u, du = (z, torch.ones_like(z)) if act == "silu" else (c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z * z))
    s, rest = torch.sigmoid(u), torch.sigmoid(-u)
    return (s * (1 + z * du * rest), 2.0 ** -20 * (2 + u.abs().clamp(max=100)) * (s + (z * du).abs() * s * rest) +
            torch.where(u.abs() < 30, 2.0 ** -22 * (z * du).abs() * s, 0.0) + 2.0 ** -110)


def buffer(dtype, odd):
    t = torch.full((ROWS, COLS + (5 if odd else 0)), 7.0, dtype=dtype, device="cuda")
    return t[:, 1:1 + COLS] if odd else t


@pytest.mark.parametrize("dtype,act,odd", [("f32", "gelu", False), ("f32", "relu", True), ("f32", "none", False), ("f32", "gelu_tanh", True),
                                           ("bf16", "silu", False), ("bf16", "gelu", True), ("bf16", "relu", False), ("bf16", "none", False),
                                           ("f16", "gelu_tanh", False), ("f16", "silu", True), ("f16", "none", True)])
def test_many_tiles(handle, dtype, act, odd):
    gen = torch.Generator(device="cuda").manual_seed(len(act) + 10 * odd)
    dt, u = DT[dtype], HALF[dtype]
    dout, pre = buffer(dt, odd), buffer(dt, odd)
    dout.copy_(torch.randn((ROWS, COLS), device="cuda", generator=gen))
    pre.copy_(2 * torch.randn((ROWS, COLS), device="cuda", generator=gen))
    dz, d_bias, q, qt = buffer(dt, odd), torch.empty(COLS, device="cuda"), dm.dmuon_mxfp8_empty(ROWS, COLS), dm.dmuon_mxfp8_empty(COLS, ROWS)
    handle.act_backward(dout, None if act == "none" else pre, act, dz=dz, d_bias=d_bias, by_rows=q, by_cols=qt)
    slope, off = slope_and_bar(pre.double(), act)
    want = dout.double() * slope
    bar = dout.double().abs() * off + 2.0 ** -23 * want.abs()
    assert ((dz.double() - want).abs() <= bar * (1 + u) + u * want.abs() + (2.0 ** -25 if dtype == "f16" else 0.0)).all()
    assert ((d_bias.double() - want.sum(0)).abs() <= bar.sum(0) + ROWS * 2.0 ** -23 * want.abs().sum(0)).all()
    if odd:
        assert (dz._base[:, 0] == 7).all() and (dz._base[:, 1 + COLS:] == 7).all()
    del slope, off, want, bar
    wide = torch.empty((ROWS, COLS), device="cuda")  # the values that are quantised, whatever the type of the call
    handle.act_backward(dout.float(), pre.float(), act, dz=wide)
    assert torch.equal(dz, wide.to(dt))

    def check(packed, values, at):
        """The lines `at` of an MXFP8 matrix, whose values these are."""
        codes, byte = ox.quantize(values.cpu().double().numpy())
        assert np.array_equal(packed[0][at].cpu().numpy(), codes.reshape(len(at), -1))
        nb = byte.shape[1]
        place = ((at // 128)[:, None] * -(-nb // 4) + np.arange(nb) // 4) * 512 + (at % 32)[:, None] * 16 + (at % 128 // 32)[:, None] * 4 + np.arange(nb) % 4
        assert np.array_equal(packed[1].cpu().numpy()[place], byte)
    r = np.random.RandomState(len(act))
    rows = np.unique(np.r_[np.arange(0, ROWS, 128) + r.randint(0, 44, -(-ROWS // 128)), ROWS - 44:ROWS])
    cols = np.unique(np.r_[np.arange(0, COLS, 128) + r.randint(0, 56, -(-COLS // 128)), COLS - 20:COLS])
    check(q, wide[torch.from_numpy(rows).cuda()], rows)
    check(qt, wide[:, torch.from_numpy(cols).cuda()].t(), cols)
    assert handle.status()[0] == 0
