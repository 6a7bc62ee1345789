"""Backward of bias and activation against fp64.

slope's bar: 2^-20 (2 + |u|) of its terms s and z u' s (1 - s), and 2^-22 of z u' s
for the difference 1 - s (none past |u| = 30, where s is 0 or 1 to the last bit);
dz then rounds once.  Codes are those of the fp32 dz, bit for bit: dz of an fp32
call quantised by the oracle.  Column sums: rows 2^-23 of the sum of magnitudes.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402
from oracle import mxfp8 as ox  # noqa: E402
from oracle import projection as op  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    h = dm.Handle(0)
    yield h
    h.close()


def buffer(rows, cols, dtype, odd, fill=7.0):
    t = torch.full((rows, cols + (5 if odd else 0)), fill, dtype=dtype, device="cuda")
    return t[:, 1:1 + cols] if odd else t


def on_gpu(t, odd):
    v = buffer(*t.shape, t.dtype, odd)
    v.copy_(t)
    return v


def packed(rows, k):
    d, s = dm.dmuon_mxfp8_empty(rows, k)
    return d.fill_(0xAB), s.fill_(0xFF)


def slope_bar(z, act):
    if act in ("none", "relu"):
        return 0 * z
    if act == "gelu":
        s = op.normal_below(z)
        return 2.0 ** -20 * (2 + z * z / 2) * (s + np.abs(z) * np.exp(-z * z / 2) * 0.4) + 2.0 ** -22 * np.abs(s)
    u, du = op.inner(z, act)
    s = op._sigmoid(u)
    return (2.0 ** -20 * (2 + np.minimum(np.abs(u), 100)) * (s + np.abs(z * du) * s * op._sigmoid(-u)) +
            np.where(np.abs(u) < 30, 2.0 ** -22 * np.abs(z * du) * s, 0) + 2.0 ** -110)


SHAPES = [(1, 1), (1, 300), (5, 33), (31, 31), (128, 128), (129, 257), (300, 64), (77, 2061), (640, 96), (2600, 520)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("act,odd", [("none", False), ("relu", True), ("silu", False), ("gelu", True), ("gelu_tanh", False), ("silu", True)])
def test_against_fp64(handle, shape, dtype, act, odd):
    rows, cols = shape
    g = torch.Generator().manual_seed(rows * 31 + cols)
    dout, pre = torch.randn(shape, generator=g).to(DT[dtype]), (2 * torch.randn(shape, generator=g)).to(DT[dtype])
    src, z = on_gpu(dout, odd), on_gpu(pre, odd)
    out = dict(dz=buffer(rows, cols, DT[dtype], odd), d_bias=torch.full((cols,), 7.0, device="cuda"), by_rows=packed(rows, cols),
               by_cols=packed(cols, rows))
    handle.act_backward(src, None if act == "none" else z, act, **out)
    d64, z64 = dout.double().numpy(), pre.double().numpy()
    want = d64 * op.slope(z64, act)
    bar = np.abs(d64) * slope_bar(z64, act) + 2.0 ** -23 * np.abs(want)
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0
    u = HALF[dtype]
    assert (np.abs(out["dz"].cpu().double().numpy() - want) <= bar * (1 + u) + u * np.abs(want) + tiny).all()
    sums = np.abs(out["d_bias"].cpu().double().numpy() - want.sum(0))
    assert (sums <= bar.sum(0) + rows * 2.0 ** -23 * np.abs(want).sum(0)).all()
    if odd:
        assert (out["dz"]._base[:, 0] == 7).all() and (out["dz"]._base[:, 1 + cols:] == 7).all()
    # the same values as fp32: their dz is what is quantised, whatever the type of the call
    wide = torch.empty(shape, device="cuda")
    handle.act_backward(dout.float().cuda(), pre.float().cuda(), act, dz=wide)
    w64 = wide.cpu().double().numpy()
    assert torch.equal(out["dz"].cpu(), wide.to(DT[dtype]).cpu())
    for got, v in ((out["by_rows"], w64), (out["by_cols"], w64.T)):
        data, scales = ox.pack(*ox.quantize(v))
        assert np.array_equal(got[0].cpu().numpy(), data) and np.array_equal(got[1].cpu().numpy(), scales)
    # every output alone, and again: the same bits
    for name in out:
        fresh = {"dz": lambda: buffer(rows, cols, DT[dtype], odd), "d_bias": lambda: torch.zeros(cols, device="cuda"),
                 "by_rows": lambda: packed(rows, cols), "by_cols": lambda: packed(cols, rows)}[name]()
        handle.act_backward(src, z, act, **{name: fresh})
        for a, b in zip(fresh if isinstance(fresh, tuple) else (fresh,), out[name] if isinstance(fresh, tuple) else (out[name],)):
            assert torch.equal(a, b)
    assert handle.status()[0] == 0


@pytest.mark.parametrize("act", ACTS)
def test_ceil_and_special_values(handle, act):
    z = torch.linspace(-6, 6, 64 * 96).view(64, 96)
    dout = torch.randn(64, 96, generator=torch.Generator().manual_seed(2))
    dout[3, 40], dout[5, 70], z[9, 1], z[11, 2], z[12, 95] = float("inf"), float("nan"), 1e30, -1e30, float("inf")
    dz, q = torch.empty((64, 96), device="cuda"), packed(64, 96)
    handle.act_backward(dout.cuda(), z.cuda(), act, dz=dz, by_rows=q, scale="ceil")
    got = dz.cpu().double().numpy()
    data, scales = ox.pack(*ox.quantize(got, "ceil"))
    assert np.array_equal(q[0].cpu().numpy(), data) and np.array_equal(q[1].cpu().numpy(), scales)
    assert got[9, 1] == float(dout[9, 1]) and got[12, 95] == float(dout[12, 95]) and got[11, 2] == (float(dout[11, 2]) if act == "none" else 0)
    assert z[5, 70] < 0 and (got[5, 70] == 0 if act == "relu" else np.isnan(got[5, 70])) and np.isfinite(got[3, :40]).all()


def test_no_rows_and_no_columns(handle):
    bias = torch.full((37,), 5.0, device="cuda")
    handle.act_backward(torch.empty((0, 37), device="cuda"), None, "none", d_bias=bias)
    assert not bias.any()
    handle.act_backward(torch.empty((4, 0), device="cuda"), None, "none", d_bias=torch.empty(0, device="cuda"), dz=torch.empty((4, 0), device="cuda"))
    handle.act_backward(torch.empty((0, 37), device="cuda"), None, "none", dz=torch.empty((0, 37), device="cuda"))


def test_refusals(handle):
    x = torch.zeros((8, 64), device="cuda")
    q = dm.dmuon_mxfp8_empty(8, 64)
    for bad in (dict(), dict(dz=x.half()), dict(d_bias=torch.zeros(63, device="cuda")), dict(by_cols=q), dict(pre=None, act="relu", dz=x)):
        with pytest.raises(ValueError):
            handle.act_backward(**dict(dict(dout=x, pre=x, act="silu"), **bad))
    for bad in (dict(dz=x), dict(by_rows=(q[0], q[0].view(-1)[:512]))):
        with pytest.raises(dm.DmuonError):
            handle.act_backward(x, x, "silu", **bad)
    with pytest.raises(KeyError):
        handle.act_backward(x, x, "swish", dz=torch.empty_like(x))
