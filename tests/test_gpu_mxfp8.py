"""MXFP8 quantisation and reading back against oracle/mxfp8.py: packed bytes
(padding included) and values have to be equal bit for bit."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402
from oracle import mxfp8 as ox  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    h = dm.Handle(0)
    yield h
    h.close()


def _values(rows, cols, seed, dtype):
    """Rows and columns of different size, exact ties, zeros and whole zero blocks."""
    r = np.random.RandomState(seed)
    x = r.randn(rows, cols) * np.exp(2 * r.randn(rows, 1)) * np.exp(r.randn(1, cols))
    tie = r.randint(-512, 513, (rows, cols)) / 16.0
    x = np.where(r.rand(rows, cols) < 0.4, tie, x)
    x = np.where(r.rand(rows, cols) < 0.05, 0.0, x)
    if rows > 40 and cols > 70:
        x[32:64, 32:64] = 0.0
    return torch.from_numpy(x).to(DT[dtype])


def on_gpu(t, odd):
    """The same values; odd: in a wider buffer, one element off, with an odd pitch."""
    if not odd:
        return t.cuda()
    rows, cols = t.shape
    buf = torch.zeros((rows, cols + 5), dtype=t.dtype, device="cuda")
    v = buf[:, 1:1 + cols]
    v.copy_(t)
    return v


def filled(rows, k):
    """Buffers that hold something else before the call."""
    d, s = dm.dmuon_mxfp8_empty(rows, k)
    return d.fill_(0xAB), s.fill_(0xFF)


def check_packed(got, codes, byte):
    data, scales = ox.pack(codes, byte)
    assert np.array_equal(got[0].cpu().numpy(), data)
    assert np.array_equal(got[1].cpu().numpy(), scales)


SHAPES = [(1, 1), (1, 32), (1, 4096), (5, 33), (31, 31), (128, 128), (129, 257), (300, 64), (77, 2061), (640, 96)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scale,odd", [("floor", False), ("ceil", True), ("ceil", False), ("floor", True)])
def test_quantize_is_exact(handle, shape, dtype, scale, odd):
    rows, cols = shape
    x = _values(rows, cols, 7 * rows + cols, dtype)
    src = on_gpu(x, odd)
    by_rows, by_cols = filled(rows, cols), filled(cols, rows)
    handle.mxfp8_quantize(src, by_rows=by_rows, by_cols=by_cols, scale=scale)
    only_rows, only_cols = filled(rows, cols), filled(cols, rows)
    handle.mxfp8_quantize(src, by_rows=only_rows, scale=scale)
    handle.mxfp8_quantize(src, by_cols=only_cols, scale=scale)
    x64 = x.double().numpy()
    for want, both, one, k in ((ox.quantize(x64, scale), by_rows, only_rows, cols), (ox.quantize(x64.T, scale), by_cols, only_cols, rows)):
        check_packed(both, *want)
        check_packed(one, *want)
        out = on_gpu(torch.empty((want[0].shape[0], k), dtype=DT[dtype]).fill_(3), odd)
        handle.mxfp8_dequantize(both, out)
        assert torch.equal(out.cpu(), torch.from_numpy(ox.values(*want, k)).to(DT[dtype]))
        if odd:  # nothing around the rows is written
            buf = out._base
            assert not buf[:, 0].any() and not buf[:, 1 + k:].any()
    assert handle.status()[0] == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_quantize_special_values(handle, dtype):
    """Infinities, NaN, the type's largest and smallest values, signed zeros:
    one special element a block, along rows and along columns."""
    info = torch.finfo(DT[dtype])
    sub = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}[dtype]
    special = [float("inf"), float("-inf"), float("nan"), info.max, info.min, info.tiny, sub, -sub, -0.0, 3 * sub]
    x = torch.randn(96, 32 * len(special), generator=torch.Generator().manual_seed(5)).to(DT[dtype])
    for i, v in enumerate(special):
        x[i, 32 * i + 7] = v
        x[32 + i, 32 * i:32 * i + 32] = 0  # alone in a row block
        x[32 + i, 32 * i + 3] = v
        x[64:, 32 * i + i] = 0             # alone in a column block
        x[70, 32 * i + i] = v
    for scale in ("floor", "ceil"):
        by_rows, by_cols = filled(*x.shape), filled(x.shape[1], x.shape[0])
        handle.mxfp8_quantize(x.cuda(), by_rows=by_rows, by_cols=by_cols, scale=scale)
        x64 = x.double().numpy()
        for want, got, k in ((ox.quantize(x64, scale), by_rows, x.shape[1]), (ox.quantize(x64.T, scale), by_cols, x.shape[0])):
            check_packed(got, *want)
            out = torch.empty((want[0].shape[0], k), dtype=torch.float32, device="cuda")
            handle.mxfp8_dequantize(got, out)
            with np.errstate(over="ignore"):  # 256 * 2^120, the nearest code of fp32's largest value under ceil, is Inf there
                assert np.array_equal(out.cpu().numpy(), ox.values(*want, k).astype(np.float32), equal_nan=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_every_code_and_scale_reads_back(handle, dtype):
    codes = np.tile(np.arange(256).reshape(8, 32), (1, 32)).reshape(256, 1, 32)[:128]
    codes = np.where(codes % 128 == 127, 0, codes)  # no NaN codes: the quantiser writes none
    for bytes_ in (np.arange(0, 128), np.arange(100, 228)):
        byte = bytes_.reshape(128, 1)
        data, scales = ox.pack(codes, byte)
        out = torch.empty((128, 32), dtype=DT[dtype], device="cuda")
        handle.mxfp8_dequantize((torch.from_numpy(data).cuda(), torch.from_numpy(scales).cuda()), out)
        assert torch.equal(out.cpu(), torch.from_numpy(ox.values(codes, byte, 32)).to(DT[dtype]))


def test_empty(handle):
    for r, c in ((0, 5), (5, 0), (0, 0)):
        handle.mxfp8_quantize(torch.empty((r, c), device="cuda"), dm.dmuon_mxfp8_empty(r, c), dm.dmuon_mxfp8_empty(c, r))
        handle.mxfp8_dequantize(dm.dmuon_mxfp8_empty(r, c), torch.empty((r, c), device="cuda"))


def test_refusals(handle):
    x = torch.zeros((8, 64), device="cuda")
    q, q4 = dm.dmuon_mxfp8_empty(8, 64), dm.dmuon_mxfp4_empty(8, 64)
    for bad in (dict(by_rows=q4), dict(by_cols=q), dict(by_rows=(q[0][:, :32], q[1]))):
        with pytest.raises(ValueError):
            handle.mxfp8_quantize(x, **bad)
    with pytest.raises(dm.DmuonError):
        handle.mxfp8_quantize(x)
    with pytest.raises(dm.DmuonError):
        handle.mxfp8_quantize(x, by_rows=q, by_cols=(q[0].new_empty((64, 32)), q[1]))  # the same scales twice
    with pytest.raises(KeyError):
        handle.mxfp8_quantize(x, by_rows=q, scale="round")
    with pytest.raises(ValueError):
        handle.mxfp8_quantize(x.double(), by_rows=q)
    with pytest.raises(ValueError):
        handle.mxfp8_dequantize(q, x.t())
