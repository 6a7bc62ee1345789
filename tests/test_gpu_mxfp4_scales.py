"""Reading back every code under every scale byte, written into the buffers:
exact up to the type's range, Inf past it, NaN under byte 255; and what the
quantiser makes of blocks at the end of fp32's and bf16's range."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402
from oracle import mxfp4 as ox  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    with dm.Handle(0) as h:
        yield h


def same(got, want):
    got = got.cpu()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(0.0, float("inf"), float("-inf")), want.nan_to_num(0.0, float("inf"), float("-inf")))
    assert torch.equal(torch.signbit(got)[~want.isnan()], torch.signbit(want)[~want.isnan()])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("odd", [0, 1])
def test_every_code_under_every_byte(handle, dtype, odd):
    byte = np.arange(256)[:, None] * np.ones((1, 3), dtype=int)  # a byte a row, all codes in each of its blocks
    codes = np.tile(np.arange(32) % 16, (256, 3, 1))
    data, scales = ox.pack(codes, byte)
    q = torch.from_numpy(data).cuda(), torch.from_numpy(scales).cuda()
    out = torch.zeros((256, 96 + 2 * odd), dtype=DT[dtype], device="cuda")[:, odd:odd + 96]
    handle.mxfp4_dequantize(q, out)
    want = torch.from_numpy(ox.values(codes, byte, 96)).to(DT[dtype])
    same(out, want)
    if dtype != "f16":  # the range stated in the header
        mag = np.abs(ox.GRID[codes % 8]).reshape(256, 96)
        over = ((byte[:, :1] == 253) & (mag >= 4)) | ((byte[:, :1] == 254) & (mag >= 2))
        assert np.array_equal(out.isinf().cpu().numpy(), over)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale,byte", [("floor", 252), ("ceil", 253)])
def test_blocks_at_the_end_of_the_range(handle, dtype, scale, byte):
    x = torch.full((4, 64), 1.0, dtype=DT[dtype])
    x[0, 3], x[1, 40] = torch.finfo(DT[dtype]).max, torch.finfo(DT[dtype]).min
    q = dm.dmuon_mxfp4_empty(4, 64)
    handle.mxfp4_quantize(x.cuda(), by_rows=q, scale=scale)
    codes, bytes_ = ox.quantize(x.double().numpy(), scale)
    assert bytes_[0, 0] == byte and bytes_[1, 1] == byte
    data, scales = ox.pack(codes, bytes_)
    assert np.array_equal(q[0].cpu().numpy(), data) and np.array_equal(q[1].cpu().numpy(), scales)
    out = torch.empty((4, 64), dtype=DT[dtype], device="cuda")
    handle.mxfp4_dequantize(q, out)
    same(out, torch.from_numpy(ox.values(codes, bytes_, 64)).to(DT[dtype]))
    assert bool(out.isinf().any()) == (scale == "ceil")
