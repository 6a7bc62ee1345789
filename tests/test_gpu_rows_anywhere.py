"""Rows on any element: every distance from a 16-byte boundary gives the same
bits, and nothing outside the rows is written."""
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "u8": torch.uint8}


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    with dm.Handle(0) as h:
        yield h


class At:
    """A matrix `off` elements into a buffer of pitch cols + pad, 7s around it."""

    def __init__(self, rows, cols, dtype, off, pad, src=None):
        self.rows, self.cols, self.pitch, self.off = rows, cols, cols + pad, off
        self.buf = torch.full((rows * self.pitch + 16,), 7, dtype=DT[dtype], device="cuda")
        self.t = self.buf[off:off + rows * self.pitch].view(rows, self.pitch)[:, :cols]
        if src is not None:
            self.t.copy_(src)

    def check(self, want):
        assert torch.equal(self.t, want)
        outside = torch.full_like(self.buf, 7)
        outside[self.off:self.off + self.rows * self.pitch].view(self.rows, self.pitch)[:, :self.cols] = self.t
        assert torch.equal(self.buf, outside)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (300, 33), (70, 50), (5, 257), (130, 515), (9, 2061)])
def test_quantise_and_read_back(handle, dtype, rows, cols):
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = torch.randn(rows, cols, device="cuda", generator=gen).to(DT[dtype])
    noise = torch.randint(0, 256, (rows, cols), dtype=torch.uint8, device="cuda", generator=gen)

    def quantise(x, noise):
        q, qt = dm.dmuon_mxfp4_empty(rows, cols), dm.dmuon_mxfp4_empty(cols, rows)
        handle.mxfp4_quantize(x, q, qt, noise=noise, scale="ceil")
        return q + qt
    cols16 = -(-cols // 16) * 16 - cols
    plain = quantise(At(rows, cols, dtype, 0, cols16, x).t, None)
    noisy = quantise(At(rows, cols, dtype, 0, cols16, x).t, At(rows, cols, "u8", 0, cols16, noise).t)
    values = At(rows, cols, dtype, 0, cols16)
    handle.mxfp4_dequantize(plain[:2], values.t)
    for off in range(16):
        pad = 1 + off % 4
        for got, want in zip(quantise(At(rows, cols, dtype, off % 8, pad, x).t, None), plain):
            assert torch.equal(got, want)
        for got, want in zip(quantise(At(rows, cols, dtype, off % 8, pad, x).t, At(rows, cols, "u8", off, pad, noise).t), noisy):
            assert torch.equal(got, want)
        if off < 8:
            out = At(rows, cols, dtype, off, pad)
            handle.mxfp4_dequantize(plain[:2], out.t)
            out.check(values.t)
    assert handle.status()[0] == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(5, 1), (40, 31), (33, 129), (20, 257), (10, 1111), (6, 4097), (5, 9001)])
def test_norms(handle, dtype, rows, cols):
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    x, f, dy, dh = (torch.randn(rows, cols, device="cuda", generator=gen).to(DT[dtype]) for _ in range(4))
    w, v, s = (torch.rand(cols, device="cuda", generator=gen) + 0.5 for _ in range(3))
    gate = torch.rand(-(-rows // 3), cols, device="cuda", generator=gen) + 0.5
    first = None
    for off in range(8):
        pad = 8 + off % 3

        def at(src=None):
            return At(rows, cols, dtype, off, pad, src)
        y, out, dx, df = at(), at(), at(), at()
        rstd, sums, dg = torch.zeros(2, rows, device="cuda"), torch.zeros(3, cols, device="cuda"), torch.zeros_like(gate)
        xs, fs = at(x), at(f)
        handle.block_norm_forward(xs.t, fs.t, w, v, y.t, out.t, rstd, gate=gate, rows_per_gate=3, res_scale=s)
        handle.block_norm_backward(at(dy).t, at(dh).t, xs.t, fs.t, y.t, w, v, rstd, dx.t, df.t, sums[0], sums[1], gate=gate,
                                   d_gate=dg, rows_per_gate=3, res_scale=s, d_res_scale=sums[2])
        mats, rest = (y, out, dx, df), (rstd, sums, dg)
        if first is None:
            first = [m.t.clone() for m in mats], [t.clone() for t in rest]
        for m, want in zip(mats, first[0]):
            m.check(want)
        for t, want in zip(rest, first[1]):
            assert torch.equal(t, want)
    assert handle.status()[0] == 0
