"""Offsets past 2^31 elements and bytes: a matrix of a long pitch gives the bits
of the same matrix stored densely, and the last rows of a long one those of
these rows alone."""
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402

pytestmark = pytest.mark.gpu

ROWS, PITCH = 70016, 32768  # 2.3e9 elements


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    _build.build()
    with dm.Handle(0) as h:
        yield h
    torch.cuda.empty_cache()


def far(cols, pitch, like=None):
    t = torch.zeros(ROWS * pitch, dtype=torch.bfloat16, device="cuda").view(ROWS, pitch)[:, :cols]
    if like is not None:
        t.copy_(like)
    return t


@pytest.mark.parametrize("cols,pitch", [(40, PITCH), (37, PITCH + 1)])
def test_long_pitch(handle, cols, pitch):
    gen = torch.Generator(device="cuda").manual_seed(cols)

    def act():
        return torch.randn(ROWS, pitch - PITCH + 40, device="cuda", generator=gen).bfloat16()[:, :cols]
    x, f, dy, dh = act(), act(), act(), act()
    w = torch.rand(cols, device="cuda", generator=gen) + 0.5

    def run(mat):
        r = {}
        y, out, dx, df = mat(None), mat(None), mat(None), mat(None)
        rstd = torch.zeros((2, ROWS), device="cuda")
        handle.block_norm_forward(mat(x), mat(f), w, w, y, out, rstd)
        sums = torch.zeros(3, cols, device="cuda")
        handle.block_norm_backward(mat(dy), mat(dh), mat(x), mat(f), y, w, w, rstd, dx, df, sums[0], sums[1], res_scale=w,
                                   d_res_scale=sums[2])
        q, qt = dm.dmuon_mxfp4_empty(ROWS, cols), dm.dmuon_mxfp4_empty(cols, ROWS)
        handle.mxfp4_quantize(out, q, qt)
        values, prod = mat(None), mat(None)
        handle.mxfp4_dequantize(q, values)
        b = dm.dmuon_mxfp4_empty(cols, cols)
        handle.mxfp4_quantize(x[:cols], b)
        handle.mxfp4_gemm(q, b, prod, cols)
        for i, t in enumerate((y, out, rstd, dx, df, sums, *q, *qt, values, prod)):
            r[i] = t.contiguous()
        torch.cuda.synchronize()
        return r

    def dense(t):
        return t if t is not None else torch.zeros(ROWS, pitch - PITCH + 40, dtype=torch.bfloat16, device="cuda")[:, :cols]
    want = run(dense)
    got = run(lambda t: far(cols, pitch, t))
    for i in want:
        assert torch.equal(got[i], want[i]), i
    assert handle.status()[0] == 0


def test_long_matrix(handle):
    k, last = 65536, 128
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty((ROWS, k), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    q, qt = dm.dmuon_mxfp4_empty(ROWS, k), dm.dmuon_mxfp4_empty(k, ROWS)
    handle.mxfp4_quantize(x, q, qt, scale="ceil")
    tail = x[ROWS - last:]
    p, pt = dm.dmuon_mxfp4_empty(last, k), dm.dmuon_mxfp4_empty(k, last)
    handle.mxfp4_quantize(tail, p, pt, scale="ceil")
    assert q[0].numel() > 2 ** 31
    assert torch.equal(q[0][ROWS - last:], p[0]) and torch.equal(q[1][-p[1].numel():], p[1])
    assert torch.equal(qt[0][:, -(last // 2):], pt[0])
    out, end = x, torch.empty_like(tail)
    handle.mxfp4_dequantize(q, out)
    handle.mxfp4_dequantize(p, end)
    assert torch.equal(out[ROWS - last:], end)
    # With every scale 1 a sum of products of 4-bit values is exact in fp32.
    q[1].fill_(127)
    p[1].fill_(127)
    b = dm.dmuon_mxfp4_empty(32, k)
    b[0].random_(0, 256, generator=gen)
    b[1].fill_(127)
    d, e = torch.zeros((ROWS, 32), device="cuda"), torch.zeros((last, 32), device="cuda")
    handle.mxfp4_gemm(q, b, d, k)
    handle.mxfp4_gemm(p, b, e, k)
    assert torch.equal(d[ROWS - last:], e)
    assert handle.status()[0] == 0
