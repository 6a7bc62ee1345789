"""Row sums of rows of millions of columns, against fp64.

Values of one size are the worst for a running fp32 sum: the same rounding falls the
same way from one power of two to the next, and 8192 terms of 0.09 are off by 7e-5.
A row's mean of squares is held to 2^-17 whatever the row's length, so rstd to 2^-18 of
it, and the gradients to 2^-17 of their terms, as for short rows.  (Where a sum keeps
what its additions lose, a thread's eight products take eight roundings, the sum over
panels two and the one over 512 threads nine: 19 2^-24.)
"""
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    h = dm.Handle(0)
    yield h
    h.close()


@pytest.mark.parametrize("cols", [20000, 1 << 22, (1 << 24) + 3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("value", [0.3, 1.1])
def test_constant_rows(handle, cols, dtype, value):
    x = torch.full((2, cols), value, device="cuda").to(dtype)
    x[1, ::3] *= -1
    w, y, h, rstd = torch.ones(cols, device="cuda"), torch.empty_like(x), torch.empty_like(x), torch.empty(2, device="cuda")
    handle.add_norm_forward(None, x, w, y, rstd, out=h, eps=0.0)
    x64, u = x.double(), HALF[dtype]
    r64 = x64.square().mean(1).rsqrt()
    assert ((rstd.double() - r64).abs() <= 2.0 ** -18 * r64).all()
    want = x64 * r64[:, None]
    assert ((h.double() - want).abs() <= (2.0 ** -17 * (1 + u) + u) * want.abs()).all()
    df, dw = torch.empty_like(x), torch.empty(cols, device="cuda")
    handle.add_norm_backward(None, h, y, w, rstd, None, df, dw)
    g, yn, r = h.double(), y.double() * rstd.double()[:, None], rstd.double()[:, None]
    mean = (g * yn).mean(1, keepdim=True)
    want = r * (g - yn * mean)
    terms = r * (g.abs() + yn.abs() * (g * yn).abs().mean(1, keepdim=True))
    assert ((df.double() - want).abs() <= 2.0 ** -17 * (1 + u) * terms + u * want.abs()).all()
    assert ((dw.double() - (g * yn).sum(0)).abs() <= 2.0 ** -20 * (g * yn).abs().sum(0)).all()
    assert handle.status()[0] == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_infinite_sum_stays_infinite(handle, dtype):
    """An Inf in a long row: 1 / Inf = 0 takes the other values to 0, as in short rows; a NaN takes them all."""
    for cols in (4096, 20000):
        x = torch.ones((3, cols), device="cuda").to(dtype)
        x[0, 7], x[1, 7] = float("inf"), float("nan")
        y, h, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(3, device="cuda")
        handle.add_norm_forward(None, x, torch.ones(cols, device="cuda"), y, rstd, out=h)
        assert rstd[0] == 0 and torch.isnan(rstd[1]) and torch.isnan(h[0, 7]) and torch.isnan(h[1]).all()
        assert not h[0, :7].any() and not h[0, 8:].any() and torch.isfinite(h[2]).all()
