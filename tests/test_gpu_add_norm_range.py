"""The residual norm's backward over rows of any size, against fp64.

The formula knows a row only as yn = y * rstd, which is of size one whatever y is, so
the bars are those of rows of size one: gradients 2^-17 of the terms' magnitudes, d_w
2^-20 and a rounding a row.  fp32 reaches sizes from 1e-20 to 1e18 with yn, rstd and
every gradient normal; rstd is given, as the forward of another program may have left
it (eps = 0, and a row of zeros under an eps of 1e-30).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402
from oracle import projection as op  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
SIZES = np.array([1e-20, 1e-14, 1e-13, 1e-9, 1.0, 1e9, 1e13, 1e14, 1e15, 1e17, 1e18, 0.0])
SEED, OFFSET = 77, 3


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    h = dm.Handle(0)
    yield h
    h.close()


def on_gpu(t, odd):
    if not odd:
        return t.cuda()
    v = torch.zeros((t.shape[0], t.shape[1] + 5), dtype=t.dtype, device="cuda")[:, 1:1 + t.shape[1]]
    v.copy_(t)
    return v


def f64(t):
    return t.detach().cpu().double().numpy()


# A part of a warp, a warp, up to eight warps, sixteen, 32 columns a thread, longer than a CTA holds.
@pytest.mark.parametrize("cols", [100, 512, 1111, 4096, 8192, 9001, 16384, 20001])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("with_dy,p,odd", [(False, 0.0, False), (True, 0.25, True)])
def test_backward(handle, cols, dtype, with_dy, p, odd):
    rows = len(SIZES)
    g = torch.Generator().manual_seed(cols)
    y = torch.randn((rows, cols), generator=g, dtype=torch.float64) * torch.from_numpy(SIZES)[:, None]
    y = y.to(DT[dtype])
    square = y.double().square().mean(1).numpy()
    rstd = torch.from_numpy(1 / np.sqrt(np.where(square > 0, square, 1e-30))).float()
    # dh lies along y, so that the term that is taken away is as large as what it is taken from.
    dh = (y.double() * rstd.double()[:, None] + 0.1 * torch.randn((rows, cols), generator=g)).to(DT[dtype])
    dy = (torch.randn((rows, cols), generator=g) * rstd[:, None]).to(DT[dtype]) if with_dy else None
    w = 1 + 0.1 * torch.randn(cols, generator=g)
    dx, df = on_gpu(torch.zeros_like(y), odd), on_gpu(torch.zeros_like(y), odd)
    dw = torch.empty(cols, device="cuda")
    handle.add_norm_backward(on_gpu(dy, odd) if with_dy else None, on_gpu(dh, odd), on_gpu(y, odd), w.cuda(), rstd.cuda(), dx, df, dw, p=p,
                             seed=SEED, offset=OFFSET)
    keep = op.factors(rows, cols, p, SEED, OFFSET)
    d64, g64, y64, w64, r64 = f64(dy) if with_dy else np.zeros(y.shape), f64(dh), f64(y), f64(w), f64(rstd)
    gx, gf, gw = op.add_norm_backward(d64, g64, y64, w64, r64, keep)
    yn = y64 * r64[:, None]
    terms = np.abs(d64) + r64[:, None] * (np.abs(g64 * w64) + np.abs(yn) * np.abs(g64 * w64 * yn).mean(1, keepdims=True))
    bar, u = 2.0 ** -17 * terms, HALF[dtype]
    for got, want, scale in ((dx, gx, 1.0), (df, gf, keep)):
        off = np.abs(f64(got) - want)
        late = ~(off <= bar * scale * (1 + u) + u * np.abs(want))
        assert not late.any(), "rows of size %s" % SIZES[late.any(1)]
    assert (np.abs(f64(dw) - gw) <= (2.0 ** -20 + rows * 2.0 ** -23) * np.abs(g64 * yn).sum(0)).all()
    assert handle.status()[0] == 0
