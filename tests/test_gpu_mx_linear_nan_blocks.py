"""A block of scale byte 255 makes the projections of its row NaN, in both formats and
on every kind of tile, through bias, activation and residual; all others are what they
are without it."""
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    h = dm.Handle(0)
    yield h
    h.close()


# Few rows of A whole and split, 64 and 128 rows, tiles of 128 split and whole, CTA pairs.
@pytest.mark.parametrize("m,n,k", [(1, 200, 96), (3, 500, 4096), (50, 300, 640), (100, 300, 320), (300, 264, 2048), (300, 1000, 100), (2100, 2600, 300)])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh"])
def test_nan_blocks(handle, m, n, k, bits, act):
    gen = torch.Generator(device="cuda").manual_seed(m + n + k)
    quantize, empty = (handle.mxfp8_quantize, dm.dmuon_mxfp8_empty) if bits == 8 else (handle.mxfp4_quantize, dm.dmuon_mxfp4_empty)
    a, b = torch.randn((m, k), device="cuda", generator=gen), torch.randn((n, k), device="cuda", generator=gen)
    bias, res = torch.randn(n, device="cuda", generator=gen), torch.randn((m, n), device="cuda", generator=gen)
    rows, cols = sorted({0, m // 2, m - 1}), sorted({1, n // 2, n - 1})

    def product(a, b):
        qa, qb = empty(m, k), empty(n, k)
        quantize(a, qa)
        quantize(b, qb)
        out, pre = torch.empty((m, n), device="cuda"), torch.empty((m, n), device="cuda")
        handle.mx_linear(qa, qb, out, k, bias=bias, act=act, pre=pre, residual=res, bits=bits)
        return out, pre
    want = product(a, b)
    for bad_rows, bad_cols in (((), cols), (rows, ()), (rows[:1], cols[:1])):
        a2, b2 = a.clone(), b.clone()
        for i, r in enumerate(bad_rows):
            a2[r, (i * 37) % k] = float("inf") if i % 2 else float("nan")
        for i, c in enumerate(bad_cols):
            b2[c, k - 1 - (i * 53) % k] = float("-inf")
        bad = torch.zeros((m, n), dtype=torch.bool, device="cuda")
        bad[list(bad_rows)] = True
        bad[:, list(bad_cols)] = True
        for got, ref in zip(product(a2, b2), want):
            assert torch.equal(torch.isnan(got), bad) and torch.equal(got[~bad], ref[~bad])
    assert handle.status()[0] == 0
