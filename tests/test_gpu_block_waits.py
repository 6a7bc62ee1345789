"""Waits that run out inside the products: the status says so, the kernel ends
with nothing in flight, and the next call is right.

A limit of one nanosecond makes a wait give up unless what it waits for is
there at the first look, so which roles give up differs from run to run; K is
taken short of the ring of stages (every copy is issued before the first wait
can fail), past it, and long.
"""
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402

pytestmark = pytest.mark.gpu

TIMEOUT = -6


@pytest.fixture
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    with dm.Handle(0) as h:
        yield h


def operand(handle, rows, k, seed):
    q = dm.dmuon_mxfp4_empty(rows, k)
    handle.mxfp4_quantize(torch.randn((rows, k), generator=torch.Generator().manual_seed(seed)).cuda(), by_rows=q)
    return q


# One CTA a tile, K split over clusters of 2, 4 and 8, CTA pairs.
@pytest.mark.parametrize("m,n,k", [(1, 30000, 512), (1, 30000, 9000), (300, 600, 300), (300, 600, 1200), (40, 4096, 1024),
                                   (1, 8192, 4096), (1, 4096, 4096), (1, 512, 8192), (200, 512, 8192), (2100, 2600, 200), (2100, 2600, 1300), (2100, 2600, 5000),
                                   (4200, 5000, 1024)])
def test_product(handle, m, n, k):
    a, b = operand(handle, m, k, 1), operand(handle, n, k, 2)
    want, out = (torch.full((m, n), 7.0, device="cuda") for _ in range(2))
    handle.mxfp4_gemm(a, b, want, k)
    assert handle.status()[0] == 0
    for _ in range(12):
        dm.dmuon_set_wait_timeout(handle.h, 1)
        handle.mxfp4_gemm(a, b, out, k)
        late = handle.status()[0]
        assert late in (0, TIMEOUT)
        assert late == TIMEOUT or torch.equal(out, want)
        dm.dmuon_set_wait_timeout(handle.h, 0)
        out.fill_(7.0)
        handle.mxfp4_gemm(a, b, out, k)
        assert handle.status()[0] == 0
        assert torch.equal(out, want)
