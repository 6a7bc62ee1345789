"""Products over no rows: out = beta * out, as the gradient of a weight whose
micro-batch or expert had no tokens."""
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
    with dm.Handle(0) as h:
        yield h


@pytest.mark.parametrize("m,n", [(1, 1), (1, 300), (129, 77), (700, 4096)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("beta", [0.0, 1.0, -0.5])
@pytest.mark.parametrize("other_stream", [False, True])
def test_product_over_no_rows(handle, m, n, dtype, beta, other_stream):
    x, g = torch.empty((0, n), dtype=dtype, device="cuda"), torch.empty((0, m), dtype=dtype, device="cuda")
    a, b = dm.dmuon_mxfp4_empty(m, 0), dm.dmuon_mxfp4_empty(n, 0)
    handle.mxfp4_quantize(g, by_cols=a)
    handle.mxfp4_quantize(x, by_cols=b)
    out = torch.randn((m, n), device="cuda").to(dtype)
    want = (out.double() * beta).to(dtype)  # exact for these factors
    if beta == 0:
        out[0, 0] = float("nan")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    handle.mxfp4_gemm(a, b, out, 0, alpha=3.0, beta=beta, stream=s if other_stream else None)
    torch.cuda.synchronize()
    assert handle.status()[0] == 0
    assert torch.equal(out, want)


def test_default_stream_from_another(handle):
    a, b = dm.dmuon_mxfp4_empty(40, 0), dm.dmuon_mxfp4_empty(64, 0)
    out = torch.ones((40, 64), device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        handle.mxfp4_gemm(a, b, out, 0, beta=0.25, stream=torch.cuda.default_stream())
    torch.cuda.synchronize()
    assert (out == 0.25).all()


def test_in_a_graph(handle):
    a, b = dm.dmuon_mxfp4_empty(200, 0), dm.dmuon_mxfp4_empty(64, 0)
    out = torch.ones((200, 64), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        handle.mxfp4_gemm(a, b, out, 0, beta=0.5)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert (out == 0.125).all()


def test_refusals_stay(handle):
    a, b = dm.dmuon_mxfp4_empty(4, 0), dm.dmuon_mxfp4_empty(8, 0)
    out = torch.zeros((4, 8), device="cuda")
    with pytest.raises(ValueError):
        handle.mxfp4_gemm(a, dm.dmuon_mxfp4_empty(8, 64), out, 0)
    with pytest.raises(dm.DmuonError):
        handle.mxfp4_gemm(a, b, out, 0, beta=float("nan"))
    handle.mxfp4_gemm(dm.dmuon_mxfp4_empty(0, 0), b, out[:0], 0)
