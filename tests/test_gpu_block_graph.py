"""A captured graph of the operators gives the same bits as the calls, also
after the handle's workspace has grown past what the graph was captured with."""
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402

pytestmark = pytest.mark.gpu


class Run:
    """Norm, both quantisations, product and backward on one set of buffers."""

    def __init__(self, h, rows, cols, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def act(random=False):
            t = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
            return t.normal_(generator=gen) if random else t
        self.h, self.rows, self.cols = h, rows, cols
        self.x, self.f, self.dy, self.dh = (act(True) for _ in range(4))
        self.y, self.out, self.dx, self.df = (act() for _ in range(4))
        self.w = torch.rand(cols, device="cuda", generator=gen) + 0.5
        self.gate = torch.rand((4, cols), device="cuda", generator=gen)
        self.rstd = torch.zeros((2, rows), device="cuda")
        self.sums = [torch.zeros_like(self.w) for _ in range(3)] + [torch.zeros_like(self.gate)]
        self.q = dm.dmuon_mxfp4_empty(rows, cols), dm.dmuon_mxfp4_empty(cols, rows)
        self.prod = torch.zeros((cols, cols), device="cuda")

    def results(self):
        return [self.y, self.out, self.rstd, self.dx, self.df, self.prod, *self.q[0], *self.q[1], *self.sums]

    def __call__(self):
        h, per = self.h, -(-self.rows // 4)
        h.block_norm_forward(self.x, self.f, self.w, self.w, self.y, self.out, self.rstd, gate=self.gate, rows_per_gate=per,
                             res_scale=self.w)
        h.mxfp4_quantize(self.out, *self.q)
        h.mxfp4_gemm(self.q[1], self.q[1], self.prod, self.rows)
        h.block_norm_backward(self.dy, self.dh, self.x, self.f, self.y, self.w, self.w, self.rstd, self.dx, self.df, self.sums[0],
                              self.sums[1], gate=self.gate, d_gate=self.sums[3], rows_per_gate=per, res_scale=self.w,
                              d_res_scale=self.sums[2])


def test_graph_outlives_workspace_growth():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    with dm.Handle(0) as h:
        small, large = Run(h, 300, 264, 1), Run(h, 2500, 1111, 2)
        small()
        torch.cuda.synchronize()
        want = [t.clone() for t in small.results()]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            small()
        with pytest.raises(dm.DmuonError), torch.cuda.graph(torch.cuda.CUDAGraph()):
            large()  # its workspace would have to grow under capture
        large()
        torch.cuda.synchronize()
        for t in small.results():
            t.zero_()
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip(small.results(), want):
            assert torch.equal(got, ref)
        assert h.status()[0] == 0
