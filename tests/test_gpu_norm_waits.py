"""Norms of rows that a cluster of CTAs holds, and their bounded waits: a short
limit is reported and leaves complete results, and what another call of the
handle left in the status has no say in them.

More rows than the device holds clusters (76 of two CTAs, fewer of four and
eight), so that a cluster walks several."""
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TIMEOUT = -6


@pytest.fixture
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    with dm.Handle(0) as h:
        yield h


class Norms:
    def __init__(self, h, rows, cols, dtype):
        gen = torch.Generator(device="cuda").manual_seed(rows + cols)

        def act():
            return torch.randn(rows, cols, device="cuda", generator=gen).to(DT[dtype])
        self.h = h
        self.x, self.f, self.dy, self.dh = act(), act(), act(), act()
        self.w, self.v, self.s = (torch.rand(cols, device="cuda", generator=gen) + 0.5 for _ in range(3))
        self.y, self.out, self.dx, self.df = (torch.empty_like(self.x) for _ in range(4))
        self.rstd, self.sums = torch.empty((2, rows), device="cuda"), torch.empty((3, cols), device="cuda")

    def __call__(self):
        results = [self.y, self.out, self.rstd, self.dx, self.df, self.sums]
        for t in results:
            t.fill_(7.0)
        self.h.block_norm_forward(self.x, self.f, self.w, self.v, self.y, self.out, self.rstd, res_scale=self.s)
        self.h.block_norm_backward(self.dy, self.dh, self.x, self.f, self.y, self.w, self.v, self.rstd, self.dx, self.df,
                                   self.sums[0], self.sums[1], res_scale=self.s, d_res_scale=self.sums[2])
        return [t.clone() for t in results]


SHAPES = [(500, 4104), (500, 9000), (400, 9001), (300, 16392), (200, 20011), (150, 32768)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_short_limit(handle, rows, cols, dtype):
    run = Norms(handle, rows, cols, dtype)
    want = run()
    assert handle.status()[0] == 0
    for _ in range(5):
        dm.dmuon_set_wait_timeout(handle.h, 1)
        got = run()
        assert handle.status()[0] in (0, TIMEOUT)
        dm.dmuon_set_wait_timeout(handle.h, 0)
        again = run()
        assert handle.status()[0] == 0
        for a, b, c in zip(got, again, want):
            assert torch.equal(a, c) and torch.equal(b, c)


@pytest.mark.parametrize("rows,cols", SHAPES[1::2])
def test_after_another_call_timed_out(handle, rows, cols):
    run = Norms(handle, rows, cols, "bf16")
    want = run()
    assert handle.status()[0] == 0
    a = dm.dmuon_mxfp4_empty(2048, 16384)
    handle.mxfp4_quantize(torch.randn((2048, 16384), device="cuda"), by_rows=a)
    out = torch.empty((2048, 2048), device="cuda")
    dm.dmuon_set_wait_timeout(handle.h, 1)
    handle.mxfp4_gemm(a, a, out, 16384)
    dm.dmuon_set_wait_timeout(handle.h, 0)
    for got, ref in zip(run(), want):
        assert torch.equal(got, ref)
    assert handle.status()[0] == TIMEOUT  # the product's, read only now
    assert handle.status()[0] == 0
