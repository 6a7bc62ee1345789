"""The operators around an 8-bit projection together: a block forward and backward
as examples/train_tinymlp_mxfp8.py runs it, every result against fp64 from what the
run itself had before it; the same bits from a captured graph, on another stream and
beside another handle; the example's steps.

Bars: z as in test_gpu_mx_linear.py; an activation, a slope and a norm pass errors of
2^-16 of their terms on (those tests have the exact bars) and round to bf16, 2^-8.
"""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402
from oracle import mxfp8 as ox  # noqa: E402
from oracle import projection as op  # noqa: E402

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
import train_tinymlp_mxfp8 as ex  # noqa: E402

U = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()


def f64(t):
    return t.detach().cpu().double().numpy()


def read(h, q, rows, k):
    out = torch.empty((rows, k), device="cuda")
    h.mxfp8_dequantize(q, out)
    return f64(out)


def near(got, want, terms, blocks=1):
    """Within one rounding to bf16 and 33 blocks 2^-23 + 2^-16 of the terms."""
    assert (np.abs(f64(got) - want) <= U * np.abs(want) + (33 * blocks * 2.0 ** -23 + 2.0 ** -16) * terms).all()


class Run:
    def __init__(self, h, rows, d, ff, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.h, self.rows, self.d, self.ff = h, rows, d, ff
        self.b = ex.Block(h, d, ff, rows, 0.1, 17, gen)
        for k in ("norm_w", "up_b", "down_b"):
            self.b.p[k].add_(0.2 * torch.randn(self.b.p[k].shape, device="cuda", generator=gen))
        self.y, self.f, self.dy, self.df = (torch.randn(rows, d, device="cuda", generator=gen).bfloat16() for _ in range(4))

    def __call__(self):
        for g in self.b.grad.values():
            g.zero_()
        self.b.forward(self.y, self.f, 5)
        return self.b.backward(self.dy, self.df)

    def results(self):
        b, n = self.b, self.b.norm
        return [n.y, n.out, n.rstd, b.pre, b.a, b.f, b.da, b.dh, n.dx, n.df, *b.grad.values(), *n.q, *b.q_a[0], *b.q_a[1], *b.q_df[0],
                *b.q_df[1], *b.q_dz[0], *b.q_dz[1]]


@pytest.mark.parametrize("rows,d,ff", [(300, 256, 512), (77, 132, 300), (1, 64, 96), (513, 1001, 260)])
def test_block_against_fp64(rows, d, ff):
    with dm.Handle(0) as h:
        run = Run(h, rows, d, ff, rows)
        run()
        b, n = run.b, run.b.norm
        keep = op.factors(rows, d, 0.1, 17, 5)
        y, hh, _ = op.add_norm_forward(f64(run.y), f64(run.f), f64(n.w), keep)
        near(n.y, y, np.abs(f64(run.y)) + np.abs(f64(run.f) * keep))
        near(n.out, hh, np.abs(hh) + 2.0 ** -6 * np.abs(f64(n.w)))
        up, down = read(h, b.q["up"][0], ff, d), read(h, b.q["down"][0], d, ff)
        blocks = -(-d // 32)
        qh = read(h, n.q, rows, d)
        z, terms = qh @ up.T + f64(b.p["up_b"]), np.abs(qh) @ np.abs(up).T + np.abs(f64(b.p["up_b"]))
        near(b.pre, z, terms, blocks)
        near(b.a, op.activation(z, "gelu_tanh"), 1.13 * terms, blocks)
        for got, want in zip((*b.q_a[0], *b.q_a[1]), (*ox.pack(*ox.quantize(f64(b.a))), *ox.pack(*ox.quantize(f64(b.a).T)))):
            assert np.array_equal(got.cpu().numpy(), want)
        qa = read(h, b.q_a[0], rows, ff)
        near(b.f, qa @ down.T + f64(b.p["down_b"]), np.abs(qa) @ np.abs(down).T + np.abs(f64(b.p["down_b"])), -(-ff // 32))
        # backward
        for got, want in zip((*b.q_df[0], *b.q_df[1]), (*ox.pack(*ox.quantize(f64(run.df), "ceil")), *ox.pack(*ox.quantize(f64(run.df).T, "ceil")))):
            assert np.array_equal(got.cpu().numpy(), want)
        assert (np.abs(f64(b.grad["down_b"]) - f64(run.df).sum(0)) <= rows * 2.0 ** -23 * np.abs(f64(run.df)).sum(0)).all()
        g, a = read(h, b.q_df[1], d, rows), read(h, b.q_a[1], ff, rows)
        bar = (33 * -(-rows // 32) * 2.0 ** -23 + 2.0 ** -22) * (np.abs(g) @ np.abs(a).T)
        assert (np.abs(f64(b.grad["down"]) - g @ a.T) <= bar).all()
        g, w = read(h, b.q_df[0], rows, d), read(h, b.q["down"][1], ff, d)
        near(b.da, g @ w.T, np.abs(g) @ np.abs(w).T, blocks)
        dz = f64(b.da) * op.slope(f64(b.pre), "gelu_tanh")
        qz = read(h, b.q_dz[0], rows, ff)
        top = np.abs(dz).max(1, keepdims=True)
        assert (np.abs(qz - dz) <= (2.0 ** -4 + 2.0 ** -16) * np.abs(dz) + 2.0 ** -16 * top).all()
        assert (np.abs(f64(b.grad["up_b"]) - dz.sum(0)) <= (rows * 2.0 ** -23 + 2.0 ** -18) * np.abs(dz).sum(0) + 2.0 ** -20 * np.abs(f64(b.da)).sum(0)).all()
        g, hc = read(h, b.q_dz[1], ff, rows), read(h, b.q_h_cols, d, rows)
        bar = (33 * -(-rows // 32) * 2.0 ** -23 + 2.0 ** -22) * (np.abs(g) @ np.abs(hc).T)
        assert (np.abs(f64(b.grad["up"]) - g @ hc.T) <= bar).all()
        w = read(h, b.q["up"][1], d, ff)
        near(b.dh, qz @ w.T, np.abs(qz) @ np.abs(w).T, -(-ff // 32))
        gx, gf, gw = op.add_norm_backward(f64(run.dy), f64(b.dh), f64(n.y), f64(n.w), f64(n.rstd), keep)
        into = np.abs(f64(n.rstd))[:, None] * np.abs(f64(b.dh) * f64(n.w))
        terms = np.abs(f64(run.dy)) + into + np.abs(f64(n.y) * f64(n.rstd)[:, None]) * into.mean(1, keepdims=True) * 4
        near(n.dx, gx, terms)
        near(n.df, gf, terms * keep)
        assert (np.abs(f64(b.grad["norm_w"]) - gw) <= (rows * 2.0 ** -23 + 2.0 ** -18) * np.abs(f64(b.dh) * f64(n.y) * f64(n.rstd)[:, None]).sum(0)).all()
        assert h.status()[0] == 0


def test_graph_stream_and_other_handle():
    with dm.Handle(0) as h, dm.Handle(0) as h2:
        run, large, beside = Run(h, 300, 256, 512, 1), Run(h, 2500, 1111, 700, 2), Run(h2, 300, 256, 512, 1)
        run()
        torch.cuda.synchronize()
        want = [t.clone() for t in run.results()]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        with pytest.raises(dm.DmuonError), torch.cuda.graph(torch.cuda.CUDAGraph()):
            large()  # its workspace would have to grow under capture
        large()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        for t in run.results():
            t.zero_()
        with torch.cuda.stream(side):  # another handle's work at the same time
            for _ in range(20):
                beside()
        for _ in range(20):
            graph.replay()
        torch.cuda.synchronize()
        for got, other, ref in zip(run.results(), beside.results(), want):
            assert torch.equal(got, ref) and torch.equal(other, ref)
        assert h.status()[0] == 0 and h2.status()[0] == 0


def test_example_runs():
    losses = ex.train(steps=3, d=64, ff=160, layers=2, rows=96, micro=2)
    assert len(losses) == 3 and all(np.isfinite(losses))
