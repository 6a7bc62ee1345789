"""The training example: all operators together, with the optimiser.

A block's forward and backward are held against automatic differentiation in
fp32 in which every product takes the values that its 4-bit operands stand for
(read back from them).  What is left is bf16 storage of activations and their
gradients: 2^-6 of each result as a whole (2-norm).  Every quantised gradient
is held against the fp32 gradient in its place: stochastic rounding to a grid
of steps 1/2 (below 2), 1 and 2 (from 4) with a block's largest between 3 and 6
has an error of 0.15 to 0.2 of a normal vector, the bar is 1/4; a wrong
operand, transpose or factor gives 1 or more.
"""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_tinymlp_mxfp4.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    spec = importlib.util.spec_from_file_location("train_tinymlp_mxfp4", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def off(got, want):
    return float((got.float() - want).norm() / want.norm())


class Product(torch.autograd.Function):
    """x w^T; every operand by the values of its quantised form: xr, xc of x
    along rows and (transposed) columns, wr, wc of w, gr, gc of the gradient."""

    @staticmethod
    def forward(ctx, x, w, xr, xc, wr, wc, gr, gc):
        ctx.save_for_backward(xc, wc, gr, gc)
        return xr @ wr.T

    @staticmethod
    def backward(ctx, g):
        xc, wc, gr, gc = ctx.saved_tensors
        assert off(gr, g) < 0.25 and off(gc.T, g) < 0.25
        return gr @ wc.T, gc @ xc.T, None, None, None, None, None, None


@pytest.mark.parametrize("rows,d,ff", [(256, 128, 512), (77, 96, 333)])
def test_block_gradients(example, rows, d, ff):
    gen = torch.Generator(device="cuda").manual_seed(rows)

    def rand(*s):
        return torch.randn(*s, device="cuda", generator=gen)

    def noise(t):
        return torch.randint(0, 256, t.shape, dtype=torch.uint8, device="cuda", generator=gen)

    with dm.Handle(0) as h:
        b = example.Block(h, d, ff, rows, gen)
        for k in example.VECTORS:
            b.p[k] += 0.3 * rand(*b.p[k].shape)
        y0, h0 = rand(rows, d).bfloat16(), rand(rows, d).bfloat16()
        y, out = b.forward(y0, h0)
        dy, dh = rand(rows, d).bfloat16(), rand(rows, d).bfloat16()
        dx, dh0 = b.backward(dy, dh, noise)

        def value(q, r, c):
            t = torch.empty((r, c), device="cuda")
            h.mxfp4_dequantize(q, t)
            return t

        def both(mx, r, c):
            return value(mx.rows, r, c), value(mx.cols, c, r)

        def product(x, name, q_x, q_g):
            r, c = b.p[name].shape
            return Product.apply(x, leaves[name], *both(q_x, rows, c), *both(b.q[name], r, c), *both(q_g, rows, r))
        leaves = {k: t.clone().requires_grad_() for k, t in b.p.items()}
        x, hh = y0.float().requires_grad_(), h0.float().requires_grad_()
        g, u = product(hh, "gate", b.q_h, b.q_dg), product(hh, "up", b.q_h, b.q_du)
        f = product(torch.nn.functional.silu(g) * u, "down", b.q_a, b.q_df)

        def rms(t):
            return t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6)
        y1 = leaves["res_scale"] * x + leaves["block_gate"] * rms(f) * leaves["post_w"]
        out1 = rms(y1) * leaves["pre_w"]
        torch.autograd.backward([y1, out1], [dy.float(), dh.float()])

        assert off(y, y1.detach()) < 2 ** -6 and off(out, out1.detach()) < 2 ** -6
        for k in leaves:
            assert off(b.grad[k], leaves[k].grad) < 2 ** -6, k
        assert off(dx, x.grad) < 2 ** -6 and off(dh0, hh.grad) < 2 ** -6
        assert h.status()[0] == 0


def test_training_learns(example):
    losses = example.train(steps=40)
    assert all(x == x for x in losses)
    # Rows and targets of unit variance: 2 at first, 1 with no more than a
    # small output; below that the map has been learned in part.
    assert 1.5 < losses[0] < 2.5
    assert losses[-1] < 0.9


def test_odd_sizes_train(example):
    losses = example.train(steps=3, d=97, ff=301, layers=2, rows=61)
    assert all(0 < x < 4 for x in losses)
