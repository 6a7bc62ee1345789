"""TinyMLP blocks trained in MXFP4: every projection's three products take
4-bit operands, the norms around a block are fused with its gate and residual
scale, matrices are updated by dmuon_step and vectors by dmuon_adamw_step.

    python examples/train_tinymlp_mxfp4.py --steps 60

Block l, on rows h (bf16):
    f = down(silu(gate h) * (up h))
    y' = res_scale * y + block_gate * rms(f) * post_w,   h' = rms(y') * pre_w
Synthetic data: a fixed random linear map of random rows is to be learned.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import newton_schulz_nesterov_gb300 as dm  # noqa: E402

MATRICES = ("gate", "up", "down")
VECTORS = ("post_w", "pre_w", "block_gate", "res_scale")


class Mx:
    """An r x c matrix in MXFP4 along its rows and, transposed, along its columns."""

    def __init__(self, h, r, c):
        self.h, self.k = h, c
        self.rows, self.cols = dm.dmuon_mxfp4_empty(r, c), dm.dmuon_mxfp4_empty(c, r)

    def set(self, src, noise=None, scale="floor"):
        self.h.mxfp4_quantize(src, self.rows, self.cols, noise=noise, scale=scale)
        return self


class Block:
    def __init__(self, h, d, ff, rows, gen):
        def rand(*shape):
            return torch.randn(*shape, device="cuda", generator=gen)

        def act(width):
            return torch.empty((rows, width), dtype=torch.bfloat16, device="cuda")
        self.h, self.d, self.ff, self.n = h, d, ff, rows
        self.p = dict(gate=rand(ff, d) / d ** 0.5, up=rand(ff, d) / d ** 0.5, down=rand(d, ff) / ff ** 0.5,
                      post_w=torch.ones(d, device="cuda"), pre_w=torch.ones(d, device="cuda"),
                      block_gate=torch.full((1, d), 0.5, device="cuda"), res_scale=torch.ones(d, device="cuda"))
        self.grad = {k: torch.zeros_like(t) for k, t in self.p.items()}
        self.sums = {k: torch.empty_like(self.p[k]) for k in VECTORS}  # of one micro-batch
        self.q = {k: Mx(h, *self.p[k].shape) for k in MATRICES}
        self.q_h, self.q_a = Mx(h, rows, d), Mx(h, rows, ff)
        self.q_df, self.q_dg, self.q_du = Mx(h, rows, d), Mx(h, rows, ff), Mx(h, rows, ff)
        self.g, self.u, self.da, self.f, self.y, self.out = act(ff), act(ff), act(ff), act(d), act(d), act(d)
        self.dx, self.df, self.dh = act(d), act(d), act(d)
        self.rstd = torch.empty((2, rows), device="cuda")
        self.requantize()

    def requantize(self):
        for k in MATRICES:
            self.q[k].set(self.p[k])

    def product(self, a, b, out, k, beta=0.0):
        self.h.mxfp4_gemm(a, b, out, k, beta=beta)

    def forward(self, y, h):
        p, q = self.p, self.q
        self.x = y
        self.q_h.set(h)
        self.product(self.q_h.rows, q["gate"].rows, self.g, self.d)
        self.product(self.q_h.rows, q["up"].rows, self.u, self.d)
        a = torch.nn.functional.silu(self.g) * self.u
        self.q_a.set(a)
        self.product(self.q_a.rows, q["down"].rows, self.f, self.ff)
        self.h.block_norm_forward(y, self.f, p["post_w"], p["pre_w"], self.y, self.out, self.rstd, gate=p["block_gate"],
                                  res_scale=p["res_scale"])
        return self.y, self.out

    def backward(self, dy, dh, noise):
        """From the gradients of y' (None = 0) and h' to those of y and h; the
        parameters' are added to self.grad."""
        p, q, s, grad = self.p, self.q, self.sums, self.grad
        self.h.block_norm_backward(dy, dh, self.x, self.f, self.y, p["post_w"], p["pre_w"], self.rstd, self.dx, self.df,
                                   s["post_w"], s["pre_w"], gate=p["block_gate"], d_gate=s["block_gate"],
                                   res_scale=p["res_scale"], d_res_scale=s["res_scale"])
        for k in VECTORS:
            grad[k] += s[k]
        self.q_df.set(self.df, noise(self.df), "ceil")  # output gradients: stochastic, no saturation
        self.product(self.q_df.cols, self.q_a.cols, grad["down"], self.n, beta=1.0)
        self.product(self.q_df.rows, q["down"].cols, self.da, self.d)
        sig = torch.sigmoid(self.g)
        dg = self.da * self.u * sig * (1 + self.g * (1 - sig))
        du = self.da * self.g * sig
        self.q_dg.set(dg, noise(dg), "ceil")
        self.q_du.set(du, noise(du), "ceil")
        self.product(self.q_dg.cols, self.q_h.cols, grad["gate"], self.n, beta=1.0)
        self.product(self.q_du.cols, self.q_h.cols, grad["up"], self.n, beta=1.0)
        self.product(self.q_dg.rows, q["gate"].cols, self.dh, self.ff)
        self.product(self.q_du.rows, q["up"].cols, self.dh, self.ff, beta=1.0)
        return self.dx, self.dh


def train(steps=60, d=128, ff=512, layers=4, rows=512, micro=2, lr=0.02, adam_lr=0.01, seed=0):
    """Losses of `steps` steps of `micro` micro-batches of `rows` rows each."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    data = torch.randn(micro, rows, d, device="cuda", generator=gen)
    target = data @ (torch.randn(d, d, device="cuda", generator=gen) / d ** 0.5)

    def noise(t):
        return torch.randint(0, 256, t.shape, dtype=torch.uint8, device="cuda", generator=gen)

    losses = []
    with dm.Handle(0) as h:
        blocks = [Block(h, d, ff, rows, gen) for _ in range(layers)]
        params = [b.p[k] for b in blocks for k in MATRICES]
        grads = [b.grad[k] for b in blocks for k in MATRICES]
        momentum = [torch.zeros_like(t) for t in params]
        vec = [b.p[k] for b in blocks for k in VECTORS]
        vec_grad = [b.grad[k] for b in blocks for k in VECTORS]
        m, v = [torch.zeros_like(t) for t in vec], [torch.zeros_like(t) for t in vec]
        for step in range(1, steps + 1):
            for g in grads + vec_grad:
                g.zero_()
            loss = torch.zeros((), device="cuda")
            for i in range(micro):
                y = out = data[i].to(torch.bfloat16)
                for b in blocks:
                    y, out = b.forward(y, out)
                diff = out.float() - target[i]
                loss += diff.square().mean() / micro
                dy, dh = None, (diff * (2.0 / (diff.numel() * micro))).to(torch.bfloat16)
                for b in reversed(blocks):
                    dy, dh = b.backward(dy, dh, noise)
            h.step(params, grads, momentum, lr=lr, mu=0.95, ns_steps=5)
            dm.dmuon_adamw_step(h.h, vec, vec_grad, m, v, lr=adam_lr, weight_decay=0.0, step=step)
            for b in blocks:
                b.requantize()
            losses.append(loss)
        code, _ = h.status(len(params))
        if code != 0:
            raise RuntimeError(dm.dmuon_error_string(code))
    return [float(x) for x in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--d", type=int, default=128)
    ap.add_argument("--ff", type=int, default=512)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--rows", type=int, default=512)
    args = ap.parse_args()
    for i, x in enumerate(train(args.steps, args.d, args.ff, args.layers, args.rows)):
        if i % 10 == 0 or i + 1 == args.steps:
            print("step %4d  loss %.4f" % (i + 1, x))
