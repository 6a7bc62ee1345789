"""TinyMLP blocks trained in MXFP8 with dropout: norms write the 8-bit operand of
the projection behind them, projections have bias, activation and the sum over
micro-batches in their epilogue, gradients leave the activation's backward in 8 bits
for both gradient products; matrices are updated by dmuon_step and vectors by
dmuon_adamw_step.

    python examples/train_tinymlp_mxfp8.py --steps 60

Block l, on the residual stream y and the block before's output f (bf16):
    y' = y + dropout(f),  h = rms(y') * norm_w,  f' = down(gelu(up h + up_b)) + down_b
Synthetic data: a fixed random linear map of random rows is to be learned from the
last norm's output.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import newton_schulz_nesterov_gb300 as dm  # noqa: E402

MATRICES = ("up", "down")
VECTORS = ("norm_w", "up_b", "down_b")


def both(r, c):
    """An r x c matrix in MXFP8 along its rows and, transposed, along its columns."""
    return dm.dmuon_mxfp8_empty(r, c), dm.dmuon_mxfp8_empty(c, r)


class Norm:
    """y' = y + dropout(f) and h = rms(y') * w, in bf16 and, by rows, in MXFP8."""

    def __init__(self, h, d, rows, p, seed):
        def act():
            return torch.empty((rows, d), dtype=torch.bfloat16, device="cuda")
        self.h, self.drop = h, dict(p=p, seed=seed)
        self.w = torch.ones(d, device="cuda")
        self.y, self.out, self.dx, self.df, self.rstd = act(), act(), act(), act(), torch.empty(rows, device="cuda")
        self.q, self.d_w = dm.dmuon_mxfp8_empty(rows, d), torch.empty(d, device="cuda")

    def forward(self, y, f, offset):
        self.drop["offset"] = offset  # another mask for every use
        if f is None:  # the first block's: nothing is added
            y, f, p = None, y, 0.0
        else:
            p = self.drop["p"]
        self.used = dict(self.drop, p=p)
        self.h.add_norm_forward(y, f, self.w, self.y, self.rstd, out=self.out, q=self.q, **self.used)
        return self.y

    def backward(self, dy, dh):
        """Gradients of y and f."""
        self.h.add_norm_backward(dy, dh, self.y, self.w, self.rstd, self.dx, self.df, self.d_w, **self.used)
        return self.dx, self.df


class Block:
    def __init__(self, h, d, ff, rows, p, seed, gen):
        def act(width):
            return torch.empty((rows, width), dtype=torch.bfloat16, device="cuda")
        self.h, self.d, self.ff, self.n = h, d, ff, rows
        self.norm = Norm(h, d, rows, p, seed)
        self.p = dict(up=torch.randn(ff, d, device="cuda", generator=gen) / d ** 0.5,
                      down=torch.randn(d, ff, device="cuda", generator=gen) / ff ** 0.5,
                      norm_w=self.norm.w, up_b=torch.zeros(ff, device="cuda"), down_b=torch.zeros(d, device="cuda"))
        self.grad = {k: torch.zeros_like(t) for k, t in self.p.items()}
        self.sums = {k: torch.empty_like(self.p[k]) for k in ("up_b", "down_b")}
        self.q = {"up": both(ff, d), "down": both(d, ff)}
        self.pre, self.a, self.f, self.da, self.dh = act(ff), act(ff), act(d), act(ff), act(d)
        self.q_a, self.q_h_cols = both(rows, ff), dm.dmuon_mxfp8_empty(d, rows)
        self.q_df, self.q_dz = both(rows, d), both(rows, ff)
        self.requantize()

    def requantize(self):
        for k in MATRICES:
            self.h.mxfp8_quantize(self.p[k], *self.q[k])

    def forward(self, y, f, offset):
        h, p = self.h, self.p
        y = self.norm.forward(y, f, offset)
        h.mx_linear(self.norm.q, self.q["up"][0], self.a, self.d, bias=p["up_b"], act="gelu_tanh", pre=self.pre)
        h.mxfp8_quantize(self.a, *self.q_a)
        h.mx_linear(self.q_a[0], self.q["down"][0], self.f, self.ff, bias=p["down_b"])
        return y, self.f

    def backward(self, dy, df):
        """From the gradients of y' and f' to those of y and f; the parameters' are added to self.grad."""
        h, s, g = self.h, self.sums, self.grad
        h.act_backward(df, None, "none", d_bias=s["down_b"], by_rows=self.q_df[0], by_cols=self.q_df[1], scale="ceil")
        h.mx_linear(self.q_df[1], self.q_a[1], g["down"], self.n, residual=g["down"])
        h.mx_linear(self.q_df[0], self.q["down"][1], self.da, self.d)
        h.act_backward(self.da, self.pre, "gelu_tanh", d_bias=s["up_b"], by_rows=self.q_dz[0], by_cols=self.q_dz[1], scale="ceil")
        h.mxfp8_quantize(self.norm.out, by_cols=self.q_h_cols)
        h.mx_linear(self.q_dz[1], self.q_h_cols, g["up"], self.n, residual=g["up"])
        h.mx_linear(self.q_dz[0], self.q["up"][1], self.dh, self.ff)
        dx, df = self.norm.backward(dy, self.dh)
        g["norm_w"] += self.norm.d_w
        for k in ("up_b", "down_b"):
            g[k] += s[k]
        return dx, df


def train(steps=60, d=128, ff=512, layers=4, rows=512, micro=2, p=0.05, lr=0.02, adam_lr=0.01, seed=0):
    """Losses of `steps` steps of `micro` micro-batches of `rows` rows each."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    data = torch.randn(micro, rows, d, device="cuda", generator=gen)
    target = data @ (torch.randn(d, d, device="cuda", generator=gen) / d ** 0.5)
    losses = []
    with dm.Handle(0) as h:
        blocks = [Block(h, d, ff, rows, p, 100 + i, gen) for i in range(layers)]
        last = Norm(h, d, rows, p, 99)
        last_grad = torch.zeros(d, device="cuda")
        params = [b.p[k] for b in blocks for k in MATRICES]
        grads = [b.grad[k] for b in blocks for k in MATRICES]
        momentum = [torch.zeros_like(t) for t in params]
        vec = [b.p[k] for b in blocks for k in VECTORS] + [last.w]
        vec_grad = [b.grad[k] for b in blocks for k in VECTORS] + [last_grad]
        m, v = [torch.zeros_like(t) for t in vec], [torch.zeros_like(t) for t in vec]
        for step in range(1, steps + 1):
            for g in grads + vec_grad:
                g.zero_()
            loss = torch.zeros((), device="cuda")
            for i in range(micro):
                y, f, offset = data[i].to(torch.bfloat16), None, step * micro + i
                for b in blocks:
                    y, f = b.forward(y, f, offset)
                last.forward(y, f, offset)
                diff = last.out.float() - target[i]
                loss += diff.square().mean() / micro
                dy, df = last.backward(None, (diff * (2.0 / (diff.numel() * micro))).to(torch.bfloat16))
                last_grad += last.d_w
                for b in reversed(blocks):
                    dy, df = b.backward(dy, df)
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
    ap.add_argument("--p", type=float, default=0.05)
    args = ap.parse_args()
    for i, x in enumerate(train(args.steps, args.d, args.ff, args.layers, args.rows, p=args.p)):
        if i % 10 == 0 or i + 1 == args.steps:
            print("step %4d  loss %.4f" % (i + 1, x))
