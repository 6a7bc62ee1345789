"""Norms of long rows, several a cluster (a CTA beyond 32768 columns), against
fp64 on the device: the sums' buffers and barriers are used again, the ring is
refilled, chunks of several rows and several chunks a CTA are added up.

Bars as in test_gpu_block_norm.py: with E = (cols / 64 + 64) 2^-24 a value that
is a sum of terms may be off by 8 E times the sum of the terms' sizes, a column
sum by (8 E + (rows + 64) 2^-24) times the sum over rows, stored values by
their type's rounding besides.
"""
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
EPS = 1e-6


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    with dm.Handle(0) as h:
        yield h
    torch.cuda.empty_cache()


def within(got, want, size, e, u, name):
    off = (got.double() - want).abs()
    bar = e * size + u * want.abs()
    assert bool((off <= bar).all()), (name, float((off / bar.clamp_min(1e-300)).max()))


def check(h, rows, cols, dtype, per, odd, dy, d_gate, d_res):
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    one, e = {"generator": gen, "device": "cuda"}, (cols / 64 + 64) * 2.0 ** -24

    def act(random=True):  # odd: one element off, with an odd pitch
        t = torch.zeros((rows, cols + 2 * odd), dtype=DT[dtype], device="cuda")[:, odd:odd + cols]
        if random:
            t.copy_(torch.randn(rows, cols, **one) * torch.exp(0.5 * torch.randn(rows, 1, **one)))
        return t
    x, f, d1, d2 = act(), act(), act() if dy else None, act()
    post, pre, res = (torch.randn(cols, **one) + 1 for _ in range(3))
    gate = torch.randn(-(-rows // per), cols, **one)
    y, out, dx, df = (act(False) for _ in range(4))
    rstd = torch.full((2, rows), 7.0, device="cuda")
    h.block_norm_forward(x, f, post, pre, y, out, rstd, gate=gate, rows_per_gate=per, res_scale=res, eps=EPS)
    sums = torch.full((2, cols), 7.0, device="cuda")
    dg = torch.full_like(gate, 7.0) if d_gate else None
    ds = torch.full_like(res, 7.0) if d_res else None

    def backward():
        h.block_norm_backward(d1, d2, x if d_res else None, f, y, post, pre, rstd, dx, df, sums[0], sums[1], gate=gate, d_gate=dg,
                              rows_per_gate=per, res_scale=res, d_res_scale=ds)
        return [t.clone() for t in (dx, df, sums, dg, ds) if t is not None]
    first = backward()
    assert all(torch.equal(a, b) for a, b in zip(first, backward()))  # the same bits
    assert h.status()[0] == 0

    x6, f6, pw, qw, s6 = (t.double() for t in (x, f, post, pre, res))
    g = gate.double().repeat_interleave(per, 0)[:rows]
    r1 = (f6.square().mean(1, keepdim=True) + EPS).rsqrt()
    n = g * (f6 * r1 * pw)
    wy = s6 * x6 + n
    r2 = (wy.square().mean(1, keepdim=True) + EPS).rsqrt()
    size = (s6 * x6).abs() + n.abs()
    spread = (size * wy.abs()).sum(1, keepdim=True) / wy.square().sum(1, keepdim=True)
    within(y, wy, size, 8 * e, U[dtype], "y")
    within(out, wy * r2 * qw, (size + spread * wy.abs()) * r2 * qw.abs(), 8 * e, U[dtype], "h")
    within(rstd[0], r1[:, 0], r1[:, 0], 8 * e, 0.0, "rstd of f")
    within(rstd[1], r2[:, 0], (r2 * spread.clamp_min(1))[:, 0], 8 * e, 0.0, "rstd of y")
    del wy, n, size

    r1, r2 = rstd[0].double()[:, None], rstd[1].double()[:, None]
    yn, fn, dh = y.double() * r2, f6 * r1, d2.double()
    into = dh * qw
    t = (d1.double() if dy else 0.0) + r2 * (into - yn * (into * yn).mean(1, keepdim=True))
    ts = (d1.double().abs() if dy else 0.0) + r2 * (into.abs() + yn.abs() * (into * yn).abs().mean(1, keepdim=True))
    within(dx, s6 * t, s6.abs() * ts, 8 * e, U[dtype], "dx")
    b, bs = g * t * pw, g.abs() * ts * pw.abs()
    within(df, r1 * (b - fn * (b * fn).mean(1, keepdim=True)), r1 * (bs + fn.abs() * (bs * fn.abs()).mean(1, keepdim=True)),
           8 * e, U[dtype], "df")
    del b, bs
    e_sum = 8 * e + (rows + 64) * 2.0 ** -24
    within(sums[0], (g * t * fn).sum(0), (g.abs() * ts * fn.abs()).sum(0), e_sum, U["f32"], "d_post_w")
    within(sums[1], (dh * yn).sum(0), (dh * yn).abs().sum(0), e_sum, U["f32"], "d_pre_w")
    if d_res:
        within(ds, (t * x6).sum(0), (ts * x6.abs()).sum(0), e_sum, U["f32"], "d_res_scale")
    if d_gate:
        at = torch.arange(rows, device="cuda") // per
        zero = torch.zeros_like(gate, dtype=torch.float64)
        within(dg, zero.index_add(0, at, t * fn * pw), zero.index_add(0, at, ts * (fn * pw).abs()), e_sum, U["f32"], "d_gate")


# Clusters of two, four and eight CTAs in the backward; two and four in the forward.
@pytest.mark.parametrize("rows,cols", [(700, 4112), (701, 8200), (400, 9000), (300, 16400), (150, 32768)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("odd", [0, 1])
def test_clusters(handle, rows, cols, dtype, odd):
    check(handle, rows, cols, dtype, 7, odd, True, True, True)
    check(handle, rows, cols - odd, dtype, rows, odd, False, False, False)


# One CTA a row: chunks of one row (several a CTA), of three, one group.
@pytest.mark.parametrize("per", [1, 7, 1300])
@pytest.mark.parametrize("dtype,odd", [("f32", 0), ("bf16", 1)])
def test_rows_in_passes(handle, per, dtype, odd):
    check(handle, 1300, 32776, dtype, per, odd, True, True, True)
    check(handle, 1300, 32776, dtype, per, odd, False, per == 7, False)
