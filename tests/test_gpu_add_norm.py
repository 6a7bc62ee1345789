"""Dropout and the residual norm with dropout on the branch, against fp64.

Which elements stay is exact.  y: two roundings of fp32 and the type's.  rstd:
sums of squares of up to 20000 terms, 16 in a row and the rest in a tree of at
most 64 additions, so 2^-18 of it, halved by the root.  h: that and y's own
error.  Codes are those of the fp32 h, bit for bit: h of an fp32 call on the same
values quantised by the oracle.  Gradients: 2^-17 of the terms' magnitudes.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402
from oracle import mxfp8 as ox  # noqa: E402
from oracle import projection as op  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -25}
SEED, OFFSET = 0xFEDCBA9876543210, (5 << 33) + 77


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    h = dm.Handle(0)
    yield h
    h.close()


def buffer(rows, cols, dtype, odd, fill=7.0):
    t = torch.full((rows, cols + (5 if odd else 0)), fill, dtype=dtype, device="cuda")
    return t[:, 1:1 + cols] if odd else t


def on_gpu(t, odd):
    v = buffer(*t.shape, t.dtype, odd)
    v.copy_(t)
    return v


def f64(t):
    return t.detach().cpu().double().numpy()


def untouched(t, cols):
    return t._base is None or ((t._base[:, 0] == 7).all() and (t._base[:, 1 + cols:] == 7).all())


SHAPES = [(1, 1), (3, 7), (1, 4096), (130, 33), (37, 100), (70, 255), (64, 256), (40, 512), (33, 777), (20, 1111), (9, 2061), (600, 4096), (7, 8192),
          (5, 9001), (3, 16384), (3, 16385), (4, 20000)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("p,res,odd", [(0.1, True, False), (0.5, False, True), (0.0, True, True), (0.9, False, False)])
def test_dropout(handle, shape, dtype, p, res, odd):
    rows, cols = shape
    g = torch.Generator().manual_seed(rows + cols)
    x, r = (torch.randn(shape, generator=g).to(DT[dtype]) for _ in range(2))
    out, xd, rd = buffer(rows, cols, DT[dtype], odd), on_gpu(x, odd), on_gpu(r, odd) if res else None
    handle.dropout(xd, out, p, SEED, OFFSET, residual=rd)
    keep = op.factors(rows, cols, p, SEED, OFFSET)
    add = f64(r) if res else 0.0
    want = f64(x) * keep + add
    bar = 2.0 ** -23 * (np.abs(f64(x) * keep) + np.abs(want))
    assert (np.abs(f64(out) - want) <= bar + HALF[dtype] * np.abs(want) + TINY[dtype]).all()
    assert np.array_equal(f64(out)[keep == 0], (np.zeros(shape) + add)[keep == 0])
    assert untouched(out, cols)
    for place in ([xd, rd] if res else [xd]):  # in place
        hold = place.clone()
        handle.dropout(xd, place, p, SEED, OFFSET, residual=rd)
        assert torch.equal(place, out) and untouched(place, cols)
        place.copy_(hold)


def test_dropout_hides_what_it_drops(handle):
    """Inf and NaN that go, go; rows and columns beyond the first tiles have masks of their own."""
    x = torch.full((300, 600), float("inf"), device="cuda")
    x[::2] = float("nan")
    out = torch.empty_like(x)
    handle.dropout(x, out, 0.5, SEED, 1)
    gone = op.factors(300, 600, 0.5, SEED, 1) == 0
    got = f64(out)
    assert not got[gone].any() and not np.isfinite(got[~gone]).any()
    masks = [op.factors(64, 64, 0.5, s, o) for s, o in ((1, 0), (2, 0), (1, 1), (1, 1 << 32), (1 + (1 << 32), 0))]
    one = torch.ones((64, 64), device="cuda")
    for (s, o), m in zip(((1, 0), (2, 0), (1, 1), (1, 1 << 32), (1 + (1 << 32), 0)), masks):
        handle.dropout(one, one.clone(), 0.5, s, o)
        got = torch.empty_like(one)
        handle.dropout(one, got, 0.5, s, o)
        assert np.array_equal(f64(got), m)
    assert all(not np.array_equal(a, b) for i, a in enumerate(masks) for b in masks[:i])


def test_empty_and_refusals(handle):
    x = torch.zeros((8, 64), device="cuda")
    for r, c in ((0, 5), (5, 0)):
        handle.dropout(torch.empty((r, c), device="cuda"), torch.empty((r, c), device="cuda"), 0.5, 1)
    for p in (-0.1, 1.0, 1.5, float("nan"), 0.999999):
        with pytest.raises(dm.DmuonError):
            handle.dropout(x, torch.empty_like(x), p, 1)
    with pytest.raises(ValueError):
        handle.dropout(x, x.half(), 0.5, 1)
    with pytest.raises(ValueError):
        handle.dropout(x, None, 0.5, 1)
    wide = torch.zeros((16, 64), device="cuda")
    with pytest.raises(dm.DmuonError):
        handle.dropout(wide[::2], wide[:8], 0.5, 1)  # the same place, other rows
    w, rstd, y = torch.ones(64, device="cuda"), torch.empty(8, device="cuda"), torch.empty_like(x)
    h, f, q = torch.empty_like(x), torch.zeros_like(x), dm.dmuon_mxfp8_empty(8, 64)
    for bad in (dict(out=None), dict(w=torch.ones(63, device="cuda")), dict(rstd=torch.empty((2, 8), device="cuda")), dict(x=x.half()),
                dict(q=dm.dmuon_mxfp4_empty(8, 64))):
        with pytest.raises(ValueError):
            handle.add_norm_forward(**dict(dict(x=x, f=f, w=w, y=y, rstd=rstd, out=h), **bad))
    for bad in (dict(y=x), dict(out=y), dict(eps=-1.0), dict(p=1.0), dict(out=f), dict(q=(q[0], q[0].view(-1)[:512])), dict(rstd=w[:8])):
        with pytest.raises(dm.DmuonError):
            handle.add_norm_forward(**dict(dict(x=x, f=f, w=w, y=y, rstd=rstd, out=h), **bad))
    dw, df, dx = torch.empty(64, device="cuda"), torch.empty_like(x), torch.empty_like(x)
    for bad in (dict(dh=None), dict(d_w=None), dict(df=df[:, :32])):
        with pytest.raises(ValueError):
            handle.add_norm_backward(**dict(dict(dy=x, dh=f, y=h, w=w, rstd=rstd, dx=dx, df=df, d_w=dw), **bad))
    for bad in (dict(df=x), dict(dx=df), dict(d_w=w), dict(p=2.0)):
        with pytest.raises(dm.DmuonError):
            handle.add_norm_backward(**dict(dict(dy=x, dh=f, y=h, w=w, rstd=rstd, dx=dx, df=df, d_w=dw), **bad))


def inputs(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    t = [(torch.randn(shape, generator=g) * torch.exp(torch.randn(shape[0], 1, generator=g))).to(DT[dtype]) for _ in range(4)]
    t[0][-1], t[1][-1] = 0, 0  # a row of zeros
    return t + [1 + 0.3 * torch.randn(shape[1], generator=g)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("p,with_x,odd,scale", [(0.1, True, False, "floor"), (0.5, False, True, "ceil"), (0.0, True, True, "floor"), (0.0, False, False, "ceil")])
def test_add_norm(handle, shape, dtype, p, with_x, odd, scale):
    rows, cols = shape
    x, f, dy, dh, w = inputs(shape, dtype, rows * 7 + cols)
    u, tiny = HALF[dtype], TINY[dtype]
    keep = op.factors(rows, cols, p, SEED, OFFSET)
    x64 = f64(x) if with_x else None
    ry, rh, rr = op.add_norm_forward(x64, f64(f), f64(w), keep)
    ybar = 2.0 ** -23 * (np.abs(f64(f) * keep) + np.abs(ry) + (np.abs(x64) if with_x else 0))

    xd, fd, wd = on_gpu(x, odd) if with_x else None, on_gpu(f, odd), w.cuda()
    y, h = buffer(rows, cols, DT[dtype], odd), buffer(rows, cols, DT[dtype], odd)
    q, rstd = tuple(t.fill_(0xAB) for t in dm.dmuon_mxfp8_empty(rows, cols)), torch.full((rows,), 7.0, device="cuda")
    drop = dict(p=p, seed=SEED, offset=OFFSET)
    handle.add_norm_forward(xd, fd, wd, y, rstd, out=h, q=q, scale=scale, **drop)
    assert (np.abs(f64(y) - ry) <= ybar * (1 + u) + u * np.abs(ry) + tiny).all()
    assert (np.abs(f64(rstd) - rr) <= 2.0 ** -18 * rr).all()
    hbar = 2.0 ** -17 * np.abs(rh) + ybar * rr[:, None] * np.abs(f64(w))
    assert (np.abs(f64(h) - rh) <= hbar * (1 + u) + u * np.abs(rh) + tiny).all()
    assert untouched(y, cols) and untouched(h, cols)
    wide = buffer(rows, cols, torch.float32, False)  # the same values as fp32
    handle.add_norm_forward(x.float().cuda() if with_x else None, f.float().cuda(), wd, torch.empty_like(wide), torch.empty_like(rstd), out=wide,
                            **drop)
    data, scales = ox.pack(*ox.quantize(f64(wide), scale))
    assert np.array_equal(q[0].cpu().numpy(), data) and np.array_equal(q[1].cpu().numpy(), scales)
    assert torch.equal(h, wide.to(DT[dtype]))
    for kw in (dict(out=torch.empty_like(h)), dict(q=tuple(torch.zeros_like(t) for t in q))):  # each alone
        y2, r2 = torch.zeros_like(y), torch.zeros_like(rstd)
        handle.add_norm_forward(xd, fd, wd, y2, r2, scale=scale, **drop, **kw)
        assert torch.equal(y2, y) and torch.equal(r2, rstd)
        assert torch.equal(kw["out"], h) if "out" in kw else all(torch.equal(a, b) for a, b in zip(kw["q"], q))

    dyd, dhd = on_gpu(dy, odd) if with_x else None, on_gpu(dh, odd)
    dx, df, dw = buffer(rows, cols, DT[dtype], odd), buffer(rows, cols, DT[dtype], odd), torch.full((cols,), 7.0, device="cuda")
    handle.add_norm_backward(dyd, dhd, y, wd, rstd, dx if with_x else None, df, dw, **drop)
    y64, r64, w64, g64 = f64(y), f64(rstd), f64(w), f64(dh)
    d64 = f64(dy) if with_x else np.zeros(shape)
    gx, gf, gw = op.add_norm_backward(d64, g64, y64, w64, r64, keep)
    yn = y64 * r64[:, None]
    terms = np.abs(d64) + r64[:, None] * (np.abs(g64 * w64) + np.abs(yn) * np.abs(g64 * w64 * yn).mean(1, keepdims=True))
    bar = 2.0 ** -17 * terms
    if with_x:
        assert (np.abs(f64(dx) - gx) <= bar * (1 + u) + u * np.abs(gx) + tiny).all() and untouched(dx, cols)
    assert (np.abs(f64(df) - gf) <= bar * keep * (1 + u) + u * np.abs(gf) + tiny).all() and untouched(df, cols)
    assert (np.abs(f64(dw) - gw) <= (2.0 ** -20 + rows * 2.0 ** -23) * np.abs(g64 * yn).sum(0)).all()
    if with_x and p == 0:
        assert torch.equal(dx, df)
    df2, dw2 = torch.zeros_like(df), torch.zeros_like(dw)
    handle.add_norm_backward(dyd, dhd, y, wd, rstd, None, df2, dw2, **drop)
    assert torch.equal(df2, df) and torch.equal(dw2, dw)
    assert handle.status()[0] == 0


def test_norm_without_rows_and_with_special_values(handle):
    e, w, dw = torch.empty((0, 40), device="cuda"), torch.ones(40, device="cuda"), torch.full((40,), 3.0, device="cuda")
    q, r = dm.dmuon_mxfp8_empty(0, 40), torch.empty(0, device="cuda")
    handle.add_norm_forward(e, e, w, e, r, out=e, q=q)
    handle.add_norm_backward(e, e, e, w, r, e, e, dw)
    assert not dw.any()
    x = torch.randn(4, 200, device="cuda")
    x[1, 3], x[2, 100] = float("inf"), float("nan")
    y, h, q, rstd = torch.empty_like(x), torch.empty_like(x), dm.dmuon_mxfp8_empty(4, 200), torch.empty(4, device="cuda")
    handle.add_norm_forward(None, x, torch.ones(200, device="cuda"), y, rstd, out=h, q=q)
    assert torch.isfinite(h[0]).all() and torch.isfinite(h[3]).all() and torch.isnan(h[1, 3]) and torch.isnan(h[2]).all()
    data, scales = ox.pack(*ox.quantize(f64(h)))
    assert np.array_equal(q[0].cpu().numpy(), data) and np.array_equal(q[1].cpu().numpy(), scales)
