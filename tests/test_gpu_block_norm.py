"""Norms around a block, forward and backward, against oracle/block_norm.py.

With E = (cols / 64 + 64) 2^-24 (fp32 rounding of a row's sums, however the
columns are split over threads, and of the few operations on each element) a
value that is a sum of terms may be off by 8 E times the sum of the terms'
sizes, a column sum by (8 E + (rows + 64) 2^-24) times the sum over rows, and
stored values by their type's rounding.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402
from oracle import block_norm as on  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
EPS = 1e-6


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    h = dm.Handle(0)
    yield h
    h.close()


class Case:
    def __init__(self, rows, cols, dtype, per=None, res=False, odd=0, seed=0):
        r = np.random.RandomState(seed + rows * 31 + cols)
        self.rows, self.cols, self.dtype, self.per, self.odd = rows, cols, dtype, per, odd

        def act():
            t = r.randn(rows, cols) * np.exp(0.5 * r.randn(rows, 1))
            return torch.from_numpy(t).to(DT[dtype])

        def par(*shape):
            return torch.from_numpy(r.randn(*shape).astype(np.float32))
        self.x, self.f, self.dy, self.dh = act(), act(), act(), act()
        self.post_w, self.pre_w = par(cols) + 1, par(cols) + 1
        self.gate = par(-(-rows // per), cols) if per else None
        self.res = par(cols) if res else None

    def dev(self, t=None):
        """A [rows, cols] activation on the GPU; odd: one element off with an odd pitch."""
        buf = torch.empty((self.rows, self.cols + 2 * self.odd), dtype=DT[self.dtype], device="cuda")
        v = buf[:, self.odd:self.odd + self.cols]
        if t is not None:
            v.copy_(t)
        return v

    def par(self, t):
        return None if t is None else t.cuda()

    def n(self, t):
        return None if t is None else t.double().numpy()

    @property
    def e(self):
        return (self.cols / 64 + 64) * 2.0 ** -24


def _within(got, want, size, e, u, name, tiny=0.0):
    off = np.abs(got.cpu().double().numpy() - want)
    bar = e * size + u * np.abs(want) + tiny
    assert (off <= bar).all(), (name, float((off / np.maximum(bar, 1e-300)).max()))


def _forward(handle, c, **kw):
    y, out = c.dev(), c.dev()
    rstd = torch.empty((2, c.rows), device="cuda")
    handle.block_norm_forward(c.dev(c.x), c.dev(c.f), c.par(c.post_w), c.par(c.pre_w), y, out, rstd, gate=c.par(c.gate),
                              rows_per_gate=c.per, res_scale=c.par(c.res), eps=EPS, **kw)
    return y, out, rstd


def _check_forward(handle, c):
    y, out, rstd = _forward(handle, c)
    x, f, pw, qw, g, res = (c.n(t) for t in (c.x, c.f, c.post_w, c.pre_w, c.gate, c.res))
    wy, wh, wr = on.forward(x, f, pw, qw, g, c.per, res, EPS)
    rows = 1.0 if g is None else g[np.arange(c.rows) // c.per]
    size = np.abs((1.0 if res is None else res) * x) + np.abs(rows * f * wr[0][:, None] * pw)
    spread = (size * np.abs(wy)).sum(1, keepdims=True) / np.maximum((wy * wy).sum(1, keepdims=True), 1e-300)
    tiny = 2.0 ** -24 if c.dtype == "f16" else 0.0
    _within(y, wy, size, 8 * c.e, U[c.dtype], "y", tiny)
    _within(out, wh, (size + spread * np.abs(wy)) * wr[1][:, None] * np.abs(qw), 8 * c.e, U[c.dtype], "h", tiny)
    # eps is a term of the second mean too: a row of zeros has only that
    terms = np.maximum(spread[:, 0], 1.0)
    _within(rstd, wr, np.stack((wr[0], wr[1] * terms)), 8 * c.e, 0.0, "rstd")


def _backward(handle, c, y, rstd, dy=True, d_gate=True, d_res=True):
    dx, df = c.dev(), c.dev()
    out = {"dx": dx, "df": df, "d_post_w": torch.full((c.cols,), 7.0, device="cuda"),
           "d_pre_w": torch.full((c.cols,), 7.0, device="cuda")}
    if c.gate is not None and d_gate:
        out["d_gate"] = torch.full(tuple(c.gate.shape), 7.0, device="cuda")
    if c.res is not None and d_res:
        out["d_res_scale"] = torch.full((c.cols,), 7.0, device="cuda")
    handle.block_norm_backward(c.dev(c.dy) if dy else None, c.dev(c.dh), c.dev(c.x) if "d_res_scale" in out else None,
                               c.dev(c.f), y, c.par(c.post_w), c.par(c.pre_w), rstd, dx, df, out["d_post_w"],
                               out["d_pre_w"], gate=c.par(c.gate), d_gate=out.get("d_gate"), rows_per_gate=c.per,
                               res_scale=c.par(c.res), d_res_scale=out.get("d_res_scale"))
    return out


def _check_backward(handle, c, **kw):
    y, _, rstd = _forward(handle, c)
    got = _backward(handle, c, y, rstd, **kw)
    x, f, pw, qw, g, res, dh = (c.n(t) for t in (c.x, c.f, c.post_w, c.pre_w, c.gate, c.res, c.dh))
    dy = c.n(c.dy) if kw.get("dy", True) else np.zeros_like(dh)
    y64, r64 = y.cpu().double().numpy(), rstd.cpu().double().numpy()
    want = on.backward(dy, dh, x, f, y64, pw, qw, r64, g, c.per, res)
    r1, r2 = r64[0][:, None], r64[1][:, None]
    yn, fn = np.abs(y64 * r2), np.abs(f * r1)
    into = np.abs(dh * qw)
    t = np.abs(dy) + r2 * (into + yn * (into * yn).mean(1, keepdims=True))
    rows = np.ones_like(t) if g is None else np.abs(g)[np.arange(c.rows) // c.per]
    back = rows * t * np.abs(pw)
    size = {"dx": np.abs(1.0 if res is None else res) * t, "df": r1 * (back + fn * (back * fn).mean(1, keepdims=True)),
            "d_post_w": (rows * t * fn).sum(0), "d_pre_w": np.abs(dh * yn).sum(0)}
    if "d_gate" in got:
        size["d_gate"] = np.zeros_like(g)
        np.add.at(size["d_gate"], np.arange(c.rows) // c.per, t * fn * np.abs(pw))
    if "d_res_scale" in got:
        size["d_res_scale"] = (t * np.abs(x)).sum(0)
    tiny = 2.0 ** -24 if c.dtype == "f16" else 0.0
    for name, v in got.items():
        if name in ("dx", "df"):
            _within(v, want[name], size[name], 8 * c.e, U[c.dtype], name, tiny)
        else:
            _within(v, want[name], size[name], 8 * c.e + (c.rows + 64) * 2.0 ** -24, U["f32"], name)
    again = _backward(handle, c, y, rstd, **kw)
    assert all(torch.equal(v, again[name]) for name, v in got.items())


SHAPES = [(1, 1), (1, 7), (3, 64), (1, 4096), (5, 100), (33, 257), (130, 512), (700, 128), (64, 1111), (40, 2048),
          (17, 4097), (350, 4096), (9, 8192), (3, 16384), (2, 20011), (5, 32768), (2, 40000)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_forward(handle, rows, cols, dtype):
    _check_forward(handle, Case(rows, cols, dtype))
    _check_forward(handle, Case(rows, cols, dtype, per=max(1, rows // 3), res=True))


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_backward(handle, rows, cols, dtype):
    _check_backward(handle, Case(rows, cols, dtype))
    _check_backward(handle, Case(rows, cols, dtype, per=max(1, rows // 3), res=True))


@pytest.mark.parametrize("per", [1, 2, 7, 100, 1299, 1300, 5000])
@pytest.mark.parametrize("cols", [96, 520])
def test_gate_groups(handle, per, cols):
    c = Case(1300, cols, "f32", per=per, res=False)
    _check_forward(handle, c)
    _check_backward(handle, c)


@pytest.mark.parametrize("rows,cols", [(33, 257), (40, 512), (6, 4096), (5, 9000)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_that_are_not_aligned(handle, rows, cols, dtype):
    c = Case(rows, cols, dtype, per=4, res=True, odd=1)
    _check_forward(handle, c)
    _check_backward(handle, c)


@pytest.mark.parametrize("kw", [dict(dy=False), dict(d_gate=False), dict(d_res=False), dict(dy=False, d_gate=False, d_res=False)])
@pytest.mark.parametrize("cols", [77, 256, 4096])
def test_backward_without_some(handle, kw, cols):
    _check_backward(handle, Case(90, cols, "bf16", per=11, res=True), **kw)


def test_zero_rows_and_nan_stay_in_their_row(handle):
    c = Case(12, 256, "f32", per=3, res=True)
    c.x[2] = 0
    c.f[2] = 0
    c.f[5] = 0
    _check_forward(handle, c)
    _check_backward(handle, c)
    c.f[7, 3] = float("nan")
    y, out, rstd = _forward(handle, c)
    bad = out.isnan().cpu()
    assert bad[7].all() and not bad[:7].any() and not bad[8:].any()
    assert not rstd[:, 8:].isnan().any()


def test_gradients_against_differences(handle):
    """Directional central differences of the fp64 forward against the
    kernels' fp32 gradients."""
    c = Case(23, 264, "f32", per=5, res=True)
    y, _, rstd = _forward(handle, c)
    got = {k: v.cpu().double().numpy() for k, v in _backward(handle, c, y, rstd).items()}
    base = {"dx": c.n(c.x), "df": c.n(c.f), "d_post_w": c.n(c.post_w), "d_pre_w": c.n(c.pre_w), "d_gate": c.n(c.gate),
            "d_res_scale": c.n(c.res)}
    r, eps = np.random.RandomState(1), 1e-6
    for name, v in base.items():
        way = r.randn(*v.shape)

        def loss(at):
            b = dict(base, **{name: at})
            wy, wh, _ = on.forward(b["dx"], b["df"], b["d_post_w"], b["d_pre_w"], b["d_gate"], c.per, b["d_res_scale"], EPS)
            return (wy * c.n(c.dy)).sum() + (wh * c.n(c.dh)).sum()
        num = (loss(v + eps * way) - loss(v - eps * way)) / (2 * eps)
        # fp32 gradients: each of the entries off by about 1e-5 of its size at most
        assert abs(num - (got[name] * way).sum()) <= 1e-5 * (np.abs(got[name] * way).sum() + 1)


def test_no_rows(handle):
    w = torch.ones(64, device="cuda")
    e = torch.empty((0, 64), device="cuda")
    r = torch.empty((2, 0), device="cuda")
    handle.block_norm_forward(e, e, w, w, e, e, r)
    a, b = torch.full((64,), 3.0, device="cuda"), torch.full((64,), 3.0, device="cuda")
    handle.block_norm_backward(e, e, e, e, e, w, w, r, e, e, a, b)
    assert not a.any() and not b.any()


def test_on_another_stream_and_in_a_graph(handle):
    c = Case(60, 512, "bf16", per=7, res=True)
    y, out, rstd = _forward(handle, c)
    want = _backward(handle, c, y, rstd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = _backward(handle, c, y, rstd)
    s.synchronize()
    assert all(torch.equal(v, got[k]) for k, v in want.items())
    ins = [c.dev(t) for t in (c.x, c.f)]
    pars = [c.par(t) for t in (c.post_w, c.pre_w)]
    y2, out2, rstd2 = c.dev(), c.dev(), torch.empty((2, c.rows), device="cuda")
    gate, res = c.par(c.gate), c.par(c.res)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        handle.block_norm_forward(*ins, *pars, y2, out2, rstd2, gate=gate, rows_per_gate=c.per, res_scale=res, eps=EPS)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out2, out) and torch.equal(rstd2, rstd)


def test_refusals(handle):
    c = Case(4, 64, "f32")
    x, f, y, out = c.dev(c.x), c.dev(c.f), c.dev(), c.dev()
    w, v = c.par(c.post_w), c.par(c.pre_w)
    rstd = torch.empty((2, 4), device="cuda")
    ok = (x, f, w, v, y, out, rstd)

    def swap(i, t):
        return ok[:i] + (t,) + ok[i + 1:]
    for bad in (swap(0, x.bfloat16()), swap(1, f[:3]), swap(2, w[:63]), swap(3, v.double()), swap(4, y.cpu()),
                swap(5, torch.empty((64, 4), device="cuda").t()), swap(6, rstd[:1])):
        with pytest.raises(ValueError):
            handle.block_norm_forward(*bad)
    for bad in (swap(5, y), swap(4, x), swap(5, f)):
        with pytest.raises(dm.DmuonError):
            handle.block_norm_forward(*bad)
    with pytest.raises(ValueError):
        handle.block_norm_forward(*ok, gate=torch.ones((1, 64), device="cuda"), rows_per_gate=3)
    with pytest.raises(ValueError):
        handle.block_norm_forward(*ok, rows_per_gate=0)
    with pytest.raises(dm.DmuonError):
        handle.block_norm_forward(*ok, eps=float("nan"))
    dx, df, a, b = c.dev(), c.dev(), torch.empty(64, device="cuda"), torch.empty(64, device="cuda")
    back = (x, x, None, f, y, w, v, rstd, dx, df, a, b)
    with pytest.raises(ValueError):
        handle.block_norm_backward(*back, d_gate=torch.ones((1, 64), device="cuda"))
    with pytest.raises(dm.DmuonError):
        handle.block_norm_backward(*back, d_res_scale=a.clone())  # no res_scale
    with pytest.raises(dm.DmuonError):
        handle.block_norm_backward(*back, res_scale=w, d_res_scale=a.clone())  # no x
    with pytest.raises(dm.DmuonError):
        handle.block_norm_backward(*(back[:9] + (dx, a, b)))
    with pytest.raises(dm.DmuonError):
        handle.block_norm_backward(*(back[:11] + (a,)))
