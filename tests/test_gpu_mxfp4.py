"""MXFP4 quantisation, reading back and product against oracle/mxfp4.py.

Quantisation and reading back are exact: packed bytes (padding included) and
values have to be equal bit for bit.  The product's bar per element is
  (blocks + 2) 2^-22 sum_k |a_k b_k|  +  u |d|
block products are exact, each of the `blocks` fp32 additions may be off by
one unit in the last place of a partial sum (truncation), alpha and beta cost
one rounding each, and u is the output type's rounding (0, 2^-8, 2^-11).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402
from oracle import mxfp4 as ox  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    h = dm.Handle(0)
    yield h
    h.close()


def _values(rows, cols, seed, dtype):
    """Rows and columns of different size, exact ties, zeros and whole zero blocks."""
    r = np.random.RandomState(seed)
    x = r.randn(rows, cols) * np.exp(2 * r.randn(rows, 1)) * np.exp(r.randn(1, cols))
    tie = r.randint(-12, 13, (rows, cols)) / 4.0
    x = np.where(r.rand(rows, cols) < 0.3, tie, x)
    x = np.where(r.rand(rows, cols) < 0.05, 0.0, x)
    if rows > 40 and cols > 70:
        x[32:64, 32:64] = 0.0
    return torch.from_numpy(x).to(DT[dtype])


def _on_gpu(t, odd):
    """The same values; odd: in a wider buffer, one element off, with an odd pitch."""
    if not odd:
        return t.cuda()
    rows, cols = t.shape
    buf = torch.empty((rows, cols + 5), dtype=t.dtype, device="cuda")
    v = buf[:, 1:1 + cols]
    v.copy_(t)
    return v


def _filled(rows, k):
    """Buffers that hold something else before the call."""
    d, s = dm.dmuon_mxfp4_empty(rows, k)
    return d.fill_(0xAB), s.fill_(0xFF)


def _check_packed(got, codes, byte):
    data, scales = ox.pack(codes, byte)
    assert np.array_equal(got[0].cpu().numpy(), data)
    assert np.array_equal(got[1].cpu().numpy(), scales)


SHAPES = [(1, 1), (1, 32), (1, 4096), (5, 33), (31, 31), (128, 128), (129, 257), (300, 64), (77, 2061), (640, 96)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scale,noisy,odd", [("floor", False, False), ("ceil", False, True), ("ceil", True, False),
                                             ("floor", True, True)])
def test_quantize_is_exact(handle, shape, dtype, scale, noisy, odd):
    rows, cols = shape
    x = _values(rows, cols, 7 * rows + cols, dtype)
    noise = torch.from_numpy(np.random.RandomState(3).randint(0, 256, shape).astype(np.uint8)) if noisy else None
    src = _on_gpu(x, odd)
    nz = _on_gpu(noise, odd) if noisy else None
    by_rows, by_cols = _filled(rows, cols), _filled(cols, rows)
    handle.mxfp4_quantize(src, by_rows=by_rows, by_cols=by_cols, noise=nz, scale=scale)
    only_rows, only_cols = _filled(rows, cols), _filled(cols, rows)
    handle.mxfp4_quantize(src, by_rows=only_rows, noise=nz, scale=scale)
    handle.mxfp4_quantize(src, by_cols=only_cols, noise=nz, scale=scale)
    x64 = x.double().numpy()
    n = noise.numpy() if noisy else None
    for want, both, one, k in ((ox.quantize(x64, scale, n), by_rows, only_rows, cols),
                               (ox.quantize(x64.T, scale, None if n is None else n.T), by_cols, only_cols, rows)):
        _check_packed(both, *want)
        _check_packed(one, *want)
        out = torch.empty((want[0].shape[0], k), dtype=DT[dtype], device="cuda")
        out = _on_gpu(out.cpu(), odd)
        handle.mxfp4_dequantize(both, out)
        assert torch.equal(out.cpu(), torch.from_numpy(ox.values(*want, k)).to(DT[dtype]))
    assert handle.status()[0] == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("noisy", [False, True])
def test_quantize_special_values(handle, dtype, noisy):
    """Infinities, NaN, the type's largest and smallest values, signed zeros:
    one special element a block, along rows and along columns."""
    info = torch.finfo(DT[dtype])
    sub = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}[dtype]
    special = [float("inf"), float("-inf"), float("nan"), info.max, info.min, info.tiny, sub, -sub, -0.0, 3 * sub]
    x = torch.randn(96, 32 * len(special), generator=torch.Generator().manual_seed(5)).to(DT[dtype])
    for i, v in enumerate(special):
        x[i, 32 * i + 7] = v
        x[32 + i, 32 * i:32 * i + 32] = 0  # alone in a row block
        x[32 + i, 32 * i + 3] = v
        x[64:, 32 * i + i] = 0             # alone in a column block
        x[70, 32 * i + i] = v
    noise = torch.from_numpy(np.random.RandomState(4).randint(0, 256, x.shape).astype(np.uint8)) if noisy else None
    for scale in ("floor", "ceil"):
        by_rows, by_cols = _filled(*x.shape), _filled(x.shape[1], x.shape[0])
        handle.mxfp4_quantize(x.cuda(), by_rows=by_rows, by_cols=by_cols, noise=noise.cuda() if noisy else None, scale=scale)
        x64, n = x.double().numpy(), noise.numpy() if noisy else None
        for want, got, k in ((ox.quantize(x64, scale, n), by_rows, x.shape[1]),
                             (ox.quantize(x64.T, scale, None if n is None else n.T), by_cols, x.shape[0])):
            _check_packed(got, *want)
            out = torch.empty((want[0].shape[0], k), dtype=DT[dtype], device="cuda")
            handle.mxfp4_dequantize(got, out)
            ref = torch.from_numpy(ox.values(*want, k)).to(DT[dtype])
            assert torch.equal(out.cpu().isnan(), ref.isnan())
            assert torch.equal(out.cpu().nan_to_num(0.0, 1.0, -1.0), ref.nan_to_num(0.0, 1.0, -1.0))


def test_stochastic_rounding_is_unbiased(handle):
    """Every byte once per value: the mean is the value within the byte's
    resolution (1/512 of a step) and no further."""
    v = torch.tensor([0.1, 0.6, 1.2, 1.9, 2.3, 3.7, 5.5, 6.0] * 4).repeat(256, 1).cuda()
    noise = torch.arange(256, dtype=torch.uint8).view(256, 1).repeat(1, 32).cuda()
    q = dm.dmuon_mxfp4_empty(256, 32)
    handle.mxfp4_quantize(v, by_rows=q, noise=noise, scale="ceil")
    out = torch.empty_like(v)
    handle.mxfp4_dequantize(q, out)
    step = torch.where(v[0] < 2, 0.5, torch.where(v[0] < 4, 1.0, 2.0))
    assert ((out.double().mean(0) - v[0].double()).abs() <= step.double() / 512 + 1e-12).all()


def test_stochastic_rounding_at_its_thresholds(handle):
    """fp32 values at every threshold of every interval, and one unit in the
    last place to either side of it."""
    lo, r = np.meshgrid(np.arange(7), np.arange(256), indexing="ij")
    at = (ox.GRID[lo] + (ox.GRID[lo + 1] - ox.GRID[lo]) * (r + 0.5) / 256).astype(np.float32).reshape(-1)
    v = np.stack((np.nextafter(at, np.float32(0)), at, np.nextafter(at, np.float32(9))))
    rows = -(-v.size // 31)
    x = np.zeros((rows, 32), dtype=np.float32)
    x[:, 31] = 6.0  # the block's largest: e = 0
    x[:, :31] = np.resize(v, (rows, 31))
    noise = np.zeros((rows, 32), dtype=np.uint8)
    noise[:, :31] = np.resize(np.tile(r.reshape(-1), 3), (rows, 31))
    q = dm.dmuon_mxfp4_empty(rows, 32)
    handle.mxfp4_quantize(torch.from_numpy(x).cuda(), by_rows=q, noise=torch.from_numpy(noise).cuda(), scale="ceil")
    _check_packed(q, *ox.quantize(x, "ceil", noise))
    codes = ox.quantize(x, "ceil", noise)[0].reshape(rows, 32)[:, :31].reshape(-1)[:v.size].reshape(3, 7, 256)
    want = np.broadcast_to(np.arange(7)[:, None], (7, 256))
    assert (codes[0] == want).all() and (codes[1] == want).all() and (codes[2] == want + 1).all()


def _operand(handle, rows, k, seed):
    """An MXFP4 matrix on the GPU and its values in fp64."""
    r = np.random.RandomState(seed)
    x = (r.randn(rows, k) * np.exp(r.randn(rows, 1))).astype(np.float32)
    q = _filled(rows, k)
    handle.mxfp4_quantize(torch.from_numpy(x).cuda(), by_rows=q)
    v = torch.empty((rows, k), device="cuda")
    handle.mxfp4_dequantize(q, v)
    return q, v.cpu().double().numpy()


def _check_gemm(handle, m, n, k, dtype, alpha=1.0, beta=0.0, pad=0, seed=0):
    a, av = _operand(handle, m, k, seed + 1)
    b, bv = _operand(handle, n, k, seed + 2)
    d0 = torch.randn((m, n + pad), generator=torch.Generator().manual_seed(seed)).to(DT[dtype])
    buf = d0.cuda()
    out = buf[:, :n]
    handle.mxfp4_gemm(a, b, out, k, alpha=alpha, beta=beta)
    assert handle.status()[0] == 0
    want = alpha * (av @ bv.T) + (beta * d0[:, :n].double().numpy() if beta else 0.0)
    got = out.cpu().double().numpy()
    u = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
    size = abs(alpha) * (np.abs(av) @ np.abs(bv).T) + (abs(beta) * np.abs(d0[:, :n].double().numpy()) if beta else 0.0)
    bar = (-(-k // 32) + 2) * 2.0 ** -22 * size + u * np.abs(want) + (2.0 ** -24 if dtype == "f16" else 0.0)
    if dtype == "f16":  # 65520 is where fp16 rounds to infinity
        over = np.abs(want) - bar >= 65520.0
        assert np.array_equal(got[over], np.copysign(np.inf, want[over]))
        near = np.isinf(got) & (np.abs(want) + bar >= 65520.0)
        got, want = np.where(near | over, 0.0, got), np.where(near | over, 0.0, want)
    off = np.abs(got - want)
    assert (off <= bar).all(), (m, n, k, dtype, float((off / bar).max()), np.argwhere(off > bar)[:5].tolist())
    if pad:
        assert torch.equal(buf[:, n:].cpu(), d0[:, n:])
    # the same bits again
    first = out.clone()
    buf.copy_(d0)
    handle.mxfp4_gemm(a, b, out, k, alpha=alpha, beta=beta)
    assert torch.equal(out, first)


@pytest.mark.parametrize("m,n,k", [
    (1, 1, 1), (1, 5, 31), (1, 128, 32), (2, 129, 64), (1, 4096, 4096), (3, 1000, 2061), (16, 512, 2048), (17, 260, 96),
    (32, 128, 256), (33, 127, 257), (64, 300, 8192), (65, 511, 513), (77, 1111, 2061), (128, 384, 1024),
    (129, 256, 320), (200, 200, 200), (256, 512, 512), (257, 100, 129), (300, 31, 700), (513, 33, 4100), (384, 640, 1088),
    (1000, 1000, 1000), (2048, 512, 2048), (512, 2048, 300), (1025, 513, 65)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_gemm(handle, m, n, k, dtype):
    _check_gemm(handle, m, n, k, dtype, seed=m + n + k)


@pytest.mark.parametrize("m,n,k", [(1, 130, 96), (40, 257, 1500), (300, 500, 4096), (520, 260, 288), (2100, 1300, 640)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("alpha,beta,pad", [(0.5, 1.0, 0), (-2.0, 0.25, 3), (1.0, 0.0, 7), (0.0, 1.0, 1)])
def test_gemm_alpha_beta_pitch(handle, m, n, k, dtype, alpha, beta, pad):
    _check_gemm(handle, m, n, k, dtype, alpha, beta, pad, seed=11)


@pytest.mark.parametrize("m,n,k", [(2500, 2560, 1024), (4100, 1030, 2080), (777, 5000, 544), (150, 12000, 320), (12001, 131, 96)])
def test_gemm_many_tiles(handle, m, n, k):
    _check_gemm(handle, m, n, k, "f32", 1.0, 1.0, 2, seed=21)
    _check_gemm(handle, m, n, k, "bf16", seed=22)


def test_gemm_beta_zero_ignores_d(handle):
    for m in (1, 300):
        a, av = _operand(handle, m, 64, 1)
        b, bv = _operand(handle, 40, 64, 2)
        out = torch.full((m, 40), float("nan"), device="cuda")
        handle.mxfp4_gemm(a, b, out, 64)
        assert np.allclose(out.cpu().double().numpy(), av @ bv.T, rtol=1e-5, atol=1e-4)


@pytest.mark.parametrize("m", [3, 700])
def test_gemm_nan_scale_spoils_its_row_only(handle, m):
    n, k = 300, 320
    x = torch.randn((m, k), generator=torch.Generator().manual_seed(1))
    x[1, 70] = float("inf")
    a = dm.dmuon_mxfp4_empty(m, k)
    handle.mxfp4_quantize(x.cuda(), by_rows=a)
    b, _ = _operand(handle, n, k, 2)
    out = torch.zeros((m, n), device="cuda")
    handle.mxfp4_gemm(a, b, out, k)
    bad = out.isnan().cpu()
    assert bad[1].all() and not bad[0].any() and not bad[2:].any()


@pytest.mark.parametrize("ea,eb", [(-120, 100), (100, -120), (-60, -60), (60, 60)])
def test_gemm_extreme_scales(handle, ea, eb):
    """Exponents far from 0 on either side: exact (small integers) wherever no
    partial sum can pass fp32's largest value."""
    r = np.random.RandomState(9)
    x, w = r.randint(-6, 7, (40, 160)).astype(np.float64), r.randint(-6, 7, (200, 160)).astype(np.float64)
    a, b = dm.dmuon_mxfp4_empty(40, 160), dm.dmuon_mxfp4_empty(200, 160)
    handle.mxfp4_quantize(torch.from_numpy((x * 2.0 ** ea).astype(np.float32)).cuda(), by_rows=a, scale="ceil")
    handle.mxfp4_quantize(torch.from_numpy((w * 2.0 ** eb).astype(np.float32)).cuda(), by_rows=b, scale="ceil")
    out = torch.empty((40, 200), device="cuda")
    handle.mxfp4_gemm(a, b, out, 160)
    xv = ox.values(*ox.quantize(x, "ceil"), 160)
    wv = ox.values(*ox.quantize(w, "ceil"), 160)
    sums = np.cumsum([xv[:, i:i + 32] @ wv[:, i:i + 32].T for i in range(0, 160, 32)], axis=0)  # block by block
    fits = np.abs(sums).max(0) * 2.0 ** (ea + eb) < np.finfo(np.float32).max
    assert fits.any()
    assert np.array_equal(out.cpu().double().numpy()[fits], ((xv @ wv.T) * 2.0 ** (ea + eb))[fits])


def test_gemm_on_another_stream(handle):
    s = torch.cuda.Stream()
    x = torch.randn((50, 512), generator=torch.Generator().manual_seed(3)).cuda()
    w = torch.randn((260, 512), generator=torch.Generator().manual_seed(4)).cuda()
    a, b = dm.dmuon_mxfp4_empty(50, 512), dm.dmuon_mxfp4_empty(260, 512)
    out = torch.empty((50, 260), device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    handle.mxfp4_quantize(x, by_rows=a, stream=s)
    handle.mxfp4_quantize(w, by_rows=b, stream=s)
    handle.mxfp4_gemm(a, b, out, 512, stream=s)
    s.synchronize()
    ref = torch.empty_like(out)
    handle.mxfp4_quantize(x, by_rows=a)
    handle.mxfp4_gemm(a, b, ref, 512)
    assert torch.equal(out, ref)


@pytest.mark.parametrize("m", [1, 600])
def test_products_in_a_graph(handle, m):
    n, k = 384, 576
    x = torch.randn((m, k), generator=torch.Generator().manual_seed(3)).cuda()
    b, bv = _operand(handle, n, k, 4)
    a, av = dm.dmuon_mxfp4_empty(m, k), torch.empty((m, k), device="cuda")
    out = torch.zeros((m, n), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        handle.mxfp4_quantize(x, by_rows=a)
        handle.mxfp4_gemm(a, b, out, k)
        handle.mxfp4_dequantize(a, av)
    x.copy_(torch.randn((m, k), generator=torch.Generator().manual_seed(8)))
    g.replay()
    want = av.cpu().double().numpy() @ bv.T
    assert np.allclose(out.cpu().double().numpy(), want, rtol=1e-5, atol=1e-3)


def test_wait_that_runs_out_is_reported(handle):
    """A limit of one nanosecond: some wait of a long product gives up, the
    status says so once, and the next product is right again."""
    a, _ = _operand(handle, 2048, 16384, 1)
    out = torch.empty((2048, 2048), device="cuda")
    dm.dmuon_set_wait_timeout(handle.h, 1)
    handle.mxfp4_gemm(a, a, out, 16384)
    assert handle.status()[0] == -6
    dm.dmuon_set_wait_timeout(handle.h, 0)
    assert handle.status()[0] == 0
    _check_gemm(handle, 300, 300, 512, "f32")


# ------------------------------------------------------------------ refusals

def test_quantize_refusals(handle):
    x = torch.zeros((8, 64), device="cuda")
    q = dm.dmuon_mxfp4_empty(8, 64)
    for bad in (x.cpu(), x[0], x.double(), x.t(), x.int()):
        with pytest.raises(ValueError):
            handle.mxfp4_quantize(bad, by_rows=q)
    with pytest.raises(ValueError):
        handle.mxfp4_quantize(x, by_cols=q)  # sizes of the wrong direction
    with pytest.raises(ValueError):
        handle.mxfp4_quantize(x, by_rows=q, noise=torch.zeros((8, 63), dtype=torch.uint8, device="cuda"))
    with pytest.raises(dm.DmuonError):
        handle.mxfp4_quantize(x)  # no output
    with pytest.raises(KeyError):
        handle.mxfp4_quantize(x, by_rows=q, scale="nearest")
    L, p = dm.load(), x.data_ptr()
    d, s = q[0].data_ptr(), q[1].data_ptr()

    def call(src=p, dt=0, r=8, c=64, ld=64, mode=0, noise=None, nld=0, d=d, s=s, cd=None, cs=None):
        return L.dmuon_mxfp4_quantize(handle.h, src, dt, r, c, ld, mode, noise, nld, d, s, cd, cs, None)
    assert call() == 0
    assert call(src=None) == -1 and call(dt=3) == -1 and call(ld=63) == -1 and call(mode=2) == -1
    assert call(r=-1) == -1 and call(c=(1 << 30) + 1) == -1 and call(noise=p, nld=63) == -1
    assert call(s=None) == -1 and call(cd=d) == -1 and call(cd=d, cs=s) == -1 and call(d=p) == -1
    assert call(src=p + 2) == -2 and call(d=d + 8) == -2
    assert call(r=0) == 0 and call(c=0, ld=0) == 0
    assert L.dmuon_mxfp4_quantize(None, p, 0, 8, 64, 64, 0, None, 0, d, s, None, None, None) == -1


def test_gemm_refusals(handle):
    a, b = dm.dmuon_mxfp4_empty(4, 64), dm.dmuon_mxfp4_empty(8, 64)
    for t in a + b:
        t.zero_()
    out = torch.zeros((4, 8), device="cuda")
    with pytest.raises(ValueError):
        handle.mxfp4_gemm(b, a, out, 64)
    with pytest.raises(ValueError):
        handle.mxfp4_gemm(a, b, out, 65)
    with pytest.raises(ValueError):
        handle.mxfp4_gemm(a, b, out.t().contiguous().t(), 64)
    with pytest.raises(dm.DmuonError):
        handle.mxfp4_gemm(a, b, out, 64, alpha=float("nan"))
    L = dm.load()
    ps = [t.data_ptr() for t in a + b]

    def call(p=ps, m=4, n=8, k=64, d=out.data_ptr(), dt=0, ldd=8, alpha=1.0, beta=0.0):
        return L.dmuon_mxfp4_gemm(handle.h, *p, m, n, k, d, dt, ldd, alpha, beta, None)
    assert call() == 0
    assert call(k=0) == -1 and call(m=-1) == -1 and call(ldd=7) == -1 and call(dt=5) == -1 and call(d=None) == -1
    assert call(p=[None] + ps[1:]) == -1 and call(p=ps[:3] + [ps[2]]) == -1 and call(d=ps[0]) == -1
    assert call(p=[ps[0] + 8] + ps[1:]) == -2 and call(d=out.data_ptr() + 2) == -2
    assert call(beta=float("inf")) == -1 and call(m=0) == 0 and call(n=0, ldd=0) == 0
    assert L.dmuon_mxfp4_dequantize(handle.h, ps[0], ps[1], 4, 64, out.data_ptr(), 0, 63, None) == -1
