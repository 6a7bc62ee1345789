"""Offsets past 2^31 elements, and rows longer than a CTA holds at once: what the last
rows hold is what a call on these rows alone gives."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402
from oracle import mxfp8 as ox  # noqa: E402
from oracle import projection as op  # noqa: E402

pytestmark = pytest.mark.gpu

ROWS, COLS, TAIL = 69 * 1024, 32001, 256  # 2.26e9 elements, odd rows


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("60 GB of device memory are wanted")
    _build.build()
    with dm.Handle(0) as h:
        yield h
    torch.cuda.empty_cache()


def f64(t):
    return t.detach().cpu().double().numpy()


@pytest.fixture(scope="module")
def x(handle):
    t = torch.empty((ROWS, COLS), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    t[-TAIL:] = torch.randn((TAIL, COLS), device="cuda", generator=gen)
    t[:-TAIL].fill_(0.5)
    return t


def test_quantise_and_act_backward(handle, x):
    q, qt = dm.dmuon_mxfp8_empty(ROWS, COLS), dm.dmuon_mxfp8_empty(COLS, ROWS)
    handle.mxfp8_quantize(x, q, qt)
    tail = x[-TAIL:].contiguous()
    data, scales = ox.pack(*ox.quantize(f64(tail)))
    assert np.array_equal(q[0][-TAIL:].cpu().numpy(), data) and np.array_equal(q[1][-len(scales):].cpu().numpy(), scales)
    rows = np.r_[0:40, COLS - 40:COLS]
    codes, byte = ox.quantize(f64(tail[:, rows]).T)
    assert np.array_equal(qt[0][rows, -TAIL:].cpu().numpy(), codes.reshape(len(rows), -1))
    back = torch.empty((TAIL, COLS), dtype=torch.bfloat16, device="cuda")
    whole = torch.empty_like(x)
    handle.mxfp8_dequantize(q, whole)
    handle.mxfp8_dequantize((q[0][-TAIL:], q[1][-len(scales):]), back)
    assert torch.equal(whole[-TAIL:], back)
    del qt
    sums, small = torch.empty(COLS, device="cuda"), torch.empty(COLS, device="cuda")
    handle.act_backward(x, x, "silu", dz=whole, d_bias=sums, by_rows=q)
    handle.act_backward(tail, tail, "silu", dz=back, d_bias=small)
    assert torch.equal(whole[-TAIL:], back)
    each = 0.5 * op.slope(np.array(0.5), "silu")
    want = f64(small) + (ROWS - TAIL) * each
    assert (np.abs(f64(sums) - want) <= 2.0 ** -12 * (ROWS - TAIL) * each).all()  # 128 to 2^11 terms a chain, 2^-24 each
    assert handle.status()[0] == 0


def test_dropout_and_norm(handle, x):
    out = torch.empty_like(x)
    handle.dropout(x, out, 0.25, 9, 3)
    keep = op.factors(TAIL, COLS, 0.25, 9, 3, first_row=ROWS - TAIL)
    want = f64(x[-TAIL:]) * keep
    assert (np.abs(f64(out[-TAIL:]) - want) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(want)).all()
    w, rstd, q = torch.ones(COLS, device="cuda"), torch.empty(ROWS, device="cuda"), dm.dmuon_mxfp8_empty(ROWS, COLS)
    y = torch.empty_like(x)
    handle.add_norm_forward(None, x, w, y, rstd, out=out, q=q, p=0.25, seed=9, offset=3)
    ry, rh, rr = op.add_norm_forward(None, f64(x[-TAIL:]), 1.0, keep)
    assert (np.abs(f64(y[-TAIL:]) - ry) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(ry)).all()
    assert (np.abs(f64(rstd[-TAIL:]) - rr) <= 2.0 ** -17 * rr).all()
    assert (np.abs(f64(out[-TAIL:]) - rh) <= (2.0 ** -8 + 2.0 ** -16) * np.abs(rh)).all()
    dw, one = torch.empty(COLS, device="cuda"), torch.empty(COLS, device="cuda")
    handle.add_norm_backward(None, x, y, w, rstd, None, out, dw, p=0.25, seed=9, offset=3)
    gx, gf, _ = op.add_norm_backward(0.0, f64(x[-TAIL:]), f64(y[-TAIL:]), 1.0, f64(rstd[-TAIL:]), keep)
    terms = np.abs(f64(rstd[-TAIL:]))[:, None] * np.abs(f64(x[-TAIL:]))
    assert (np.abs(f64(out[-TAIL:]) - gf) <= 2.0 ** -8 * np.abs(gf) + 2.0 ** -14 * (terms + terms.mean(1, keepdims=True) * 4) * keep).all()
    assert handle.status()[0] == 0


def test_projection(handle):
    m, n, k = 128 * 400, 44000, 64  # D: 2.25e9 elements
    gen = torch.Generator(device="cuda").manual_seed(2)
    a, b = dm.dmuon_mxfp8_empty(m, k), dm.dmuon_mxfp8_empty(n, k)
    handle.mxfp8_quantize(torch.randn((m, k), device="cuda", generator=gen), a)
    handle.mxfp8_quantize(torch.randn((n, k), device="cuda", generator=gen), b)
    bias = torch.randn(n, device="cuda", generator=gen)
    out, pre = (torch.empty((m, n), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    handle.mx_linear(a, b, out, k, bias=bias, act="gelu", pre=pre, residual=None)
    rows = 128 * 3
    s = a[1].view(m // 128, -1)
    last = (a[0][-rows:].contiguous(), s[-rows // 128:].contiguous().view(-1))
    o, p = (torch.empty((rows, n), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    handle.mx_linear(last, b, o, k, bias=bias, act="gelu", pre=p)
    assert torch.equal(out[-rows:], o) and torch.equal(pre[-rows:], p)
    assert handle.status()[0] == 0
