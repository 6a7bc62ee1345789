"""The residual norm where every unit of threads goes through many rows, so that each
slot of its ring is fetched again and again and the halves of its sums alternate,
against fp64 on the device.  Bars as in test_gpu_add_norm.py; codes are those of the
fp32 values, bit for bit: of an fp32 call's h, by the quantisation.
"""
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -25}
P, SEED, OFFSET, EPS = 0.25, 0x123456789ABCDEF0, (3 << 33) + 5, 1e-6


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    h = dm.Handle(0)
    yield h
    h.close()


def factors(rows, cols):
    """0 or 1 / (1 - p) of every element, from Philox4x32-10 in integers of 64 bits."""
    low, groups = 0xFFFFFFFF, -(-cols // 8)
    at = torch.arange(rows * groups, device="cuda")
    c = [at % groups, at // groups, torch.full_like(at, OFFSET & low), torch.full_like(at, OFFSET >> 32)]
    k0, k1 = SEED & low, SEED >> 32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32 & low) ^ c[1] ^ k0, b & low, (a >> 32 & low) ^ c[3] ^ k1, a & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack(c, -1)
    bits = torch.stack((words & 0xFFFF, words >> 16), -1).view(rows, groups * 8)[:, :cols]
    cut = int(P * 65536)
    return (bits >= cut) * (65536 / (65536 - cut))


def buffer(rows, cols, dtype, odd):
    t = torch.full((rows, cols + (5 if odd else 0)), 7.0, dtype=dtype, device="cuda")
    return t[:, 1:1 + cols] if odd else t


def untouched(t, cols):
    return t._base is None or bool((t._base[:, 0] == 7).all() and (t._base[:, 1 + cols:] == 7).all())


# Five rows a unit at least on up to 160 SMs: part of a warp, a warp, three warps, eight, sixteen, 32 columns a thread.
@pytest.mark.parametrize("rows,cols", [(160000, 33), (160000, 64), (24000, 512), (8000, 1111), (3000, 4096), (1000, 8192), (2000, 9001), (900, 16384)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("odd", [False, True])
def test_many_rows(handle, rows, cols, dtype, odd):
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    dt, u, tiny = DT[dtype], HALF[dtype], TINY[dtype]

    def act():
        v = buffer(rows, cols, dt, odd)
        v.copy_(torch.randn((rows, cols), device="cuda", generator=gen) * torch.exp(torch.randn((rows, 1), device="cuda", generator=gen)))
        return v
    x, f, dy, dh = act(), act(), act(), act()
    w = 1 + 0.3 * torch.randn(cols, device="cuda", generator=gen)
    w64, keep = w.double(), factors(rows, cols)
    drop = dict(p=P, seed=SEED, offset=OFFSET)

    dropped = f.double() * keep
    y64 = x.double() + dropped
    r64 = (y64.square().mean(1, keepdim=True) + EPS).rsqrt()
    ybar = 2.0 ** -23 * (dropped.abs() + y64.abs() + x.double().abs())
    y, h, rstd, q = buffer(rows, cols, dt, odd), buffer(rows, cols, dt, odd), torch.empty(rows, device="cuda"), dm.dmuon_mxfp8_empty(rows, cols)
    handle.add_norm_forward(x, f, w, y, rstd, out=h, q=q, eps=EPS, **drop)
    assert ((y.double() - y64).abs() <= ybar * (1 + u) + u * y64.abs() + tiny).all()
    assert ((rstd.double() - r64[:, 0]).abs() <= 2.0 ** -18 * r64[:, 0]).all()
    want = y64 * r64 * w64
    assert ((h.double() - want).abs() <= (2.0 ** -17 * want.abs() + ybar * r64 * w64.abs()) * (1 + u) + u * want.abs() + tiny).all()
    assert untouched(y, cols) and untouched(h, cols)
    wide, codes = torch.empty((rows, cols), device="cuda"), dm.dmuon_mxfp8_empty(rows, cols)
    handle.add_norm_forward(x.float(), f.float(), w, torch.empty_like(wide), torch.empty_like(rstd), out=wide, eps=EPS, **drop)
    handle.mxfp8_quantize(wide, by_rows=codes)
    assert torch.equal(h, wide.to(dt)) and torch.equal(q[0], codes[0]) and torch.equal(q[1], codes[1])

    dx, df, dw = buffer(rows, cols, dt, odd), buffer(rows, cols, dt, odd), torch.empty(cols, device="cuda")
    handle.add_norm_backward(dy, dh, y, w, rstd, dx, df, dw, **drop)
    r = rstd.double()[:, None]
    yn, into = y.double() * r, dh.double() * w64
    want = dy.double() + r * (into - yn * (into * yn).mean(1, keepdim=True))
    bar = 2.0 ** -17 * (dy.double().abs() + r * (into.abs() + yn.abs() * (into * yn).abs().mean(1, keepdim=True)))
    assert ((dx.double() - want).abs() <= bar * (1 + u) + u * want.abs() + tiny).all()
    assert ((df.double() - want * keep).abs() <= bar * keep * (1 + u) + u * (want * keep).abs() + tiny).all()
    assert untouched(dx, cols) and untouched(df, cols)
    terms = dh.double() * yn
    assert ((dw.double() - terms.sum(0)).abs() <= (2.0 ** -20 + rows * 2.0 ** -23) * terms.abs().sum(0)).all()
    assert handle.status()[0] == 0
