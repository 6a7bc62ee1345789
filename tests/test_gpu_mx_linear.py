"""The projection with its epilogue against fp64.

z's bar per element is (33 blocks 2^-23 + 2^-22) sum_k |a_k b_k| + 2^-23 |z|: an
instruction adds 32 products of at most 8 bits and the sum so far, each cut below
2^-23 of the largest of them, and alpha and the bias cost a rounding each.
Small whole numbers add up exactly, so there the bar is 0 and every place of
codes and scales counts.  An activation passes z's error on with a slope below
1.13 and adds 2^-21 (2 + |u|) of its value (u the exponent it takes: a rounding
or two of u, exp2 and reciprocal within 2^-22 each, the fitted erfcx 5e-7).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402
from oracle import mxfp4, mxfp8  # noqa: E402
from oracle import projection as op  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
ORACLE = {4: mxfp4, 8: mxfp8}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    h = dm.Handle(0)
    yield h
    h.close()


def operand(x, bits):
    """(device matrix, the values it stands for)."""
    o = ORACLE[bits]
    codes, byte = o.quantize(x)
    data, scales = o.pack(codes, byte)
    return (torch.from_numpy(data).cuda(), torch.from_numpy(scales).cuda()), o.values(codes, byte, x.shape[1])


def buffer(m, n, dtype, odd, fill=7.0):
    t = torch.full((m, n + (5 if odd else 0)), fill, dtype=DT[dtype], device="cuda")
    return t[:, 1:1 + n] if odd else t


def act_bar(z, act):
    u = {"none": 0 * z, "relu": 0 * z, "gelu": z * z / 2}.get(act)
    if u is None:
        u = op.inner(z, act)[0]
    return 2.0 ** -21 * (2 + np.minimum(np.abs(u), 100)) * np.abs(op.activation(z, act)) + 2.0 ** -120


# One CTA a tile with few rows of A; K split 2, 4 and 8 ways; 64 and 128 rows; CTA pairs.
SIZES = [(1, 1, 1), (1, 4096, 333), (1, 300, 14336), (2, 1000, 4100), (3, 129, 2061), (4, 33, 6000), (5, 600, 4096), (8, 200, 2080), (9, 600, 4096), (33, 257, 96), (50, 1111, 640), (77, 300, 31), (128, 128, 129),
         (200, 130, 1024), (300, 264, 64), (257, 1000, 4097), (2100, 2600, 1300), (2560, 2304, 257)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("odd", [False, True])
def test_whole_numbers_are_exact(handle, m, n, k, bits, odd):
    """Codes 0, 1, 2 with a sign and scales 1, 2, 4 (|sum| < 2^24)."""
    r = np.random.RandomState(m + n + k)

    def whole(rows):
        x = r.randint(-2, 3, (rows, k)).astype(np.float64) * 2.0 ** r.randint(0, 3, (rows, 1))
        x[:, ::32] = np.where(r.rand(rows, x[:, ::32].shape[1]) < 0.5, 0, x[:, ::32])
        return x
    (a, av), (b, bv) = operand(whole(m), bits), operand(whole(n), bits)
    bias = r.randint(-50, 51, n).astype(np.float64)
    res = r.randint(-50, 51, (m, n)).astype(np.float64)
    z = torch.from_numpy(av) @ torch.from_numpy(bv).t() + torch.from_numpy(bias)
    assert z.abs().max() < 2 ** 24
    out, pre, c = buffer(m, n, "f32", odd), buffer(m, n, "f32", odd), buffer(m, n, "f32", odd)
    c.copy_(torch.from_numpy(res))
    handle.mx_linear(a, b, out, k, bias=torch.from_numpy(bias).float().cuda(), act="relu", pre=pre, residual=c, beta=-1.0, bits=bits)
    assert torch.equal(pre.cpu().double(), z)
    assert torch.equal(out.cpu().double(), z.clamp(min=0) - torch.from_numpy(res))
    handle.mx_linear(a, b, out, k, alpha=2.0, bits=bits)
    assert torch.equal(out.cpu().double(), 2 * (z - torch.from_numpy(bias)))
    handle.mx_linear(a, b, out, k, residual=out, bits=bits)  # in place
    assert torch.equal(out.cpu().double(), 3 * (z - torch.from_numpy(bias)))
    for t in (out, pre):
        if odd:
            assert (t._base[:, 0] == 7).all() and (t._base[:, 1 + n:] == 7).all()
    assert handle.status()[0] == 0


@pytest.mark.parametrize("m,n,k", [(1, 4096, 333), (2, 100, 9000), (3, 129, 2061), (4, 700, 1024), (8, 55, 300), (9, 300, 3000), (50, 1111, 640), (200, 130, 1024), (257, 1000, 4097), (2100, 2600, 300)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bits,act,with_bias,with_res,odd", [(8, "none", True, True, False), (8, "relu", False, False, True),
                                                             (8, "silu", True, True, True), (8, "gelu", True, False, False),
                                                             (8, "gelu_tanh", False, True, False), (4, "gelu_tanh", True, True, True),
                                                             (4, "silu", False, False, False)])
def test_against_fp64(handle, m, n, k, dtype, bits, act, with_bias, with_res, odd):
    r = np.random.RandomState(m + 3 * n + k)
    (a, av), (b, bv) = operand(r.randn(m, k) * np.exp(0.5 * r.randn(m, 1)), bits), operand(1.5 * r.randn(n, k) / k ** 0.5, bits)
    bias = np.float32(0.3 * r.randn(n)).astype(np.float64) if with_bias else np.zeros(n)
    res = torch.from_numpy(r.randn(m, n)).to(DT[dtype]) if with_res else None
    alpha, beta = 0.75, 1.25
    ta, tb = torch.from_numpy(av), torch.from_numpy(bv).t()
    z = alpha * (ta @ tb).numpy() + bias
    bar = (33 * -(-k // 32) * 2.0 ** -23 + 2.0 ** -22) * alpha * (ta.abs() @ tb.abs()).numpy() + 2.0 ** -23 * np.abs(z)
    out, pre = buffer(m, n, dtype, odd), buffer(m, n, dtype, odd)
    c = None
    if with_res:
        c = buffer(m, n, dtype, odd)
        c.copy_(res)
    handle.mx_linear(a, b, out, k, bias=torch.from_numpy(bias).float().cuda() if with_bias else None, act=act, pre=pre, residual=c,
                     alpha=alpha, beta=beta, bits=bits)
    u = HALF[dtype]
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0  # half a subnormal step
    assert (np.abs(pre.cpu().double().numpy() - z) <= bar * (1 + u) + u * np.abs(z) + tiny).all()
    add = beta * res.double().numpy() if with_res else 0.0
    want = op.activation(z, act) + add
    wide = 1.13 * bar + act_bar(z, act) + 2.0 ** -23 * np.abs(want)
    assert (np.abs(out.cpu().double().numpy() - want) <= wide * (1 + u) + u * np.abs(want) + tiny).all()
    again = buffer(m, n, dtype, odd)
    handle.mx_linear(a, b, again, k, bias=torch.from_numpy(bias).float().cuda() if with_bias else None, act=act, residual=c, alpha=alpha,
                     beta=beta, bits=bits)
    assert torch.equal(again, out)
    assert handle.status()[0] == 0


@pytest.mark.parametrize("act", ACTS)
def test_activation_far_out(handle, act):
    """z over many sizes by the bias alone, to infinity and NaN."""
    z = np.concatenate([np.linspace(-14, 14, 2001), np.array([0.0, -0.0, 40, -40, 90, -90, 1e4, -1e4, 3e9, -3e9, 1e30, -1e30, 3e38])])
    z = np.float32(z).astype(np.float64)
    n = len(z)
    (a, _), (b, _) = operand(np.zeros((2, 32)), 8), operand(np.zeros((n, 32)), 8)
    out, pre = buffer(2, n, "f32", False), buffer(2, n, "f32", False)
    handle.mx_linear(a, b, out, 32, bias=torch.from_numpy(z).float().cuda(), act=act, pre=pre)
    assert torch.equal(pre[1].cpu().double(), torch.from_numpy(z))
    want = op.activation(np.where(np.abs(z) > 1e4, 0, z), act)
    want = np.where(np.abs(z) > 1e4, np.where(z > 0, z, z if act == "none" else 0.0), want)
    got = out[0].cpu().double().numpy()
    assert (np.abs(got - want) <= np.where(np.abs(z) > 1e4, 0, act_bar(np.clip(z, -1e4, 1e4), act)) + 2.0 ** -23 * np.abs(want)).all()
    special = torch.tensor([float("inf"), float("nan")], device="cuda")
    (b2, _), out2 = operand(np.zeros((2, 32)), 8), buffer(1, 2, "f32", False)
    (a1, _) = operand(np.zeros((1, 32)), 8)
    handle.mx_linear(a1, b2, out2, 32, bias=special, act=act)
    assert out2[0, 0] == float("inf") and torch.isnan(out2[0, 1])


def test_no_rows_of_k_and_empty(handle):
    out, bias = buffer(3, 5, "f32", False), torch.arange(5, device="cuda", dtype=torch.float32)
    for make, bits in ((dm.dmuon_mxfp8_empty, 8), (dm.dmuon_mxfp4_empty, 4)):
        out.fill_(7.0)
        handle.mx_linear(make(3, 0), make(5, 0), out, 0, bias=bias, bits=bits)
        assert torch.equal(out, bias.expand(3, 5))
    for m, n in ((0, 5), (3, 0)):
        handle.mx_linear(dm.dmuon_mxfp8_empty(m, 64), dm.dmuon_mxfp8_empty(n, 64), torch.empty((m, n), device="cuda"), 64)


def test_a_residual_of_no_weight_is_not_read(handle):
    a, b = dm.dmuon_mxfp8_empty(3, 64), dm.dmuon_mxfp8_empty(200, 64)
    handle.mxfp8_quantize(torch.randn(3, 64, device="cuda"), a)
    handle.mxfp8_quantize(torch.randn(200, 64, device="cuda"), b)
    out, want = buffer(3, 200, "f32", False, float("nan")), buffer(3, 200, "f32", False)
    handle.mx_linear(a, b, want, 64)
    handle.mx_linear(a, b, out, 64, residual=out, beta=0.0)
    assert torch.equal(out, want)


def test_refusals(handle):
    a, b, a4 = dm.dmuon_mxfp8_empty(8, 64), dm.dmuon_mxfp8_empty(16, 64), dm.dmuon_mxfp4_empty(8, 64)
    out = torch.zeros((8, 16), device="cuda")
    for bad in (dict(a=a4), dict(bias=torch.zeros(15, device="cuda")), dict(bias=torch.zeros(16, device="cuda").half()),
                dict(pre=torch.zeros((8, 16), device="cuda").half()), dict(residual=torch.zeros((8, 15), device="cuda")), dict(k=128), dict(bits=4), dict(bits=6)):
        with pytest.raises(ValueError):
            handle.mx_linear(**dict(dict(a=a, b=b, out=out, k=64), **bad))
    with pytest.raises(KeyError):
        handle.mx_linear(a, b, out, 64, act="tanh")
    wide = torch.zeros((8, 32), device="cuda")
    for bad in (dict(pre=out), dict(alpha=float("nan")), dict(beta=float("inf")), dict(out=wide[:, :16], residual=wide.view(16, 16)[:8])):
        with pytest.raises(dm.DmuonError):
            handle.mx_linear(**dict(dict(a=a, b=b, out=out, k=64), **bad))
    assert not out.any()


@pytest.mark.parametrize("m,n,k", [(9, 30000, 4500), (300, 600, 600), (9, 4096, 4096), (2100, 2600, 650), (2100, 2600, 2500)])
def test_waits_that_run_out(handle, m, n, k):
    r = np.random.RandomState(1)
    a, b = dm.dmuon_mxfp8_empty(m, k), dm.dmuon_mxfp8_empty(n, k)
    handle.mxfp8_quantize(torch.from_numpy(r.randn(m, k)).float().cuda(), a)
    handle.mxfp8_quantize(torch.from_numpy(r.randn(n, k)).float().cuda(), b)
    want, out = (torch.full((m, n), 7.0, device="cuda") for _ in range(2))
    handle.mx_linear(a, b, want, k, act="silu")
    assert handle.status()[0] == 0
    for _ in range(6):
        dm.dmuon_set_wait_timeout(handle.h, 1)
        handle.mx_linear(a, b, out, k, act="silu")
        late = handle.status()[0]
        assert late in (0, -6) and (late or torch.equal(out, want))
        dm.dmuon_set_wait_timeout(handle.h, 0)
        out.fill_(7.0)
        handle.mx_linear(a, b, out, k, act="silu")
        assert handle.status()[0] == 0 and torch.equal(out, want)
