"""Each matrix of a call at a distance of its own from a 16-byte boundary and with a
pitch of its own: the same bits as from matrices that are whole, and nothing written
beside the rows.  Projections, whose epilogue may round in another order, get whole
numbers."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
DROP = dict(p=0.25, seed=5, offset=9)


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    h = dm.Handle(0)
    yield h
    h.close()


class Places:
    """Matrices in larger buffers of 7s, the ith i + shift elements off and i + shift + extra apart."""

    def __init__(self, shift, extra):
        self.shift, self.extra, self.all = shift, extra, []

    def __call__(self, like):
        if like is None:
            return None
        rows, cols = like.shape
        off = len(self.all) * 3 + self.shift
        pitch = cols + off + self.extra + 2 * len(self.all)
        buf = torch.full((rows * pitch + 64,), 7.0, dtype=like.dtype, device="cuda")
        v = torch.as_strided(buf, (rows, cols), (pitch, 1), off)
        v.copy_(like)
        self.all.append((buf, v))
        return v

    def check(self):
        for buf, v in self.all:
            v.fill_(7.0)
            assert (buf == 7).all()


SHAPES = [(5, 33), (130, 100), (40, 300), (37, 777), (20, 4099), (9, 9000), (3, 17000)]
PLACES = [(0, 0), (1, 0), (3, 2), (6, 1)]


def rand(shape, dtype, seed):
    return torch.randn(shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).to(DT[dtype])


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shift,extra", PLACES)
def test_norm_and_dropout(handle, shape, dtype, shift, extra):
    rows, cols = shape
    x, f, dy, dh = (rand(shape, dtype, i) for i in range(4))
    w = 1 + 0.1 * torch.randn(cols + 1, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9))
    want = [torch.empty_like(x) for _ in range(5)]
    rstd, dw, q = torch.empty(rows, device="cuda"), torch.empty(cols, device="cuda"), dm.dmuon_mxfp8_empty(rows, cols)
    handle.add_norm_forward(x, f, w[:-1].clone(), want[0], rstd, out=want[1], q=q, **DROP)
    handle.add_norm_backward(dy, dh, want[0], w[:-1].clone(), rstd, want[2], want[3], dw, **DROP)
    handle.dropout(x, want[4], residual=f, **DROP)
    at = Places(shift, extra)
    xs, fs, dys, dhs = at(x), at(f), at(dy), at(dh)
    out = [at(torch.zeros_like(x)) for _ in range(5)]
    w2 = torch.empty(cols + 1, device="cuda")[1:] if shift & 1 else torch.empty(cols, device="cuda")
    w2.copy_(w[:-1])
    rstd2, q2 = torch.empty(rows + 1, device="cuda")[1:], dm.dmuon_mxfp8_empty(rows, cols)
    dw2 = torch.empty(cols + 1, device="cuda")[1:]
    handle.add_norm_forward(xs, fs, w2, out[0], rstd2, out=out[1], q=q2, **DROP)
    handle.add_norm_backward(dys, dhs, out[0], w2, rstd2, out[2], out[3], dw2, **DROP)
    handle.dropout(xs, out[4], residual=fs, **DROP)
    for got, ref in zip(out + [rstd2, dw2, *q2], want + [rstd, dw, *q]):
        assert torch.equal(got, ref)
    at.check()
    assert handle.status()[0] == 0


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shift,extra", PLACES)
def test_act_backward(handle, shape, dtype, shift, extra):
    rows, cols = shape
    dout, pre = rand(shape, dtype, 1), rand(shape, dtype, 2)
    dz, db, q, qt = torch.empty_like(dout), torch.empty(cols, device="cuda"), dm.dmuon_mxfp8_empty(rows, cols), dm.dmuon_mxfp8_empty(cols, rows)
    handle.act_backward(dout, pre, "gelu", dz=dz, d_bias=db, by_rows=q, by_cols=qt)
    back = torch.empty_like(dout)
    handle.mxfp8_dequantize(q, back)
    at = Places(shift, extra)
    dout2, pre2, dz2, back2 = at(dout), at(pre), at(torch.zeros_like(dout)), at(torch.zeros_like(dout))
    db2, q2, qt2 = torch.empty(cols + 1, device="cuda")[1:], dm.dmuon_mxfp8_empty(rows, cols), dm.dmuon_mxfp8_empty(cols, rows)
    handle.act_backward(dout2, pre2, "gelu", dz=dz2, d_bias=db2, by_rows=q2, by_cols=qt2)
    handle.mxfp8_dequantize(q2, back2)
    for got, ref in zip([dz2, db2, back2, *q2, *qt2], [dz, db, back, *q, *qt]):
        assert torch.equal(got, ref)
    at.check()


# Whole, split 2, 4 and 8 ways; A of few and of many rows, B of few and of many; CTA pairs.
@pytest.mark.parametrize("m,n,k", [(3, 129, 300), (5, 600, 4096), (50, 333, 640), (300, 20, 5000), (1000, 64, 4100), (5000, 100, 96), (20000, 1, 100), (513, 7, 64),
                                   (300, 130, 2100), (2100, 2603, 160)])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("moved,dtype", [("out", "f16"), ("pre", "f32"), ("res", "f16"), ("bias", "f32"), ("all", "f32"), ("all", "f16")])
def test_projection(handle, m, n, k, bits, moved, dtype):
    """Codes 0 and 1 with a sign, few enough for fp16's whole numbers to 2048."""
    r = np.random.RandomState(m + n + k)
    quantize, empty = (handle.mxfp8_quantize, dm.dmuon_mxfp8_empty) if bits == 8 else (handle.mxfp4_quantize, dm.dmuon_mxfp4_empty)
    share = min(1.0, 12 / k ** 0.5)
    av, bv = (torch.from_numpy(r.choice([-1.0, 0.0, 1.0], (rows, k), p=[share / 2, 1 - share, share / 2])).cuda() for rows in (m, n))
    a, b = empty(m, k), empty(n, k)
    quantize(av.float(), a)
    quantize(bv.float(), b)
    bias, res = (torch.from_numpy(r.randint(-50, 51, s).astype(np.float64)).cuda() for s in (n, (m, n)))
    z = av @ bv.t() + bias
    assert z.abs().max() < 1900
    at = Places(1, 2)
    place = {name: at if moved in (name, "all") else torch.clone for name in ("out", "pre", "res")}
    out, pre, c = (place[name](t.to(DT[dtype])) for name, t in (("out", 0 * res), ("pre", 0 * res), ("res", res)))
    line = torch.empty(n + 1, device="cuda")[1:] if moved in ("bias", "all") else torch.empty(n, device="cuda")
    line.copy_(bias)
    handle.mx_linear(a, b, out, k, bias=line, act="relu", pre=pre, residual=c, beta=-1.0, bits=bits)
    assert torch.equal(pre.double(), z) and torch.equal(out.double(), z.clamp(min=0) - res)
    at.check()
    assert handle.status()[0] == 0
