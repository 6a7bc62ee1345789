"""Waits of the projection that run out: under a limit of one nanosecond a wait gives up
unless what it waits for is there at the first look.  The operands here do not fit L2
together with what came before, so the first stage never is: the status has to say so,
for both formats and every kind of tile, and the next call is right."""
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402

pytestmark = pytest.mark.gpu

TIMEOUT = -6


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    with dm.Handle(0) as h:
        yield h


# 32 columns of the MMA whole and split, 64 split, 128 split and whole, CTA pairs.
@pytest.mark.parametrize("m,n,k", [(9, 30000, 9000), (1, 8192, 32768), (50, 8192, 32768), (300, 600, 262144), (300, 3840, 40000), (2100, 2600, 60000)])
@pytest.mark.parametrize("bits", [8, 4])
def test_late_and_right_again(handle, m, n, k, bits):
    quantize, empty = (handle.mxfp8_quantize, dm.dmuon_mxfp8_empty) if bits == 8 else (handle.mxfp4_quantize, dm.dmuon_mxfp4_empty)
    gen = torch.Generator(device="cuda").manual_seed(k)
    a, b = empty(m, k), empty(n, k)
    quantize(torch.randn((m, k), device="cuda", generator=gen), a)
    quantize(torch.randn((n, k), device="cuda", generator=gen), b)
    want, out = (torch.full((m, n), 7.0, device="cuda") for _ in range(2))
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    handle.mx_linear(a, b, want, k, act="silu", bits=bits)
    assert handle.status()[0] == 0
    late = 0
    for _ in range(5):
        dm.dmuon_set_wait_timeout(handle.h, 1)
        flush.fill_(1)
        handle.mx_linear(a, b, out, k, act="silu", bits=bits)
        code = handle.status()[0]
        assert code in (0, TIMEOUT)
        late += code == TIMEOUT
        dm.dmuon_set_wait_timeout(handle.h, 0)
        out.fill_(7.0)
        handle.mx_linear(a, b, out, k, act="silu", bits=bits)
        assert handle.status()[0] == 0 and torch.equal(out, want)
    assert late
