"""Waits that run out inside the Newton-Schulz kernels, on every tile kind and
backend and with few and many K blocks: the status says so, nothing stays in
flight, and the next step gives the bits of a step that never timed out."""
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shapes", [[(200, 200)], [(384, 200), (200, 640)], [(1100, 700), (300, 2000), (640, 640)]])
@pytest.mark.parametrize("tiles,fused,backend", [(1, 0, "direct"), (1, 1, "direct"), (2, 0, "direct"), (2, 1, "direct"),
                                                 (3, 0, "direct"), (3, 1, "direct"), (2, 2, "gram")])
def test_step(shapes, tiles, fused, backend):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    gen = torch.Generator().manual_seed(len(shapes))
    lists = [[torch.randn(s, generator=gen) for s in shapes] for _ in range(3)]
    with dm.Handle(0) as h:
        dm.dmuon_set_tile_mode(h.h, tiles)
        dm.dmuon_set_fused_phases(h.h, fused)

        def step():
            W, G, M = ([t.cuda() for t in x] for x in lists)
            h.step(W, G, M, backend=backend)
            return h.status(len(shapes))[0], W + M
        code, want = step()
        assert code == 0
        for _ in range(6):
            dm.dmuon_set_wait_timeout(h.h, 1)
            assert step()[0] in (0, -6)
            dm.dmuon_set_wait_timeout(h.h, 0)
            code, got = step()
            assert code == 0 and all(torch.equal(a, b) for a, b in zip(got, want))
