"""Host side of the MXFP4 and block-norm entry points (no GPU needed): sizes,
refusals that come before any device work, and the binding's own checks."""
import ctypes
import os
import re

import pytest

import newton_schulz_nesterov_gb300 as dm
from newton_schulz_nesterov_gb300 import _build
from oracle import mxfp4 as om

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return dm.load()


@pytest.mark.parametrize("rows,k", [(0, 0), (0, 64), (64, 0), (1, 1), (1, 32), (1, 33), (128, 128), (129, 129), (777, 2061),
                                    (14336, 4096), (1 << 30, 1 << 30)])
def test_mxfp4_bytes(lib, rows, k):
    data, scales = dm.dmuon_mxfp4_bytes(rows, k)
    assert data == rows * -(-k // 32) * 16
    assert scales == -(-rows // 128) * -(-k // 128) * 512
    if 0 < rows * k < 1 << 24:
        import numpy as np
        d, s = om.pack(*om.quantize(np.zeros((rows, k))))
        assert d.size == data and s.size == scales


@pytest.mark.parametrize("rows,k", [(-1, 4), (4, -1), ((1 << 30) + 1, 4), (4, (1 << 30) + 1)])
def test_mxfp4_bytes_refusals(lib, rows, k):
    with pytest.raises(dm.DmuonError):
        dm.dmuon_mxfp4_bytes(rows, k)


def test_mxfp4_bytes_null_outputs(lib):
    n = ctypes.c_size_t(0)
    assert lib.dmuon_mxfp4_bytes(4, 64, None, None) == 0
    assert lib.dmuon_mxfp4_bytes(4, 64, None, ctypes.byref(n)) == 0 and n.value == 512


def test_null_handle_is_refused(lib):
    assert lib.dmuon_mxfp4_quantize(None, None, 0, 4, 4, 4, 0, None, 0, None, None, None, None, None) == -1
    assert lib.dmuon_mxfp4_dequantize(None, None, None, 4, 4, None, 0, 4, None) == -1
    assert lib.dmuon_mxfp4_gemm(None, None, None, None, None, 4, 4, 4, None, 0, 4, 1.0, 0.0, None) == -1
    p, q = dm.BlockNorm(), dm.BlockNormGrad()
    assert lib.dmuon_block_norm_forward(None, p, None) == -1
    assert lib.dmuon_block_norm_backward(None, p, q, None) == -1


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros((8, 64))
    q = (torch.zeros((8, 32), dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8))
    with pytest.raises(ValueError):
        dm.dmuon_mxfp4_quantize(None, x, by_rows=q)
    with pytest.raises(ValueError):
        dm.dmuon_mxfp4_dequantize(None, q, x)
    with pytest.raises(ValueError):
        dm.dmuon_mxfp4_gemm(None, q, q, torch.zeros((8, 8)), 64)
    w = torch.zeros(64)
    with pytest.raises(ValueError):
        dm.dmuon_block_norm_forward(None, x, x, w, w, x, x, torch.zeros((2, 8)))
    with pytest.raises(ValueError):
        dm.dmuon_block_norm_backward(None, None, x, x, x, x, w, w, torch.zeros((2, 8)), x, x, w, w)


def test_kinds_match_the_header(lib):
    src = open(os.path.join(ROOT, "include", "dmuon.h")).read()
    kinds = dict((int(v), k) for k, v in re.findall(r"#define DMUON_KIND_(\w+)\s+(\d+)", src))
    assert len(dm.KIND_NAMES) == int(re.search(r"#define DMUON_NUM_KINDS\s+(\d+)", src).group(1))
    assert [kinds[i] for i in range(12, 17)] == ["MX_QUANTIZE", "MX_DEQUANTIZE", "MX_GEMM", "NORM_FWD", "NORM_BWD"]
