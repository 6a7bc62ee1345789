"""Host side of the operators around an 8-bit projection (no GPU needed): sizes,
refusals that come before any device work, tensors of another device."""
import ctypes
import os
import re

import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return dm.load()


@pytest.mark.parametrize("rows,k", [(0, 0), (0, 64), (64, 0), (1, 1), (1, 33), (129, 129), (777, 2061), (1 << 30, 1 << 30)])
def test_mxfp8_bytes(lib, rows, k):
    assert dm.dmuon_mxfp8_bytes(rows, k) == (rows * -(-k // 32) * 32, -(-rows // 128) * -(-k // 128) * 512)


@pytest.mark.parametrize("rows,k", [(-1, 4), (4, -1), ((1 << 30) + 1, 4), (4, (1 << 30) + 1)])
def test_mxfp8_bytes_refusals(lib, rows, k):
    with pytest.raises(dm.DmuonError):
        dm.dmuon_mxfp8_bytes(rows, k)
    assert lib.dmuon_mxfp8_bytes(4, 64, None, None) == 0


def test_null_handle_is_refused(lib):
    assert lib.dmuon_mxfp8_quantize(None, None, 0, 4, 4, 4, 0, None, None, None, None, None) == -1
    assert lib.dmuon_mxfp8_dequantize(None, None, None, 4, 4, None, 0, 4, None) == -1
    assert lib.dmuon_mx_linear(None, dm.MxLinear(), None) == -1
    assert lib.dmuon_act_backward(None, dm.ActBackward(), None) == -1
    assert lib.dmuon_add_norm_forward(None, dm.AddNorm(), None) == -1
    assert lib.dmuon_add_norm_backward(None, dm.AddNorm(), dm.AddNormGrad(), None) == -1
    assert lib.dmuon_dropout(None, None, 0, 4, 4, 4, None, 0, None, 4, 0.5, 1, 0, None) == -1


def test_kinds_and_activations_match_the_header(lib):
    src = open(os.path.join(ROOT, "include", "dmuon.h")).read()
    kinds = dict((int(v), k) for k, v in re.findall(r"#define DMUON_KIND_(\w+)\s+(\d+)", src))
    assert [kinds[i] for i in range(17, 21)] == ["ACT_BWD", "ADD_NORM_FWD", "ADD_NORM_BWD", "DROPOUT"]
    assert [n.upper() for n in dm.KIND_NAMES[17:]] == [kinds[i] for i in range(17, 21)]
    assert {k.lower(): int(v) for k, v in re.findall(r"#define DMUON_ACT_(\w+)\s+(\d+)", src)} == dm.ACTIVATIONS


class On:
    """What the binding reads of a tensor, on device `index`."""

    def __init__(self, index, *shape, dtype=torch.float32):
        self.index, self.shape, self.dtype, self.is_cuda = index, torch.Size(shape), dtype, index >= 0

    def get_device(self):
        return self.index

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return (self.shape[-1], 1)[-len(self.shape):]

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


class HandleOn:
    def __init__(self, device):
        self.device = device


class Launched(Exception):
    pass


@pytest.fixture
def no_library(monkeypatch):
    class Library:
        def __getattr__(self, name):
            def call(*args):
                raise Launched(name)
            return call
    monkeypatch.setattr(dm, "load", lambda path=None: Library())
    monkeypatch.setattr(dm, "_raw_stream", lambda index: index)


def mx(index, rows, k):
    nb = -(-k // 32)
    return (On(index, rows, nb * 32, dtype=torch.uint8), On(index, -(-rows // 128) * -(-nb // 4) * 512, dtype=torch.uint8))


CALLS = {
    "quantize": (dm.dmuon_mxfp8_quantize, lambda i: dict(src=On(i, 8, 64), by_rows=mx(i, 8, 64), by_cols=mx(i, 64, 8))),
    "dequantize": (dm.dmuon_mxfp8_dequantize, lambda i: dict(q=mx(i, 8, 64), out=On(i, 8, 64))),
    "linear": (dm.dmuon_mx_linear, lambda i: dict(a=mx(i, 8, 64), b=mx(i, 4, 64), out=On(i, 8, 4), k=64, bias=On(i, 4), pre=On(i, 8, 4),
                                                  residual=On(i, 8, 4))),
    "act_backward": (dm.dmuon_act_backward, lambda i: dict(dout=On(i, 8, 64), pre=On(i, 8, 64), act="silu", dz=On(i, 8, 64), d_bias=On(i, 64),
                                                           by_rows=mx(i, 8, 64), by_cols=mx(i, 64, 8))),
    "add_norm_forward": (dm.dmuon_add_norm_forward, lambda i: dict(x=On(i, 8, 64), f=On(i, 8, 64), w=On(i, 64), y=On(i, 8, 64), rstd=On(i, 8),
                                                                   out=On(i, 8, 64), q=mx(i, 8, 64))),
    "add_norm_backward": (dm.dmuon_add_norm_backward, lambda i: dict(dy=On(i, 8, 64), dh=On(i, 8, 64), y=On(i, 8, 64), w=On(i, 64), rstd=On(i, 8),
                                                                     dx=On(i, 8, 64), df=On(i, 8, 64), d_w=On(i, 64))),
    "dropout": (dm.dmuon_dropout, lambda i: dict(x=On(i, 8, 64), out=On(i, 8, 64), p=0.5, seed=1, residual=On(i, 8, 64))),
}
TENSORS = [(n, a) for n, (_, args) in CALLS.items() for a in args(0) if a not in ("k", "act", "p", "seed")]


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("device", [0, 1])
def test_all_on_the_handles_device(no_library, name, device):
    call, args = CALLS[name]
    with pytest.raises(Launched):
        call(HandleOn(device), **args(device))
    with pytest.raises(Launched):  # and by the first tensor's, for a handle that does not tell
        call(None, **args(device))


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("device,index", [(0, 1), (1, 0), (0, -1)])
def test_all_on_another_device(no_library, name, device, index):
    call, args = CALLS[name]
    with pytest.raises(ValueError):
        call(HandleOn(device), **args(index))


@pytest.mark.parametrize("name,arg", TENSORS)
@pytest.mark.parametrize("index", [1, -1])
def test_one_on_another_device(no_library, name, arg, index):
    call, args = CALLS[name]
    with pytest.raises(ValueError):
        call(HandleOn(0), **dict(args(0), **{arg: args(index)[arg]}))


@pytest.mark.parametrize("name", ["add_norm_forward", "add_norm_backward", "dropout"])
@pytest.mark.parametrize("bad", [dict(seed=-1), dict(seed=1 << 64), dict(offset=-1), dict(offset=1 << 64)])
def test_seeds_and_offsets_have_64_bits(no_library, name, bad):
    call, args = CALLS[name]
    with pytest.raises(ValueError):
        call(HandleOn(0), **dict(args(0), **bad))


def test_structures_match_the_header(tmp_path):
    """The sizes and last fields' offsets that the compiler sees."""
    import subprocess
    names = {"MxLinear": ("dmuon_mx_linear_t", "ldd"), "ActBackward": ("dmuon_act_backward_t", "col_scales"),
             "AddNorm": ("dmuon_add_norm_t", "rstd"), "AddNormGrad": ("dmuon_add_norm_grad_t", "d_w")}
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "dmuon.h"\nint main(void) {\n' + "".join(
        'printf("%%zu %%zu\\n", sizeof(%s), offsetof(%s, %s));\n' % (t, t, f) for t, f in names.values()) + "return 0; }\n")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    for (cls, (_, last)), size, at in zip(names.items(), lines[::2], lines[1::2]):
        c = getattr(dm, cls)
        assert ctypes.sizeof(c) == int(size) and getattr(c, last).offset == int(at)
