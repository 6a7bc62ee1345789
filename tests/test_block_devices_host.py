"""Tensors of another device than the handle's are refused by the binding before
anything is launched (stand-ins for tensors and handles: no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402


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


@pytest.fixture(autouse=True)
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
    return (On(index, rows, nb * 16, dtype=torch.uint8), On(index, -(-rows // 128) * -(-nb // 4) * 512, dtype=torch.uint8))


CALLS = {
    "quantize": (dm.dmuon_mxfp4_quantize, lambda i: dict(src=On(i, 8, 64), by_rows=mx(i, 8, 64), by_cols=mx(i, 64, 8),
                                                         noise=On(i, 8, 64, dtype=torch.uint8))),
    "dequantize": (dm.dmuon_mxfp4_dequantize, lambda i: dict(q=mx(i, 8, 64), out=On(i, 8, 64))),
    "gemm": (dm.dmuon_mxfp4_gemm, lambda i: dict(a=mx(i, 8, 64), b=mx(i, 4, 64), out=On(i, 8, 4), k=64)),
    "forward": (dm.dmuon_block_norm_forward, lambda i: dict(
        x=On(i, 8, 64), f=On(i, 8, 64), post_w=On(i, 64), pre_w=On(i, 64), y=On(i, 8, 64), out=On(i, 8, 64), rstd=On(i, 2, 8),
        gate=On(i, 1, 64), res_scale=On(i, 64))),
    "backward": (dm.dmuon_block_norm_backward, lambda i: dict(
        dy=On(i, 8, 64), dh=On(i, 8, 64), x=On(i, 8, 64), f=On(i, 8, 64), y=On(i, 8, 64), post_w=On(i, 64), pre_w=On(i, 64),
        rstd=On(i, 2, 8), dx=On(i, 8, 64), df=On(i, 8, 64), d_post_w=On(i, 64), d_pre_w=On(i, 64), gate=On(i, 1, 64),
        d_gate=On(i, 1, 64), res_scale=On(i, 64), d_res_scale=On(i, 64))),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("device", [0, 1])
def test_all_on_the_handles_device(name, device):
    call, args = CALLS[name]
    with pytest.raises(Launched):
        call(HandleOn(device), **args(device))


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("device,index", [(0, 1), (1, 0), (0, -1)])
def test_all_on_another_device(name, device, index):
    call, args = CALLS[name]
    with pytest.raises(ValueError):
        call(HandleOn(device), **args(index))


@pytest.mark.parametrize("name,arg", [(n, a) for n, (_, args) in CALLS.items() for a in args(0) if a != "k"])
@pytest.mark.parametrize("index", [1, -1])
def test_one_on_another_device(name, arg, index):
    call, args = CALLS[name]
    with pytest.raises(ValueError):
        call(HandleOn(0), **dict(args(0), **{arg: args(index)[arg]}))


@pytest.mark.parametrize("part", [0, 1])
def test_codes_and_scales_on_two_devices(part):
    q = list(mx(0, 8, 64))
    q[part] = mx(1, 8, 64)[part]
    with pytest.raises(ValueError):
        dm.dmuon_mxfp4_quantize(HandleOn(0), On(0, 8, 64), by_rows=q)


def test_a_handle_that_does_not_tell_takes_the_first_tensors_device():
    with pytest.raises(Launched):
        dm.dmuon_mxfp4_quantize(None, On(1, 8, 64), by_rows=mx(1, 8, 64))
    with pytest.raises(ValueError):
        dm.dmuon_mxfp4_quantize(None, On(1, 8, 64), by_rows=mx(0, 8, 64))
