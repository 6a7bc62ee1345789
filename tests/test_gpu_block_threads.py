"""Handles in different host threads, and one graph of several sizes: no call
depends on the size that another call of the same kernel had."""
import ctypes
import os
import subprocess
import threading

import pytest

torch = pytest.importorskip("torch")

import newton_schulz_nesterov_gb300 as dm  # noqa: E402
from newton_schulz_nesterov_gb300 import _build  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()


def norms(h, rows, cols):
    """One forward and backward on buffers of its own; returns (call, results)."""
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x, f, dy, dh = (torch.randn(rows, cols, device="cuda", generator=gen).bfloat16() for _ in range(4))
    y, out, dx, df = (torch.zeros_like(x) for _ in range(4))
    w = torch.rand(cols, device="cuda", generator=gen) + 0.5
    rstd, sums = torch.zeros((2, rows), device="cuda"), torch.zeros((3, cols), device="cuda")

    def call(stream=None):
        h.block_norm_forward(x, f, w, w, y, out, rstd, res_scale=w, stream=stream)
        h.block_norm_backward(dy, dh, x, f, y, w, w, rstd, dx, df, sums[0], sums[1], res_scale=w, d_res_scale=sums[2], stream=stream)
    return call, [y, out, rstd, dx, df, sums]


def quantise(h, rows, cols):
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(rows, cols, device="cuda", generator=gen).bfloat16()
    q = dm.dmuon_mxfp4_empty(rows, cols)
    return (lambda stream=None: h.mxfp4_quantize(x, q, stream=stream)), list(q)


# Widths of one kernel whose shared memory differs; rows on 16 bytes and not.
# Several threads a width, so that calls meet often.
@pytest.mark.parametrize("make,sizes", [(norms, [(2, 4096), (2, 512)]), (norms, [(2, 9000), (2, 16384)]),
                                        (quantise, [(1, 256), (1, 255)])])
def test_threads_with_a_handle_each(make, sizes):
    errors, results, wanted = [], [], {}
    with dm.Handle(0) as h:
        for s in sizes:
            call, res = make(h, *s)
            call()
            torch.cuda.synchronize()
            wanted[s] = [t.clone() for t in res]
    start = threading.Barrier(4 * len(sizes))

    def work(s):
        try:
            stream = torch.cuda.Stream()
            with dm.Handle(0) as h, torch.cuda.stream(stream):
                call, res = make(h, *s)
                start.wait(60)
                for _ in range(1500):
                    call(stream)
                got = [t.clone() for t in res]
                stream.synchronize()
                results.append((s, got))
                assert h.status()[0] == 0
        except Exception as e:  # noqa: BLE001 -- shown by the assertion below
            errors.append((s, repr(e)))
    threads = [threading.Thread(target=work, args=(s,)) for s in sizes * 4]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for s, got in results:
        for g, w in zip(got, wanted[s]):
            assert torch.equal(g, w)


HAMMER = """
#include <thread>
#include "dmuon.h"
struct Side { dmuon_handle_t h; const void* src; long long rows, cols, ld; void *data, *scales, *stream; int failed; };
extern "C" void hammer(Side* s, int sides, int calls) {
  std::thread t[8];
  for (int i = 0; i < sides; ++i)
    t[i] = std::thread([=] {
      for (int k = 0; k < calls; ++k)
        s[i].failed += dmuon_mxfp4_quantize(s[i].h, s[i].src, DMUON_BF16, s[i].rows, s[i].cols, s[i].ld, 0, nullptr, 0, s[i].data,
                                            s[i].scales, nullptr, nullptr, s[i].stream) != 0;
    });
  for (int i = 0; i < sides; ++i) t[i].join();
}
"""


class Side(ctypes.Structure):
    _fields_ = [("h", ctypes.c_void_p), ("src", ctypes.c_void_p), ("rows", ctypes.c_longlong), ("cols", ctypes.c_longlong),
                ("ld", ctypes.c_longlong), ("data", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("stream", ctypes.c_void_p),
                ("failed", ctypes.c_int)]


def test_native_threads(tmp_path):
    """The same from threads that hold no interpreter lock: rows on 16 bytes and
    not take one kernel with different amounts of shared memory."""
    dm.load()
    (tmp_path / "hammer.cpp").write_text(HAMMER)
    lib = str(tmp_path / "hammer.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-pthread", "-I", _build.INCLUDE, "-o", lib,
                    str(tmp_path / "hammer.cpp"), _build.LIB, "-Wl,-rpath," + os.path.dirname(_build.LIB)], check=True)
    handles = [dm.Handle(0) for _ in range(4)]
    streams = [torch.cuda.Stream() for _ in handles]
    sides, kept = (Side * 4)(), []
    for i, (h, st) in enumerate(zip(handles, streams)):
        cols = 256 - i % 2
        x, q = torch.randn((64, cols), device="cuda").bfloat16(), dm.dmuon_mxfp4_empty(64, cols)
        kept.append((x, q))
        sides[i] = Side(h.h, x.data_ptr(), 64, cols, cols, q[0].data_ptr(), q[1].data_ptr(), st.cuda_stream, 0)
    torch.cuda.synchronize()
    ctypes.CDLL(lib).hammer(sides, 4, 5000)
    torch.cuda.synchronize()
    assert [s.failed for s in sides] == [0] * 4
    for h in handles:
        h.close()


def test_large_and_small_in_one_graph():
    with dm.Handle(0) as h:
        runs = [norms(h, 40, 4096), norms(h, 40, 512), quantise(h, 64, 255), quantise(h, 64, 256)]
        for call, _ in runs:
            call()
        torch.cuda.synchronize()
        want = [[t.clone() for t in res] for _, res in runs]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for call, _ in runs:
                call()
        for _, res in runs:
            for t in res:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for (_, res), ref in zip(runs, want):
            for got, w in zip(res, ref):
                assert torch.equal(got, w)
        assert h.status()[0] == 0
