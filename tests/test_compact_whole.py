"""Pulling a pool together (GPU): the book stays whole if only the first of the
call's kernels runs."""
import ctypes
import glob

import numpy as np
import pytest
import torch

import speculative_decoding_drafter_k3_gb300 as k3da
from test_pages import Both, i32

pytestmark = pytest.mark.gpu


def test_without_its_second_kernel_the_book_is_as_it_was():
    """A call is two launches where the rows are long.  If the second is refused
    the call fails, and table, lengths and counts still belong together.  The
    call is captured, and its first kernel alone replayed."""
    rt = None
    for name in ["libcudart.so.13"] + glob.glob("/usr/local/cuda*/lib64/libcudart.so*"):
        try:
            rt = ctypes.CDLL(name)
            break
        except OSError:
            pass
    assert rt is not None

    def ok(rc):
        assert rc == 0, rc

    R, S, P = 40, 700, 60000
    x = Both(R, S, P)
    rng = np.random.default_rng(3)
    x.resize(rng.integers(1, S * 64, R))
    x.resize(np.where(rng.random(R) < 0.5, 0, -1))
    copies, num = torch.zeros(3, P, dtype=torch.int32, device="cuda"), i32([-1])
    ws = k3da.alloc_compact_workspace(P)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    handle = ctypes.c_void_p(stream.cuda_stream)
    graph, run = ctypes.c_void_p(), ctypes.c_void_p()
    ok(rt.cudaStreamBeginCapture(handle, 1))
    k3da.k3da_pages_compact(*x.t, copies, num, workspace=ws, status=x.status, stream=stream)
    ok(rt.cudaStreamEndCapture(handle, ctypes.byref(graph)))
    nodes, roots, n, first = (ctypes.c_void_p * 2)(), (ctypes.c_void_p * 1)(), ctypes.c_size_t(2), ctypes.c_size_t(1)
    ok(rt.cudaGraphGetNodes(graph, nodes, ctypes.byref(n)))
    ok(rt.cudaGraphGetRootNodes(graph, roots, ctypes.byref(first)))
    assert n.value == 2 and first.value == 1
    for node in nodes:
        if node != roots[0]:
            ok(rt.cudaGraphDestroyNode(ctypes.c_void_p(node)))
    ok(rt.cudaGraphInstantiate(ctypes.byref(run), graph, ctypes.c_ulonglong(0)))
    ok(rt.cudaGraphLaunch(run, handle))
    stream.synchronize()
    ok(rt.cudaGraphExecDestroy(run))
    ok(rt.cudaGraphDestroy(graph))
    x.same()
    x.flags(0)
    # And the whole call moves them.
    assert x.compact(P)
