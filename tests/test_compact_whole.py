"""Pulling a pool together (GPU): what is violated is reported whether or not
pages move (counts by resize too), and the book stays whole if only the first of the call's kernels
runs."""
import ctypes
import glob

import numpy as np
import pytest
import torch

import speculative_decoding_drafter_k3_gb300 as k3da
from test_pages import Both, i32

pytestmark = pytest.mark.gpu
SIZES = [(4, 3, 30), (30, 100, 5000)]  # rows rewritten by the first kernel, and by a second one


def compact(x, limit=8):
    copies, num = torch.full((3, limit), 77, dtype=torch.int32, device="cuda"), i32([-1])
    k3da.k3da_pages_compact(*x.t, copies, num, workspace=k3da.alloc_compact_workspace(len(x.b.refs)), status=x.status)
    return int(num)


@pytest.mark.parametrize("R,S,P", SIZES)
@pytest.mark.parametrize("moves", [0, 1])
def test_lengths_are_looked_at(R, S, P, moves):
    x = Both(R, S, P)
    x.resize([64] * R)
    if moves:
        x.resize([0] + [-1] * (R - 1))
    for bad in (-1, S * 64 + 1):
        x.t[1][2] = bad
        compact(x)
        x.flags(k3da.STATUS_BAD_LENGTH)
        x.t[1][2] = 64
        compact(x)
        x.flags(0)


@pytest.mark.parametrize("R,S,P", SIZES + [(2, 3, 140001)])
def test_counts_below_zero_are_reported(R, S, P):
    for page in (0, 1, P // 2, P - 1):
        x = Both(R, S, P)
        x.t[2][page] = -1
        compact(x)
        x.flags(k3da.STATUS_BAD_COUNT)
        x = Both(R, S, P)
        x.t[2][page] = -2 ** 31
        k3da.k3da_pages_resize(*x.t, i32([64] + [0] * (R - 1)), x.copies, status=x.status)
        x.flags(k3da.STATUS_BAD_COUNT)
        assert int(x.t[2][page]) == -2 ** 31 and int(x.t[0][0, 0]) == (page == 0)


def test_a_page_that_is_written_next_but_not_counted_is_reported():
    x = Both(3, 4, 20)
    x.resize([130, 70, 20])
    x.t[2][int(x.t[0][1, 1])] = 0
    k3da.k3da_pages_resize(*x.t, i32([-1, 71, 21]), x.copies, status=x.status)
    x.flags(k3da.STATUS_BAD_COUNT)


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
