"""The cache calls at the edges of what their documentation allows (GPU)."""
import os
import subprocess
import sys

import pytest
import torch

import speculative_decoding_drafter_k3_gb300 as k3da
from cache_cases import Batch, D
from test_chunk_attn import call, check, dev
from test_kv_cache import bits, expected_plain, heads

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def with_odd_bits(b):
    """NaN of both signs with payloads, infinities, zeros, subnormal numbers
    among the rows."""
    odd = [0x7F81, 0xFF81, 0x7FC0, 0xFFC0, 0x7FFF, 0xFFFF, 0x7FA5, 0x7F80, 0xFF80, 0x8000, 0x0001, 0x807F]
    raw = b.qkv.view(torch.int16)
    g = torch.Generator().manual_seed(5)
    for x in odd:
        at = torch.randint(0, raw.numel(), (200,), generator=g)
        raw.view(-1)[at] = x - 0x10000 if x >= 0x8000 else x
    return b


@pytest.mark.parametrize("hq,hkv", [(6, 1), (24, 4)])
def test_a_plain_append_copies_every_bit(hq, hkv):
    b = with_odd_bits(Batch([60, 3, 200], [5, 64, 1000], hq, hkv, "bf16", 1, seed=41))
    pool, _, qkv, table, lens, cu = dev(b)
    k3da.k3da_kv_append(pool, qkv, table, lens, cu, **heads(b))
    want, _ = expected_plain(b)
    assert torch.equal(bits(pool.cpu()), bits(want))
    k, v = (torch.zeros(b.T, hkv * D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k3da.k3da_kv_gather(k, v, pool, table, lens, cu, num_kv_heads=hkv)
    assert torch.equal(bits(k[:b.rows]), bits(qkv[:b.rows, hq * D:(hq + hkv) * D]))
    assert torch.equal(bits(v[:b.rows]), bits(qkv[:b.rows, (hq + hkv) * D:]))


@pytest.mark.parametrize("hq,hkv", [(6, 1), (24, 4)])
def test_append_qknorm_copies_every_bit_of_v(hq, hkv):
    """The norm+RoPE cell, then a plain append, with NaN in V."""
    b = with_odd_bits(Batch([60, 3], [5, 64], hq, hkv, "bf16", 1, seed=42))
    b.qkv[:, :(hq + hkv) * D] = 1.5
    pool, _, qkv, table, lens, cu = dev(b)
    two = pool.clone()
    args = b.positions.cuda(), b.q_w.cuda(), b.k_w.cuda()
    k3da.k3da_kv_append_qknorm(pool, qkv, table, lens, cu, *args, **heads(b))
    cell = k3da.k3da_qk_norm_rope(qkv.clone(), *args, **heads(b))
    k3da.k3da_kv_append(two, cell, table, lens, cu, **heads(b))
    assert torch.equal(bits(pool), bits(two))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_tokens_of_one_slot_leave_every_other_row_alone(cache):
    """A page in the tables of two requests, and twice in one: the rows that
    two tokens share are anything; the others are what they should be."""
    b = Batch([300, 300, 200], [0, 0, 0], 24, 4, cache, seed=43)
    b.table[1, 2] = b.table[0, 2]
    b.table[2, 3] = b.table[2, 1]
    pool, scales, qkv, table, lens, cu = dev(b)
    shared = [int(b.table[0, 2]), int(b.table[2, 1])]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want_pool, want_scales = expected_plain(b)
    for _ in range(5):
        k3da.k3da_kv_append(pool, qkv, table, lens, cu, kv_scales=scales, status=status, **heads(b))
    assert int(status) == 0
    fine = [p for p in range(b.pages) if p not in shared]
    got, want = (bits(t.cpu()).view(*t.shape[:-1], -1) for t in (pool, want_pool))
    assert torch.equal(got[fine], want[fine])
    # Request 2's second table entry of the page has tokens 192 to 199 only.
    rest = shared[1]
    assert torch.equal(got[rest, :, :, 8:], want[rest, :, :, 8:])
    if scales is not None:
        got, want = scales.view(torch.uint8).cpu(), want_scales.view(torch.uint8)
        assert torch.equal(got[fine], want[fine]) and torch.equal(got[rest, :, :, 8:], want[rest, :, :, 8:])


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_rows_behind_the_last_sequence_make_no_difference(cache):
    """They hold NaN and infinities, and positions from nowhere."""
    b = Batch([3, 70, 1], [500, 0, 63], 6, 1, cache, 30, seed=46, stride=1300)
    clean = dev(b)
    b.qkv[b.rows:] = torch.tensor([float("nan"), float("inf"), float("-inf"), 3e38]).repeat(128)[:b.qkv.shape[1]].to(torch.bfloat16)
    dirty = dev(b)
    pos = b.positions.to(torch.int64)
    far = pos.clone()
    far[b.rows:] = torch.tensor([-1, 2 ** 62, -2 ** 63]).repeat(10)
    results = []
    for d, where in ((clean, pos), (dirty, far)):
        pool, scales, qkv, table, lens, cu = d
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kw = dict(kv_scales=scales, status=status)
        q, out = (torch.full((b.T, 6 * D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        k, v = (torch.full((b.T, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        lse = torch.full((b.T, 6), 7.0, device="cuda")
        ws = k3da.alloc_chunk_workspace(b.T, b.R, 6, 1, b.stride)
        k3da.k3da_kv_append_qknorm(pool, qkv, table, lens, cu, where.cuda(), b.q_w.cuda(), b.k_w.cuda(), q_out=q, **heads(b), **kw)
        k3da.k3da_kv_append(pool, qkv, table, lens, cu, **heads(b), **kw)
        k3da.k3da_chunk_attn(out, qkv[:, :6 * D], pool, table, lens, cu, lse=lse, workspace=ws, **heads(b), **kw)
        k3da.k3da_kv_gather(k, v, pool, table, lens, cu, num_kv_heads=1, **kw)
        assert int(status) == 0
        for t in (q, out, k, v, lse):
            assert (t[b.rows:] == 7).all() and not (t[:b.rows] == 7).all()
        results.append([bits(t) for t in (pool, q, out, k, v, lse)])
    for x, y in zip(*results):
        assert torch.equal(x, y)


@pytest.mark.parametrize("new,ctx", [([1, 2], [100, 30]), ([1], [20000]), ([40], [100]), ([30], [9000])])
def test_scores_that_are_all_minus_infinity(new, ctx):
    """Such a row's weights are all zero: out 0 and lse -inf, as for a row
    that sees nothing."""
    b = Batch(new, ctx, 6, 1, "bf16", seed=44, stride=1300)
    b.pool[:, 0] = 0
    b.pool[:, 0, :, :, 0] = float("-inf")
    b.qkv[:, :6 * D] = 1.0
    out, lse = call(b)
    assert (out == 0).all() and (lse == float("-inf")).all()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_a_capture_that_forks_and_joins(cache):
    """Two requests' appends on two streams, joined before the attention over
    both, which a torch kernel on a third stream precedes too."""
    b = Batch([40, 130], [300, 70], 6, 1, cache, seed=45)
    pool, scales, qkv, table, lens, cu = dev(b)
    ws = k3da.alloc_chunk_workspace(b.T, b.R, 6, 1, b.stride)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(kv_scales=scales, status=status)
    halves = [(table[r:r + 1], lens[r:r + 1], torch.tensor([0, n], dtype=torch.int32, device="cuda"),
               qkv[b.cu[r]:b.cu[r + 1]].clone()) for r, n in enumerate(b.new)]
    staged = qkv.clone()

    def work(out, lse, source):
        main = torch.cuda.current_stream()
        sides = [torch.cuda.Stream() for _ in range(3)]
        for s in sides:
            s.wait_stream(main)
        for s, (t, l, c, rows) in zip(sides, halves):
            with torch.cuda.stream(s):
                k3da.k3da_kv_append(pool, rows, t, l, c, **heads(b), **kw)
        with torch.cuda.stream(sides[2]):
            staged.copy_(source)
            staged.mul_(1.0)
        for s in sides:
            main.wait_stream(s)
        k3da.k3da_chunk_attn(out, staged[:, :6 * D], pool, table, lens, cu, num_q_heads=6, num_kv_heads=1, lse=lse,
                             workspace=ws, **kw)

    want_pool, want_scales = expected_plain(b)
    out = torch.full((b.T, 6 * D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.T, 6), 7.0, device="cuda")
    work(out, lse, qkv)
    torch.cuda.synchronize()
    first = out.clone(), lse.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work(out, lse, qkv)
    start = b.pool.cuda()
    for _ in range(5):
        pool.view(torch.uint8).copy_(start.view(torch.uint8))
        staged.zero_()
        out.zero_()
        lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(out), bits(first[0])) and torch.equal(lse, first[1])
    assert int(status) == 0
    assert torch.equal(bits(pool.cpu()), bits(want_pool))
    b.pool, b.scales = want_pool, want_scales
    check(b, out, lse)


def child(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]


def test_a_refused_launch_leaves_no_error_behind():
    """The runtime refuses a launch on a stream whose capture has become
    invalid; the library's next call must not report that."""
    child("""
import sys; sys.path[:0] = ['.', 'tests']
import torch
import speculative_decoding_drafter_k3_gb300 as k3da
from cache_cases import Batch
from test_chunk_attn import call, check, dev
b = Batch([4], [100], 6, 1, "bf16", seed=1)
pool, scales, qkv, table, lens, cu = dev(b)
pos, qw, kw = b.positions.cuda(), b.q_w.cuda(), b.k_w.cuda()
heads = dict(num_q_heads=6, num_kv_heads=1)
k3da.k3da_qk_norm_rope(qkv.clone(), pos, qw, kw, **heads)
k3da.k3da_kv_append(pool, qkv, table, lens, cu, **heads)
spare = qkv.clone()
torch.cuda.synchronize()
side = torch.cuda.Stream()
graph = torch.cuda.CUDAGraph()
refused = False
with torch.cuda.stream(side):
    graph.capture_begin()
    try:
        side.synchronize()  # not allowed now: the capture ends here
    except Exception:
        pass
    try:
        k3da.k3da_kv_append(pool, qkv, table, lens, cu, **heads)
    except k3da.K3daError:
        refused = True
    try:
        graph.capture_end()
    except Exception:
        pass
assert refused
k3da.k3da_qk_norm_rope(spare, pos, qw, kw, **heads)
torch.cuda.synchronize()
""")


def test_the_calls_go_on_after_a_device_reset():
    """The device's context made anew (cudaDeviceReset, which ends this
    process's own context, with nothing in flight): kernels' attributes are
    set up again."""
    child("""
import ctypes, glob, os, sys
sys.path[:0] = ['.']
import torch
import speculative_decoding_drafter_k3_gb300 as k3da
names = ["libcudart.so.13"] + glob.glob("/usr/local/cuda*/lib64/libcudart.so*")
rt = None
for name in names:
    try:
        rt = ctypes.CDLL(name)
        break
    except OSError:
        pass
assert rt is not None
driver, lib = ctypes.CDLL("libcuda.so.1"), k3da.load_library()

def ok(rc):
    assert rc == 0, rc

def context():
    number = ctypes.c_ulonglong()
    ok(driver.cuCtxGetId(None, ctypes.byref(number)))
    return number.value

def run():
    ok(rt.cudaSetDevice(0))
    base = ctypes.c_void_p()
    ok(rt.cudaMalloc(ctypes.byref(base), ctypes.c_size_t(1 << 28)))
    ok(rt.cudaMemset(base, 0, ctypes.c_size_t(1 << 28)))
    at, mb = base.value, 1 << 20
    cu = (ctypes.c_int32 * 2)(0, 40)
    ok(rt.cudaMemcpy(ctypes.c_void_p(at), cu, ctypes.c_size_t(8), 1))
    pool, table, lens, q, out, ws = (at + k * mb for k in (1, 32, 33, 34, 40, 64))
    need = lib.k3da_chunk_workspace_bytes(40, 1, 6, 1, 2000)
    for tokens in (40, 1):  # both kernels
        rc = lib.k3da_chunk_attn(out, None, q, 384, tokens, pool, 0, None, 64, table, 2000, lens, at, 1, 6, 1, 64, 0, 0.125,
                                 ws, need, None, None)
        assert rc == 0, k3da.load_library().k3da_error_string(rc)
    ok(rt.cudaDeviceSynchronize())

run()
first = context()
ok(rt.cudaDeviceReset())
run()
assert context() != first  # it was another context
""")


def test_more_elements_than_32_bits_count():
    """1024 requests of 4200 tokens, 16 heads: rows of q, out, lse and qkv past
    2^32 elements.  The last request's against the definition, and against
    itself in a call of its own."""
    R, n, hq = 1024, 4200, 16
    T, stride = R * n, -(-n // 64)
    g = torch.Generator(device="cuda").manual_seed(47)
    qkv = torch.randn(T, (hq + 2) * D, generator=g, device="cuda", dtype=torch.bfloat16)
    pool, _ = k3da.alloc_cache(R * stride, 1)
    table = torch.arange(R * stride, dtype=torch.int32, device="cuda").view(R, stride)
    lens = torch.zeros(R, dtype=torch.int32, device="cuda")
    cu = torch.arange(0, T + 1, n, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(num_q_heads=hq, num_kv_heads=1, status=status)
    out, lse = torch.empty(T, hq * D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, hq, device="cuda")
    assert out.numel() > 1 << 32
    k3da.k3da_kv_append(pool, qkv, table, lens, cu, **kw)
    ws = k3da.alloc_chunk_workspace(T, R, hq, 1, stride)
    k3da.k3da_chunk_attn(out, qkv[:, :hq * D], pool, table, lens, cu, lse=lse, workspace=ws, **kw)
    k, v = (torch.empty(T, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k3da.k3da_kv_gather(k, v, pool, table, lens, cu, num_kv_heads=1, status=status)
    assert int(status) == 0
    assert torch.equal(k[-n:], qkv[-n:, hq * D:(hq + 1) * D]) and torch.equal(v[-n:], qkv[-n:, (hq + 1) * D:])
    alone, alse = torch.empty_like(out[:n]), torch.empty_like(lse[:n])
    k3da.k3da_chunk_attn(alone, qkv[-n:, :hq * D], pool, table[-1:].contiguous(), lens[:1], cu[:2], lse=alse, workspace=ws, **kw)
    kd, vd = k[-n:].double(), v[-n:].double()
    for i in (0, 1, 63, 2000, n - 1):
        q = qkv[T - n + i, :hq * D].double().view(hq, D)
        x = q @ kd[:i + 1].T * 0.125
        p = torch.softmax(x, -1)
        want, mag = p @ vd[:i + 1], p @ vd[:i + 1].abs()
        for got, l in ((out[T - n + i], lse[T - n + i]), (alone[i], alse[i])):
            err = (got.double().view(hq, D) - want).abs() - (2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -10) * mag)
            assert err.max() <= 1e-7
            # Scores: 64 terms of |q k| / 8 below 64; sums of 4200; ex2, log2.
            assert (l.double() - torch.logsumexp(x, -1)).abs().max() <= (64 * 64 + n) * 2.0 ** -24 + 2.0 ** -17
