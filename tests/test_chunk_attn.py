"""k3da_chunk_attn against its definition in fp64 (GPU).

Tolerance, from the arithmetic: every weight p is rounded to bf16 once before
P.V (half a step, 2^-8 of it), so the output is off by at most 2^-8 times the
weighted mean of |v|; the output is rounded to bf16 once, 2^-8 |o|; the fp32
rest (64-term scores of |q k| sums up to a few tens, ex2 within 2^-22, sums)
is below 2^-10 of the weighted mean.  lse, all in fp32: the score's error is
at most 64 * 2^-24 of its sum of |q k| scale, the sum's at most its length *
2^-24, and ex2 and log2 add 2^-21."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_drafter_k3_gb300 as k3da
from cache_cases import Batch, D, attend

pytestmark = pytest.mark.gpu
MASKS = ["causal", "full", "context"]
HEADS = [(6, 1), (24, 4), (8, 8), (16, 1), (5, 1)]
BATCHES = [  # (new tokens, cached tokens, rows of padding)
    ([1], [0], 0),
    ([1], [300], 0),
    ([8], [2041], 2),
    ([1, 1, 1, 1, 1, 1], [0, 1, 63, 64, 127, 128], 1),
    ([0, 3, 0, 22, 0], [64, 0, 7, 129, 0], 5),
    ([21, 22, 42, 43], [0, 107, 86, 1000], 0),
    ([150], [0], 0),
    ([97, 1, 260], [31, 515, 700], 40),
]


def dev(b):
    scales = None if b.scales is None else b.scales.view(torch.uint8).cuda().view(torch.float8_e8m0fnu)
    return b.pool.cuda(), scales, b.qkv.cuda(), b.table.cuda(), b.lens().cuda(), b.cu_t().cuda()


def call(b, mask="causal", d=None, out=None, lse=None, ws=None, status=None, stream=None, scale=0.125):
    pool, scales, qkv, table, lens, cu = d or dev(b)
    if out is None:
        out = torch.full((b.T, b.hq * D), 7.0, dtype=torch.bfloat16, device="cuda")
    if lse is None:
        lse = torch.full((b.T, b.hq), 7.0, device="cuda")
    if ws is None:
        ws = k3da.alloc_chunk_workspace(b.T, b.R, b.hq, b.hkv, b.stride)
        ws.fill_(0xFF)
    k3da.k3da_chunk_attn(out, qkv[:, :b.hq * D], pool, table, lens, cu, num_q_heads=b.hq, num_kv_heads=b.hkv,
                         softmax_scale=scale, mask=mask, kv_scales=scales, lse=lse, workspace=ws, status=status,
                         stream=stream)
    return out, lse


def check(b, out, lse, mask="causal", scale=0.125):
    want, wlse, mag, grain = attend(b, mask, scale)
    got, glse = out.cpu().double().view(b.T, b.hq, D), lse.cpu().double()
    n = b.rows
    assert (got[n:] == 7).all() and (glse[n:] == 7).all(), "rows behind the last sequence changed"
    got, glse, want, wlse, mag = got[:n], glse[:n], want[:n], wlse[:n], mag[:n]
    assert torch.equal(got.isnan(), want.isnan()), "NaN in other places"
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine].nan_to_num(), want[~fine].nan_to_num())
    err = (got - want).abs() - (2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -10) * mag)
    assert err[fine].numel() == 0 or err[fine].max() <= 1e-7, f"out off by {err[fine].max():.3e} over its bound"
    empty = wlse == -math.inf
    assert torch.equal(glse == -math.inf, empty) and (got[empty] == 0).all()
    ok = torch.isfinite(wlse)
    longest = max(c + m for c, m in zip(b.ctx, b.new))
    tol = (64 * grain + longest) * 2.0 ** -24 + 2.0 ** -21 * (1 + wlse[ok].abs())
    assert ((glse - wlse)[ok].abs() <= tol).all()


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("new,ctx,pad", BATCHES)
def test_matches_the_definition(new, ctx, pad, hq, hkv, cache, mask):
    b = Batch(new, ctx, hq, hkv, cache, pad, seed=sum(new) + hq)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = call(b, mask, status=status)
    assert int(status) == 0
    check(b, out, lse, mask)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("scale", [1.0, 0.01])
def test_sharp_and_flat_softmax(cache, scale):
    """Scores of several hundred (the running maximum is passed again and
    again) and of nearly nothing."""
    b = Batch([60, 3], [700, 1500], 6, 1, cache, seed=3, scale=4.0 if scale == 1.0 else 1.0)
    out, lse = call(b, scale=scale)
    check(b, out, lse, scale=scale)


@pytest.mark.parametrize("new", [1, 30, 100])
def test_rising_scores(new):
    """Every key beats the last: the running maximum moves at every tile."""
    b = Batch([new], [1400], 6, 1, "bf16", seed=4)
    u = torch.randn(D, generator=torch.Generator().manual_seed(1))
    u /= u.norm()
    b.qkv[:, :6 * D] = (u * 8).repeat(6).to(torch.bfloat16)
    for c in range(1400 + new):
        b.pool[int(b.table[0, c // 64]), 0, 0, c % 64] = (u * (c * 0.1 - 70)).to(torch.bfloat16)
    out, lse = call(b)
    check(b, out, lse)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,ctx", [([1], [20000]), ([5, 1], [9000, 33]), ([700], [2500]), ([64] * 20, [100] * 20),
                                     ([1] * 300, [130] * 300), ([2000, 3], [0, 5000])])
def test_longer_batches(new, ctx, cache):
    b = Batch(new, ctx, 6, 1, cache, seed=5)
    if len(new) == 300:
        b = Batch(new, list(range(300)), 8, 8, cache, seed=6)
    out, lse = call(b)
    check(b, out, lse)


def test_a_thousand_requests():
    g = np.random.default_rng(5)
    b = Batch(g.integers(0, 4, 1024).tolist(), g.integers(0, 200, 1024).tolist(), 6, 1, "bf16", 2, seed=9)
    out, lse = call(b)
    check(b, out, lse)


def test_pages_far_into_a_large_pool():
    """Byte offsets past 2^32, page ids past 2^16."""
    b = Batch([5, 40], [200, 77], 24, 4, "bf16", seed=10)
    pool, scales, qkv, table, lens, cu = dev(b)
    pages = 90000  # 5.9 GB
    big = torch.zeros(pages, 2, 4, 64, D, dtype=torch.bfloat16, device="cuda")
    shift = pages - b.pages
    big[shift:] = pool
    moved = torch.where((table >= 0) & (table < b.pages), table + shift, table)
    out, lse = call(b, d=(big, scales, qkv, moved, lens, cu))
    check(b, out, lse)
    del big
    torch.cuda.empty_cache()


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_stale_slots_do_not_leak(cache, mask):
    """Slots past a request's last token hold NaN and infinities."""
    b = Batch([3, 30, 1], [61, 100, 128], 6, 1, cache, seed=11)
    want_pool = b.pool.clone()
    seen = torch.zeros(b.pages, 64, dtype=torch.bool)
    for r, n in enumerate(b.new):
        for c in range(b.ctx[r] + (0 if mask == "context" else n)):
            seen[int(b.table[r, c // 64]), c % 64] = True
    for p in range(b.pages):
        stale = ~seen[p]
        if cache == "bf16":
            b.pool[p, :, :, stale] = torch.tensor([float("nan"), float("inf"), float("-inf")]).repeat(22)[:D].to(torch.bfloat16)
        else:
            b.pool.view(torch.uint8)[p, :, :, stale] = 0x7F
            b.scales.view(torch.uint8)[p, :, :, stale] = 255
    assert not torch.equal(b.pool.view(torch.uint8), want_pool.view(torch.uint8))
    out, lse = call(b, mask)
    assert torch.isfinite(out[:b.rows].float()).all()
    check(b, out, lse, mask)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("new,ctx", [([50], [100]), ([7], [125]), ([300], [0])])
def test_a_nan_reaches_only_rows_that_see_it(new, ctx, what, cache):
    b = Batch(new, ctx, 6, 1, cache, seed=12)
    at = ctx[0] + new[0] // 2
    page, slot = int(b.table[0, at // 64]), at % 64
    kv = "kv".index(what)
    if cache == "bf16":
        b.pool[page, kv, 0, slot, 5] = float("nan")
        b.pool[page, kv, 0, slot, 9] = float("nan")
    else:
        b.scales.view(torch.uint8)[page, kv, 0, slot] = 255
    out, lse = call(b)
    check(b, out, lse)
    assert torch.isfinite(out[:new[0] // 2].float()).all()


@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
def test_an_infinite_value_reaches_only_rows_that_see_it(value):
    b = Batch([50], [100], 6, 1, "bf16", seed=13)
    at = 120
    b.pool[int(b.table[0, at // 64]), 1, 0, at % 64, 3] = value
    out, lse = call(b)
    got = out.cpu().double().view(50, 6, D)
    assert torch.isfinite(got[:20]).all() and (got[20:, :, 3] == value).all()
    others = [d for d in range(D) if d != 3]
    assert torch.isfinite(got[:, :, others]).all()


def test_bad_pages_and_lengths_are_flagged():
    b = Batch([4, 4], [100, 62], 6, 1, "bf16", seed=14)
    d = list(dev(b))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d[3] = d[3].clone()
    d[3][0, 0] = -3
    out, lse = call(b, d=d, status=status)
    assert int(status) == k3da.STATUS_BAD_PAGE
    zeros = Batch([4, 4], [100, 62], 6, 1, "bf16", seed=14)
    zeros.pool[int(zeros.table[0, 0])] = 0   # served as zeros
    check(zeros, out, lse)
    status.zero_()
    d = list(dev(b))
    d[4] = torch.tensor([b.stride * 64 - 1, -5], dtype=torch.int32, device="cuda")
    out, lse = call(b, "full", d=d, status=status)
    assert int(status) & k3da.STATUS_BAD_LENGTH
    assert torch.isfinite(out.float()).all()
    status.zero_()
    d = list(dev(b))
    d[5] = torch.tensor([0, 100, 5], dtype=torch.int32, device="cuda")  # past the rows, then falling
    out, lse = call(b, d=d, status=status)
    assert int(status) & k3da.STATUS_BAD_LENGTH
    assert torch.isfinite(out.float()).all()


def test_no_tokens():
    b = Batch([0, 0], [5, 70], 6, 1, "bf16", seed=1)
    call(b)
    b = Batch([0, 0], [5, 70], 6, 1, "bf16", pad=9, seed=1)
    out, lse = call(b)
    assert (out == 7).all() and (lse == 7).all()


@pytest.mark.parametrize("new,ctx", [([1], [3000]), ([200, 7], [1000, 4000])])
def test_reruns_bitwise_with_any_workspace_and_stream(new, ctx):
    b = Batch(new, ctx, 24, 4, "bf16", seed=15)
    d = dev(b)
    first, flse = call(b, d=d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.zeros_like(k3da.alloc_chunk_workspace(b.T, b.R, 24, 4, b.stride))
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again, alse = call(b, d=d, ws=ws)
    third, tlse = call(b, d=d, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.int16), again.view(torch.int16)) and torch.equal(flse, alse)
    assert torch.equal(first.view(torch.int16), third.view(torch.int16)) and torch.equal(flse, tlse)
    q = d[2][:, :24 * D].contiguous()
    out = torch.empty_like(first)
    k3da.k3da_chunk_attn(out, q, d[0], *d[3:], num_q_heads=24, num_kv_heads=4, workspace=ws)  # other strides, no lse
    assert torch.equal(first.view(torch.int16), out.view(torch.int16))


def test_a_captured_call_follows_rewritten_inputs():
    b = Batch([3, 60], [10, 2000], 6, 1, "bf16", seed=16)
    d = dev(b)
    ws = k3da.alloc_chunk_workspace(b.T, b.R, 6, 1, b.stride)
    out, lse = call(b, d=d, ws=ws)
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call(b, d=d, out=out, lse=lse, ws=ws, stream=s)
    b2 = Batch([50, 13], [1500, 40], 6, 1, "bf16", seed=17, stride=b.stride)
    assert b2.pages <= b.pages and b2.T == b.T
    d[0][:b2.pages].copy_(b2.pool)
    for dst, src in zip(d[2:], (b2.qkv, b2.table, b2.lens(), b2.cu_t())):
        dst.copy_(src)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    check(b2, out, lse)


def test_calls_on_two_streams_at_once():
    bs = [Batch([100], [3000], 24, 4, "bf16", seed=18), Batch([1, 2, 3], [500, 9000, 40], 6, 1, "e4m3", seed=19)]
    ds = [dev(b) for b in bs]
    alone = [call(b, d=d) for b, d in zip(bs, ds)]
    wss = [k3da.alloc_chunk_workspace(b.T, b.R, b.hq, b.hkv, b.stride) for b in bs]
    outs = [(torch.empty_like(o), torch.empty_like(l)) for o, l in alone]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(20):
        for b, d, (o, l), ws, s in zip(bs, ds, outs, wss, streams):
            call(b, d=d, out=o, lse=l, ws=ws, stream=s)
    torch.cuda.synchronize()
    for (o, l), (x, y) in zip(outs, alone):
        assert torch.equal(o.view(torch.int16), x.view(torch.int16)) and torch.equal(l, y)


@pytest.mark.parametrize("config", ["mixed_8x8", "heads_24_4", "w6_8x6"])
def test_a_block_that_joins_the_cache_attends_as_the_drafters_block(config):
    """norm, RoPE and append of the draft block, then attention with the full
    mask: the drafter's block attention, whose block never enters the pool.
    And over the contexts alone, merged with the block's own part by lse.
    Both outputs are within their own bounds of the definition; the workloads'
    tolerance (2e-2 + 2e-2 |o|) covers the sum."""
    from speculative_decoding_drafter_k3_gb300 import workloads
    from common import assert_close, oracle_for
    case = getattr(workloads, config)(device="cuda")
    want = oracle_for(case)
    R, B, Hq, Hkv = case.R, case.B, case.Hq, case.Hkv
    # Room for the block: a table one page wider than the context needs.
    table = torch.cat([case.page_table, torch.full((R, 1), -1, dtype=torch.int32, device="cuda")], 1)
    used = set(case.page_table.cpu().flatten().tolist())
    spare = iter(p for p in range(case.num_pages) if p not in used)
    for r, L in enumerate(case.lens_list()):
        for page in range(-(-L // 64), -(-(L + B) // 64)):
            table[r, page] = next(spare)
    cu = torch.arange(0, R * B + 1, B, dtype=torch.int32, device="cuda")
    pool = case.pool.clone()
    q = torch.empty(R * B, Hq * D, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(num_q_heads=Hq, num_kv_heads=Hkv, status=status)
    ws = k3da.alloc_chunk_workspace(R * B, R, Hq, Hkv, table.shape[1])
    ctx_out, ctx_lse = torch.empty_like(q), torch.empty(R * B, Hq, device="cuda")
    k3da.k3da_kv_append_qknorm(pool, case.qkv, table, case.ctx_lens, cu, case.positions, case.q_norm_w, case.k_norm_w,
                               q_out=q, eps=case.eps, rope_base=case.rope_base, **kw)
    out = torch.empty_like(q)
    k3da.k3da_chunk_attn(out, q, pool, table, case.ctx_lens, cu, mask="full", workspace=ws, **kw)
    k3da.k3da_chunk_attn(ctx_out, q, pool, table, case.ctx_lens, cu, mask="context", lse=ctx_lse, workspace=ws, **kw)
    assert int(status) == 0
    assert_close(out, want, f"{config}: append, then full mask")
    k, v = (torch.empty(R * B, Hkv * D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k3da.k3da_kv_gather(k, v, pool, table, case.ctx_lens, cu, num_kv_heads=Hkv)
    g = Hq // Hkv
    qb = q.double().view(R, B, Hkv, g, D)
    x = torch.einsum("rihgd,rjhd->rihgj", qb, k.double().view(R, B, Hkv, D)) * case.scale
    own_lse = torch.logsumexp(x, -1).view(R * B, Hq, 1)
    own = torch.einsum("rihgj,rjhd->rihgd", torch.softmax(x, -1), v.double().view(R, B, Hkv, D)).reshape(R * B, Hq, D)
    total = torch.logaddexp(own_lse, ctx_lse.double()[..., None])
    merged = own * (own_lse - total).exp() + ctx_out.double().view(R * B, Hq, D) * (ctx_lse.double()[..., None] - total).exp()
    assert_close(merged.reshape(R * B, Hq * D).float(), want, f"{config}: context and block merged")
