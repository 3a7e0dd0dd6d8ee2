"""k3da_kv_append, k3da_kv_append_qknorm and k3da_kv_gather against their
definitions in fp64 (GPU).

Tolerances, from the arithmetic.  A plain append copies bits or rounds a bf16
times a power of two (exact) to e4m3 once: compared bit for bit.  The fused
form's fp32 norm and rotation are within 2^-20 of the value and of the pair's
magnitude (64-term sums, a few roundings of 2^-24, rsqrt within 2^-22, angles
within 1e-7): bf16 adds half a step, 2^-8 |y|; a code adds half a step, 2^-4
|y|, or half the smallest code, 2^-10, times the row's scale."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_drafter_k3_gb300 as k3da
from cache_cases import Batch, D, dequantise, quantise

pytestmark = pytest.mark.gpu
HEADS = [(6, 1), (24, 4), (8, 8), (5, 1), (32, 2)]
BATCHES = [  # (new tokens, cached tokens, rows of padding)
    ([1], [0], 0),
    ([8], [300], 3),
    ([1, 1, 1, 1, 1], [63, 64, 65, 127, 1000], 1),
    ([0, 70, 0, 0, 5, 129, 0], [5, 60, 0, 640, 63, 1, 12], 40),
    ([333], [0], 0),
]


def bits(t):
    return t.contiguous().view(torch.uint8)


def dev(b):
    pool, scales = b.pool.cuda(), None if b.scales is None else b.scales.view(torch.uint8).cuda().view(torch.float8_e8m0fnu)
    return pool, scales, b.qkv.cuda(), b.table.cuda(), b.lens().cuda(), b.cu_t().cuda()


def heads(b):
    return dict(num_q_heads=b.hq, num_kv_heads=b.hkv)


def expected_plain(b):
    """(pool, scales) after a plain append, by the definition."""
    pool, scales = b.pool.clone(), None if b.scales is None else b.scales.clone()
    x = b.qkv.view(b.T, -1, D)[:, b.hq:].reshape(b.T, 2, b.hkv, D)
    if b.cache == "e4m3":
        code, byte = quantise(x.double())
    for t, page, slot in b.where():
        if b.cache == "bf16":
            pool[page, :, :, slot] = x[t]
        else:
            bits(pool).view(pool.shape)[page, :, :, slot] = code[t].view(torch.uint8)
            scales.view(torch.uint8)[page, :, :, slot] = byte[t]
    return pool, scales


def assert_cache(b, pool, scales, want_pool, want_scales):
    if b.cache == "bf16":
        assert torch.equal(bits(pool.cpu()), bits(want_pool))
        return
    byte, want = scales.view(torch.uint8).cpu(), want_scales.view(torch.uint8)
    assert torch.equal(byte, want)
    fine = want != 255  # codes of a NaN row say nothing
    assert torch.equal(bits(pool.cpu()).view(pool.shape)[fine], bits(want_pool).view(pool.shape)[fine])


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("new,ctx,pad", BATCHES)
def test_append_writes_the_chunk_and_nothing_else(new, ctx, pad, hq, hkv, cache):
    b = Batch(new, ctx, hq, hkv, cache, pad, seed=len(new) + hq, scale=3.0)
    pool, scales, qkv, table, lens, cu = dev(b)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k3da.k3da_kv_append(pool, qkv, table, lens, cu, kv_scales=scales, status=status, **heads(b))
    torch.cuda.synchronize()
    assert int(status) == 0
    assert_cache(b, pool, scales, *expected_plain(b))
    assert torch.equal(bits(qkv.cpu()), bits(b.qkv))


def test_append_many_requests():
    g = np.random.default_rng(5)
    new, ctx = g.integers(0, 4, 1024).tolist(), g.integers(0, 200, 1024).tolist()
    b = Batch(new, ctx, 6, 1, "e4m3", 2, seed=9)
    pool, scales, qkv, table, lens, cu = dev(b)
    k3da.k3da_kv_append(pool, qkv, table, lens, cu, kv_scales=scales, **heads(b))
    assert_cache(b, pool, scales, *expected_plain(b))


@pytest.mark.parametrize("hq,hkv", [(6, 1), (24, 4)])
def test_quantised_rows_at_the_borders(hq, hkv):
    """Largest magnitudes at and next to 448 * 2^k, ties of codes, zero rows,
    the type's largest and smallest values, infinities and NaN."""
    b = Batch([40], [50], hq, hkv, "e4m3", seed=2)
    x = b.qkv.view(40, -1, D)
    special = [448.0, 450.0, 446.0, 7.0, 7.03125, 6.96875, 3.38e38, 1e-38, 9.2e-41, 0.0, float("inf"), float("-inf"),
               float("nan"), -448.0, 2.0 ** -120]
    for t, v in enumerate(special):
        x[t, hq:] = 0
        x[t, hq:, t] = v
        if v == v and abs(v) < 3e38:
            x[t, hq:, 40:] = torch.linspace(-1, 1, 24).to(torch.bfloat16) * v
    x[20, hq:] = torch.tensor([256.0] + [16.0 + i * 0.5 for i in range(63)]).to(torch.bfloat16)  # ties
    x[21, hq:] = torch.tensor([256.0] + [i * 2.0 ** -11 for i in range(63)]).to(torch.bfloat16)   # below the smallest
    pool, scales, qkv, table, lens, cu = dev(b)
    k3da.k3da_kv_append(pool, qkv, table, lens, cu, kv_scales=scales, **heads(b))
    want_pool, want_scales = expected_plain(b)
    assert_cache(b, pool, scales, want_pool, want_scales)
    k, v = torch.zeros(40, hkv * D, dtype=torch.bfloat16, device="cuda"), torch.zeros(40, hkv * D, dtype=torch.bfloat16, device="cuda")
    k3da.k3da_kv_gather(k, v, pool, table, lens, cu, num_kv_heads=hkv, kv_scales=scales)
    code, byte = quantise(x[:, hq:].double())
    want = dequantise(code, byte).to(torch.bfloat16)
    got = torch.stack([k.cpu(), v.cpu()], 1).view(40, 2 * hkv, D)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(), want.nan_to_num())
    assert got[10:13].isnan().all() and not got[13:].isnan().any()


def norm_rope_oracle(b, yarn):
    kw = dict(num_q_heads=b.hq, num_kv_heads=b.hkv)
    if yarn is not None:
        kw["yarn"] = yarn.as_dict()
    return oracle.qk_norm_rope(b.qkv, b.positions, b.q_w, b.k_w, **kw)


def rope_fp64(b):
    """Normalised and roped q and k head rows in fp64 [T, Hq + Hkv, 64]."""
    x = b.qkv.view(b.T, -1, D)[:, :b.hq + b.hkv].double()
    w = torch.cat([b.q_w.double().expand(b.hq, D), b.k_w.double().expand(b.hkv, D)])
    y = x / (x.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w
    a = b.positions.double()[:, None] * 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
    c, s = a.cos()[:, None], a.sin()[:, None]
    lo, hi = y[..., :32], y[..., 32:]
    return torch.cat([lo * c - hi * s, hi * c + lo * s], -1)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("new,ctx,pad", BATCHES)
def test_append_qknorm_against_the_definition(new, ctx, pad, hq, hkv, cache):
    b = Batch(new, ctx, hq, hkv, cache, pad, seed=3 * len(new) + hq)
    pool, scales, qkv, table, lens, cu = dev(b)
    q = torch.full((b.T, hq * D), 7.0, dtype=torch.bfloat16, device="cuda")
    k3da.k3da_kv_append_qknorm(pool, qkv, table, lens, cu, b.positions.cuda(), b.q_w.cuda(), b.k_w.cuda(), q_out=q,
                               kv_scales=scales, **heads(b))
    torch.cuda.synchronize()
    y = rope_fp64(b)
    pair = (y[..., :32].square() + y[..., 32:].square()).sqrt().repeat(1, 1, 2)
    fp32 = 2.0 ** -20 * pair + 1e-30
    got_q = q.cpu().double().view(b.T, hq, D)
    assert (got_q[:b.rows] - y[:b.rows, :hq]).abs().sub(2.0 ** -8 * y[:b.rows, :hq].abs() + fp32[:b.rows, :hq]).max() <= 0
    assert (got_q[b.rows:] == 7.0).all()
    want_pool, want_scales = expected_plain(b)   # right for v and for every slot that is not the chunk's
    k_of = {t: (page, slot) for t, page, slot in b.where()}
    got, byte = pool.cpu(), None if scales is None else scales.view(torch.uint8).cpu()
    for t, (page, slot) in k_of.items():
        k, tol = y[t, hq:], fp32[t, hq:]
        if cache == "bf16":
            assert ((got[page, 0, :, slot].double() - k).abs() <= 2.0 ** -8 * k.abs() + tol).all()
            got[page, 0, :, slot] = want_pool[page, 0, :, slot]
        else:
            s = torch.exp2(byte[page, 0, :, slot].double() - 127)[:, None]
            top = k.abs().amax(-1)
            assert (top <= 448 * (1 + 2.0 ** -19) * s[:, 0]).all() and (top > 224 * (1 - 2.0 ** -19) * s[:, 0]).all()
            val = dequantise(got[page, 0, :, slot], byte[page, 0, :, slot])
            assert ((val - k).abs() <= torch.maximum(2.0 ** -4 * k.abs(), 2.0 ** -10 * s) + tol).all()
            bits(got).view(got.shape)[page, 0, :, slot] = bits(want_pool).view(got.shape)[page, 0, :, slot]
            byte[page, 0, :, slot] = want_scales.view(torch.uint8)[page, 0, :, slot]
    assert_cache(b, got, None if byte is None else byte.view(torch.float8_e8m0fnu), want_pool, want_scales)


@pytest.mark.parametrize("hq,hkv", [(6, 1), (24, 4)])
@pytest.mark.parametrize("pos", [torch.int32, torch.int64])
@pytest.mark.parametrize("yarn", [False, True])
def test_append_qknorm_gives_the_cells_bits(hq, hkv, pos, yarn):
    """norm+RoPE cell, then a plain append: the same bits in q and cache."""
    b = Batch([5, 64, 1], [1000, 0, 63], hq, hkv, "bf16", 2, seed=6)
    y = k3da.Yarn.of(4.0, 4096.0) if yarn else None
    pool, _, qkv, table, lens, cu = dev(b)
    two = pool.clone()
    q = torch.zeros(b.T, hq * D, dtype=torch.bfloat16, device="cuda")
    args = (b.positions.to(pos).cuda(), b.q_w.cuda(), b.k_w.cuda())
    k3da.k3da_kv_append_qknorm(pool, qkv, table, lens, cu, *args, q_out=q, yarn=y, **heads(b))
    cell = k3da.k3da_qk_norm_rope(qkv.clone(), *args, yarn=y, **heads(b))
    k3da.k3da_kv_append(two, cell, table, lens, cu, **heads(b))
    assert torch.equal(bits(pool), bits(two))
    assert torch.equal(bits(q[:b.rows]), bits(cell[:b.rows, :hq * D]))
    alone = b.pool.cuda()
    k3da.k3da_kv_append_qknorm(alone, qkv, table, lens, cu, *args, yarn=y, **heads(b))  # no q wanted
    assert torch.equal(bits(alone), bits(two)) and torch.equal(bits(qkv.cpu()), bits(b.qkv))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("hkv", [1, 4, 8, 64])
@pytest.mark.parametrize("new,ctx,pad", BATCHES)
def test_gather_reads_back_what_the_cache_holds(new, ctx, pad, hkv, cache):
    b = Batch(new, ctx, hkv, hkv, cache, pad, seed=hkv)
    pool, scales, _, table, lens, cu = dev(b)
    k = torch.full((b.T, hkv * D), 7.0, dtype=torch.bfloat16, device="cuda")
    v = torch.full((b.T, hkv * D), 9.0, dtype=torch.bfloat16, device="cuda")
    k3da.k3da_kv_gather(k, v, pool, table, lens, cu, num_kv_heads=hkv, kv_scales=scales)
    torch.cuda.synchronize()
    for r, n in enumerate(new):
        wk, wv = b.cached(r, ctx[r] + n)
        rows = slice(b.cu[r], b.cu[r] + n)
        assert torch.equal(k[rows].cpu().double().view(n, hkv, D), wk[ctx[r]:])
        assert torch.equal(v[rows].cpu().double().view(n, hkv, D), wv[ctx[r]:])
    assert (k[b.rows:] == 7).all() and (v[b.rows:] == 9).all()


def test_long_gather_of_a_quantised_cache():
    b = Batch([20001, 7, 13003], [5, 0, 100], 4, 4, "e4m3", 3, seed=8)
    pool, scales, _, table, lens, cu = dev(b)
    k, v = (torch.zeros(b.T, 4 * D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k3da.k3da_kv_gather(k, v, pool, table, lens, cu, num_kv_heads=4, kv_scales=scales)
    for r, n in enumerate(b.new):
        wk, wv = b.cached(r, b.ctx[r] + n)
        rows = slice(b.cu[r], b.cu[r] + n)
        assert torch.equal(k[rows].cpu().double().view(n, 4, D), wk[b.ctx[r]:])
        assert torch.equal(v[rows].cpu().double().view(n, 4, D), wv[b.ctx[r]:])


def test_bad_pages_and_lengths_are_flagged_and_skipped():
    b = Batch([4, 4, 4], [100, 62, 3], 6, 1, "bf16", seed=4)
    want, _ = expected_plain(b)
    pool, _, qkv, table, lens, cu = dev(b)
    table[1, 1] = b.pages  # request 1: tokens 64, 65
    lens[2] = b.stride * 64 - 2  # request 2: its last two tokens have no slot
    table[2, :] = table[0, :]    # ... and its first two would be request 0's rows past its own
    for t, page, slot in b.where():
        if t in (6, 7) or t >= 8:
            want[page, :, :, slot] = b.pool[page, :, :, slot]
    at = b.stride * 64 - 2
    page = int(table[0, at // 64])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if 0 <= page < b.pages:
        x = b.qkv.view(b.T, -1, D)[:, 6:].reshape(b.T, 2, 1, D)
        want[page, :, :, at % 64], want[page, :, :, at % 64 + 1] = x[8], x[9]
    k3da.k3da_kv_append(pool, qkv, table, lens, cu, status=status, **heads(b))
    assert int(status) == k3da.STATUS_BAD_PAGE | k3da.STATUS_BAD_LENGTH
    assert torch.equal(bits(pool.cpu()), bits(want))
    k, v = (torch.full((b.T, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    status.zero_()
    k3da.k3da_kv_gather(k, v, pool, table, lens, cu, num_kv_heads=1, status=status)
    assert int(status) == k3da.STATUS_BAD_PAGE | k3da.STATUS_BAD_LENGTH
    assert (k[6:8] == 0).all() and (v[6:8] == 0).all() and (k[10:] == 0).all()
    assert torch.equal(bits(k[:6]), bits(qkv[:6, 6 * D:7 * D]))
    lens[0] = -50
    status.zero_()
    k3da.k3da_kv_append(pool.clone(), qkv, table, lens, cu, status=status, **heads(b))
    assert int(status) & k3da.STATUS_BAD_LENGTH


def test_no_tokens_is_a_call_that_does_nothing():
    b = Batch([0, 0], [5, 70], 6, 1, "bf16", seed=1)
    pool, _, qkv, table, lens, cu = dev(b)
    k3da.k3da_kv_append(pool, qkv, table, lens, cu, **heads(b))
    k3da.k3da_kv_append_qknorm(pool, qkv, table, lens, cu, torch.zeros(0, dtype=torch.int64, device="cuda"), b.q_w.cuda(),
                               b.k_w.cuda(), q_out=torch.zeros(0, 6 * D, dtype=torch.bfloat16, device="cuda"), **heads(b))
    e = torch.zeros(0, D, dtype=torch.bfloat16, device="cuda")
    k3da.k3da_kv_gather(e, e.clone(), pool, table, lens, cu, num_kv_heads=1)
    torch.cuda.synchronize()
    assert torch.equal(bits(pool.cpu()), bits(b.pool))


def test_a_captured_append_and_gather_follow_rewritten_lengths():
    b = Batch([3, 6], [10, 200], 24, 4, "e4m3", seed=12)
    pool, scales, qkv, table, lens, cu = dev(b)
    k, v = (torch.zeros(b.T, 4 * D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s = torch.cuda.Stream()

    def both():
        k3da.k3da_kv_append(pool, qkv, table, lens, cu, kv_scales=scales, stream=s, **heads(b))
        k3da.k3da_kv_gather(k, v, pool, table, lens, cu, num_kv_heads=4, kv_scales=scales, stream=s)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        both()
    b2 = Batch([7, 2], [60, 150], 24, 4, "e4m3", seed=13, stride=b.stride)
    assert b2.pages <= b.pages
    n = b2.pages
    pool[:n].copy_(b2.pool.cuda())
    scales.view(torch.uint8)[:n].copy_(b2.scales.view(torch.uint8).cuda())
    for dst, src in ((qkv, b2.qkv), (table, b2.table), (lens, b2.lens()), (cu, b2.cu_t())):
        dst.copy_(src.cuda())
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    want_pool, want_scales = expected_plain(b2)
    assert_cache(b2, pool[:n], scales[:n], want_pool, want_scales)
    code, byte = quantise(b2.qkv.view(9, -1, D)[:, 24:].double())
    want = dequantise(code, byte).reshape(9, 2, 4 * D)
    assert torch.equal(k.cpu().double(), want[:, 0]) and torch.equal(v.cpu().double(), want[:, 1])


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,new", [(24, 4, [2000, 0, 3000, 1001]), (6, 1, [20011, 3]), (64, 64, [300, 157]), (64, 4, [900])])
def test_a_long_append_is_its_pieces(hq, hkv, new, cache, norm):
    """Many tokens a CTA against few: one call against calls of 200 tokens,
    bit for bit, and what a gather reads back against what was written."""
    ctx = [37, 5, 0, 640][:len(new)]
    b = Batch(new, ctx, hq, hkv, cache, pad=2, seed=hq)
    pool, scales, qkv, table, lens, cu = dev(b)
    w = b.q_w.cuda(), b.k_w.cuda()
    pos = b.positions.cuda()

    def append(pool, scales, rows, table, lens, cu, pos, q):
        if norm:
            k3da.k3da_kv_append_qknorm(pool, rows, table, lens, cu, pos, *w, q_out=q, kv_scales=scales, **heads(b))
        else:
            k3da.k3da_kv_append(pool, rows, table, lens, cu, kv_scales=scales, **heads(b))

    whole = pool.clone(), None if scales is None else scales.view(torch.uint8).clone().view(torch.float8_e8m0fnu)
    qs = [torch.full((b.T, hq * D), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    append(*whole, qkv, table, lens, cu, pos, qs[0])
    for r, n in enumerate(new):
        for i in range(0, n, 200):
            m, at = min(200, n - i), b.cu[r] + i
            append(pool, scales, qkv[at:at + m], table[r:r + 1], torch.tensor([ctx[r] + i], dtype=torch.int32, device="cuda"),
                   torch.tensor([0, m], dtype=torch.int32, device="cuda"), pos[at:at + m], qs[1][at:at + m])
    assert torch.equal(bits(whole[0]), bits(pool)) and torch.equal(bits(qs[0]), bits(qs[1]))
    assert scales is None or torch.equal(bits(whole[1]), bits(scales))
    k, v = (torch.full((b.T, hkv * D), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k3da.k3da_kv_gather(k, v, pool, table, lens, cu, num_kv_heads=hkv, kv_scales=scales)
    # Values as the cache's definition has them; V is raw in either form.
    t, page, slot = (torch.tensor(x, device="cuda") for x in zip(*b.where()))
    if cache == "bf16":
        want = pool[page, :, :, slot]
        assert torch.equal(want[:, 1].reshape(-1, hkv * D), qkv[:b.rows, (hq + hkv) * D:])
    else:
        code, byte = bits(pool).view(pool.shape)[page, :, :, slot], scales.view(torch.uint8)[page, :, :, slot]
        want = (code.cpu().view(torch.float8_e4m3fn).double() * torch.exp2(byte.cpu().double() - 127.0)[..., None]).to(torch.bfloat16).cuda()
    assert torch.equal(k[t], want[:, 0].reshape(-1, hkv * D)) and torch.equal(v[t], want[:, 1].reshape(-1, hkv * D))
    assert (k[b.rows:] == 3).all() and (v[b.rows:] == 3).all()
