"""k3da_chunk_attn on batches that mix what its kernels handle apart: chunks
of at most 16 query rows a kv head beside long ones, key tiles shared by an
item's slots or taken in turn, items cut over many CTAs (GPU).

Tolerances: those of the definition (see test_chunk_attn.py).  Weights that
meet codes are half precision (2^-12 of themselves, less than the bf16 bound),
but those below 2^-14 of the reference are off by 2^-25 of it, and the
reference is at most 2^10 above the row's largest: 2^-15 of that a key, within
the 2^-10 that the bound allows for the fp32 rest."""
import numpy as np
import pytest
import torch

import speculative_decoding_drafter_k3_gb300 as k3da
from cache_cases import Batch, D
from test_chunk_attn import BATCHES, HEADS, MASKS, call, check, dev

pytestmark = pytest.mark.gpu


WIDE = 1300  # pages a request: a table for which a call is not small, whatever the lengths


def random_batch(seed, cache, hq=6, hkv=1):
    g = np.random.default_rng(seed)
    R = int(g.integers(20, 120))
    sizes = [0, 1, 1, 1, 2, 3, 16 * hkv // hq, 16 * hkv // hq + 1, 21, 22, 40, 43, 85, 130]
    new = [int(g.choice(sizes)) for _ in range(R)]
    ctx = [int(g.integers(0, 40 + 400 * (seed % 4))) for _ in range(R)]
    return Batch(new, ctx, hq, hkv, cache, pad=3, seed=seed, stride=WIDE if seed % 2 else None)


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("new,ctx,pad", BATCHES + [([2] * 8 + [3], [70 * r for r in range(9)], 1)])
def test_small_lengths_in_wide_tables(new, ctx, pad, hq, hkv, cache, mask):
    b = Batch(new, ctx, hq, hkv, cache, pad, seed=sum(new) + hq, stride=WIDE)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = call(b, mask, status=status)
    assert int(status) == 0
    check(b, out, lse, mask)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("seed,hq,hkv", [(1, 6, 1), (2, 24, 4), (3, 6, 1), (4, 16, 2), (5, 12, 2)])
def test_mixed_batches(seed, hq, hkv, cache):
    """Against the definition, and bit by bit the same with a cold L2: what
    runs beside what then is another matter."""
    b = random_batch(seed, cache, hq, hkv)
    d = dev(b)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = call(b, d=d, status=status)
    check(b, out, lse)
    ws = k3da.alloc_chunk_workspace(b.T, b.R, hq, hkv, b.stride)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(12):
        if i % 2:
            flush.fill_(i)
        again, alse = call(b, d=d, ws=ws, status=status)
        assert torch.equal(again.view(torch.int16), out.view(torch.int16)) and torch.equal(alse, lse)
    assert int(status) == 0


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv", [(g, 1) for g in range(1, 17)] + [(33, 11), (64, 64), (64, 4)])
def test_every_group_of_heads(hq, hkv, cache):
    """Rows to a slot and to a small chunk by the heads that share a kv head."""
    b = Batch([1, 130 // hkv + 3, 2, 17, 0, 3], [70, 10, 200, 63, 5, 129], hq, hkv, cache, pad=1, seed=hq, stride=WIDE)
    out, lse = call(b)
    check(b, out, lse)


def test_items_whose_slots_end_apart():
    """The second slot of an item sees a tile more than the first, behind
    items of one slot, over and over."""
    new = [43 if r % 3 == 0 else 40 if r % 3 == 1 else 1 for r in range(300)]
    ctx = [(97 * r) % 700 - (97 * r) % 700 % 128 + 128 - 21 for r in range(300)]  # the 21st token's last key ends a tile
    b = Batch(new, ctx, 6, 1, "bf16", seed=6)
    d = dev(b)
    out, lse = call(b, d=d)
    check(b, out, lse)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(20):
        flush.fill_(i)
        again, alse = call(b, d=d)
        assert torch.equal(again.view(torch.int16), out.view(torch.int16)) and torch.equal(alse, lse)


@pytest.mark.parametrize("new,hq", [([1, 1], 6), ([2, 1], 6), ([3], 5), ([1], 16), ([60], 6)])
@pytest.mark.parametrize("spread", [3, 9, 14, 25])
def test_rows_of_very_different_scales(new, hq, spread):
    """V's exponents close together, at the border, far apart, and with them
    rows of zeros (the smallest scale there is); K's a little apart."""
    b = Batch(new, [900, 70][:len(new)], hq, 1, "e4m3", seed=20 + spread, stride=WIDE)
    g = torch.Generator().manual_seed(spread)
    byte = b.scales.view(torch.uint8)
    low = torch.randint(0, spread + 1, byte.shape, generator=g, dtype=torch.uint8)
    low[:, 0] = low[:, 0].clamp(max=2)
    byte -= low
    out, lse = call(b)
    check(b, out, lse)
    page, slot = int(b.table[0, 5]), 17  # one key's K and V are zeros
    b.pool.view(torch.uint8)[page, :, 0, slot] = 0
    byte[page, :, 0, slot] = 0
    out, lse = call(b)
    check(b, out, lse)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("new,hq,ctx", [([2], 6, [125]), ([3], 5, [126]), ([2], 8, [63]), ([16], 1, [120])])
def test_a_nan_in_a_small_chunk_reaches_only_rows_that_see_it(new, hq, ctx, what, cache):
    b = Batch(new, ctx, hq, 1, cache, seed=12, stride=WIDE)
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
@pytest.mark.parametrize("at", [40, 122])
def test_an_infinite_value_in_a_small_chunk(value, at):
    b = Batch([4], [120], 4, 1, "bf16", seed=13)
    b.pool[int(b.table[0, at // 64]), 1, 0, at % 64, 3] = value
    out, lse = call(b)
    got = out.cpu().double().view(4, 4, D)
    first = max(0, at - 120)
    assert torch.isfinite(got[:first]).all() and (got[first:, :, 3] == value).all()
    others = [d for d in range(D) if d != 3]
    assert torch.isfinite(got[:, :, others]).all()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_bad_pages_of_a_small_chunk_are_zeros(cache):
    b = Batch([1, 2], [300, 62], 6, 1, cache, seed=14, stride=WIDE)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = list(dev(b))
    d[3] = d[3].clone()
    d[3][0, 2] = -3
    out, lse = call(b, d=d, status=status)
    assert int(status) == k3da.STATUS_BAD_PAGE
    b.pool.view(torch.uint8)[int(b.table[0, 2])] = 0
    if cache == "e4m3":
        b.scales.view(torch.uint8)[int(b.table[0, 2])] = 0
    check(b, out, lse)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_many_long_contexts_over_the_same_pages(cache):
    """64 requests that share one cache of 60000 tokens: pieces of hundreds of
    pages."""
    R, ctx = 64, 60000
    one = Batch([1], [ctx], 6, 1, cache, seed=21)
    pool, scales, _, table, _, _ = dev(one)
    g = torch.Generator().manual_seed(22)
    q = torch.randn(R, 6 * D, generator=g).to(torch.bfloat16).cuda()
    out, lse = torch.empty_like(q), torch.empty(R, 6, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k3da.k3da_chunk_attn(out, q, pool, table.expand(R, -1).contiguous(), torch.full((R,), ctx, dtype=torch.int32, device="cuda"),
                         torch.arange(R + 1, dtype=torch.int32, device="cuda"), num_q_heads=6, num_kv_heads=1,
                         kv_scales=scales, lse=lse, workspace=k3da.alloc_chunk_workspace(R, R, 6, 1, one.stride), status=status)
    assert int(status) == 0
    k, v = (x[:, 0].cuda() for x in one.cached(0, ctx + 1))
    x = q.double().view(-1, D) @ k.T * 0.125
    p = torch.softmax(x, -1)
    want, mag = p @ v, p @ v.abs()
    err = (out.double().view(-1, D) - want).abs() - (2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -10) * mag)
    assert err.max() <= 1e-7
    grain = float((q.double().view(-1, D).abs() @ k.abs().T).max()) * 0.125
    wlse = torch.logsumexp(x, -1)
    assert ((lse.double().view(-1) - wlse).abs() <= (64 * grain + ctx) * 2.0 ** -24 + 2.0 ** -21 * (1 + wlse.abs())).all()


def test_two_captured_graphs_share_a_workspace():
    """Replayed one after the other on a stream, in either order."""
    bs = [Batch([1] * 9, [700 * r for r in range(9)], 6, 1, "bf16", seed=23, stride=WIDE), Batch([60, 1, 130], [1000, 9000, 40], 6, 1, "bf16", seed=24)]
    ds = [dev(b) for b in bs]
    want = [call(b, d=d) for b, d in zip(bs, ds)]
    ws = k3da.alloc_chunk_workspace(max(b.T for b in bs), 9, 6, 1, max(b.stride for b in bs))
    outs = [(torch.empty_like(o), torch.empty_like(l)) for o, l in want]
    s, graphs = torch.cuda.Stream(), []
    torch.cuda.synchronize()
    for b, d, (o, l) in zip(bs, ds, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call(b, d=d, out=o, lse=l, ws=ws, stream=s)
        graphs.append(graph)
    for order in ([0, 1], [1, 0], [0, 0, 1, 1, 0]):
        for o, l in outs:
            o.zero_()
            l.zero_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for (o, l), (x, y) in zip(outs, want):
            assert torch.equal(o.view(torch.int16), x.view(torch.int16)) and torch.equal(l, y)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_small_chunks_far_into_a_large_pool(cache):
    """Byte offsets past 2^32 (codes: past 2^31), and in the appends and the
    read-back of the same pages."""
    b = Batch([1, 2], [200, 77], 24, 4, cache, seed=10)
    pool, scales, qkv, table, lens, cu = dev(b)
    pages = 90000 if cache == "bf16" else 100000
    shift = pages - b.pages
    big = torch.zeros(pages, 2, 4, 64, D * pool.element_size(), dtype=torch.uint8, device="cuda")
    big[shift:] = pool.view(torch.uint8).view(b.pages, 2, 4, 64, -1)
    big = big.view(pool.dtype)
    if scales is not None:
        large = torch.zeros(pages, 2, 4, 64, dtype=torch.uint8, device="cuda")
        large[shift:] = scales.view(torch.uint8)
        large = large.view(scales.dtype)
    moved = torch.where((table >= 0) & (table < b.pages), table + shift, table)
    d = big, None if scales is None else large, qkv, moved, lens, cu
    out, lse = call(b, d=d)
    check(b, out, lse)
    k3da.k3da_kv_append(big, qkv, moved, lens, cu, num_q_heads=24, num_kv_heads=4, kv_scales=d[1])
    k3da.k3da_kv_append(pool, qkv, table, lens, cu, num_q_heads=24, num_kv_heads=4, kv_scales=scales)
    assert torch.equal(big[shift:].view(torch.uint8), pool.view(torch.uint8)) and not big[:shift].view(torch.uint8).any()
    got = [torch.zeros(3, 4 * D, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    k3da.k3da_kv_gather(*got[:2], big, moved, lens, cu, num_kv_heads=4, kv_scales=d[1])
    k3da.k3da_kv_gather(*got[2:], pool, table, lens, cu, num_kv_heads=4, kv_scales=scales)
    assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3]) and got[0].any()
    del big, d
    torch.cuda.empty_cache()
