"""What a cache call writes may overlap nothing else that it is given: refused
on the host, pair by pair (CPU: every call made here is refused), and tensors
that touch without overlapping are taken (GPU)."""
import pytest
import torch

import speculative_decoding_drafter_k3_gb300 as k3da
from speculative_decoding_drafter_k3_gb300 import build as kbuild

T, R, HQ, HKV, PAGES, STRIDE = 64, 8, 24, 4, 16, 5
POOL, SCALES, QKV, ROWS_Q, ROWS_KV = PAGES * 2 * HKV * 64 * 64, PAGES * 2 * HKV * 64, T * (HQ + 2 * HKV) * 128, T * HQ * 128, T * HKV * 128


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return k3da.load_library()


def sizes(what, lib):
    """Bytes of every tensor, those that are written first."""
    ints = dict(table=R * STRIDE * 4, lens=R * 4, cu=(R + 1) * 4, status=4)
    if what == "gather":
        return dict(k=ROWS_KV, v=ROWS_KV), dict(pool=POOL, scales=SCALES, **ints)
    if what == "attn":
        return (dict(out=ROWS_Q, lse=T * HQ * 4, ws=lib.k3da_chunk_workspace_bytes(T, R, HQ, HKV, STRIDE)),
                dict(q=ROWS_Q, pool=POOL, scales=SCALES, **ints))
    if what == "append":
        return dict(pool=POOL, scales=SCALES), dict(qkv=QKV, **ints)
    return dict(pool=POOL, scales=SCALES, q_out=ROWS_Q), dict(qkv=QKV, positions=T * 8, qw=128, kw=128, **ints)


def call(what, lib, a):
    cache = [a["pool"], k3da.CACHE_E4M3, a["scales"], PAGES, a["table"], STRIDE, a["lens"], a["cu"], R]
    if what == "gather":
        return lib.k3da_kv_gather(a["k"], a["v"], *cache, T, HKV, 64, a["status"], None)
    if what == "attn":
        return lib.k3da_chunk_attn(a["out"], a["lse"], a["q"], HQ * 64, T, *cache, HQ, HKV, 64, 0, 0.125, a["ws"], 1 << 40,
                                   a["status"], None)
    if what == "append":
        return lib.k3da_kv_append(*cache, a["qkv"], T, HQ, HKV, 64, a["status"], None)
    return lib.k3da_kv_append_qknorm(*cache, a["qkv"], T, HQ, HKV, 64, a["positions"], k3da.POS_I64, a["qw"], a["kw"], 1e-5,
                                     1e4, None, a["q_out"], a["status"], None)


@pytest.mark.parametrize("what", ["append", "append_qknorm", "gather", "attn"])
def test_every_overlap_is_refused(lib, what):
    written, read = sizes(what, lib)
    size = {**written, **read}
    for w in written:
        for other in size:
            if other == w:
                continue
            step = 256 if "ws" in (w, other) else 16  # what a tensor's address has to be a multiple of
            end_w, end_o = (size[x] - 1 - (size[x] - 1) % step for x in (w, other))
            for a, b in ((0, 0), (0, end_w), (end_o, 0)):  # at the start, in the other's last bytes, the other way round
                at = {name: (i + 1) << 44 for i, name in enumerate(size)}
                at[w] += a
                at[other] = at[w] - a + b
                assert call(what, lib, at) == k3da.EINVAL, (w, other, a, b)


@pytest.mark.gpu
def test_tensors_that_touch_are_taken():
    """Everything of an append, an attention and a read-back in one piece of
    memory, end to end."""
    from cache_cases import Batch, D
    from test_chunk_attn import check, dev
    from test_kv_cache import bits
    b = Batch([40, 1], [90, 300], 6, 1, "e4m3", seed=51)
    src = dict(zip(("pool", "scales", "qkv", "table", "lens", "cu"), dev(b)))
    need = k3da.chunk_workspace_bytes(b.T, b.R, 6, 1, b.stride)
    src.update(out=torch.full((b.T, 6 * D), 7.0, dtype=torch.bfloat16, device="cuda"), ws=torch.zeros(need, dtype=torch.uint8, device="cuda"),
               lse=torch.full((b.T, 6), 7.0, device="cuda"), q=b.qkv[:, :6 * D].contiguous().cuda(),
               k=torch.zeros(b.T, D, dtype=torch.bfloat16, device="cuda"), v=torch.zeros(b.T, D, dtype=torch.bfloat16, device="cuda"))
    raw = torch.zeros(sum(t.numel() * t.element_size() + 256 for t in src.values()), dtype=torch.uint8, device="cuda")
    at, t = 0, {}
    for name in ("ws", "pool", "scales", "qkv", "out", "q", "k", "v", "lse", "table", "lens", "cu"):
        s = src[name]
        n = s.numel() * s.element_size()
        t[name] = raw[at:at + n].view(s.dtype).view(s.shape)
        t[name].view(torch.uint8).copy_(s.view(torch.uint8))
        at += n
        assert at % 4 == 0
    kw = dict(num_kv_heads=1, kv_scales=t["scales"])
    k3da.k3da_chunk_attn(t["out"], t["q"], t["pool"], t["table"], t["lens"], t["cu"], num_q_heads=6, lse=t["lse"],
                         workspace=t["ws"], **kw)
    check(b, t["out"], t["lse"])
    k3da.k3da_kv_append(t["pool"], t["qkv"], t["table"], t["lens"], t["cu"], num_q_heads=6, **kw)
    k3da.k3da_kv_gather(t["k"], t["v"], t["pool"], t["table"], t["lens"], t["cu"], **kw)
    k3da.k3da_kv_append(src["pool"], src["qkv"], src["table"], src["lens"], src["cu"], num_q_heads=6, num_kv_heads=1,
                        kv_scales=src["scales"])
    assert torch.equal(bits(t["pool"]), bits(src["pool"])) and torch.equal(bits(t["scales"]), bits(src["scales"]))
    for r, n in enumerate(b.new):
        pages = src["table"][r].long().cpu()
        for i in range(n):
            c = b.ctx[r] + i
            code = bits(src["pool"]).view(src["pool"].shape)[int(pages[c // 64]), :, 0, c % 64].view(torch.float8_e4m3fn).double()
            e = src["scales"].view(torch.uint8)[int(pages[c // 64]), :, 0, c % 64].double() - 127
            want = (code * torch.exp2(e)[:, None]).to(torch.bfloat16)
            assert torch.equal(t["k"][b.cu[r] + i], want[0]) and torch.equal(t["v"][b.cu[r] + i], want[1])
