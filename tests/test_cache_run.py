"""The cache calls in a row, as a server makes them (GPU): prefill in pieces,
then decode steps whose lengths torch operations advance between the calls,
nothing waited for; eager, and captured as one graph.  Each kernel may start
while the one in front of it ends, so what is checked is that every call sees
all that was written before it: results are bit for bit those of the same
calls with a synchronisation after each, and those are checked against the
definition."""
import pytest
import torch

import speculative_decoding_drafter_k3_gb300 as k3da
from cache_cases import Batch, D
from test_chunk_attn import check, dev

pytestmark = pytest.mark.gpu


class Server:
    """Requests over one cache; `steps` appends each step's tokens, attends
    and advances the lengths."""

    def __init__(self, b, norm):
        self.b, self.norm = b, norm
        self.pool, self.scales, _, self.table, self.lens, _ = dev(b)
        g = torch.Generator().manual_seed(31)
        self.chunks = [[5, 130, 1, 40], [1, 1, 1, 1], [1, 1, 1, 1], [3, 0, 17, 1], [1, 1, 1, 1]]
        self.inputs = []
        for new in self.chunks:
            T = sum(new)
            qkv = torch.randn(T, (b.hq + 2 * b.hkv) * D, generator=g).to(torch.bfloat16).cuda()
            cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
            step = torch.tensor(new, dtype=torch.int32, device="cuda")
            pos = torch.arange(T, dtype=torch.int32, device="cuda")
            ws = k3da.alloc_chunk_workspace(T, len(new), b.hq, b.hkv, b.stride)
            bufs = [torch.zeros(T, n * D, dtype=torch.bfloat16, device="cuda") for n in (b.hq, b.hq, b.hkv, b.hkv)]
            self.inputs.append((qkv, cu, step, pos, ws, *bufs, torch.zeros(T, b.hq, device="cuda")))
        self.start = [x.clone() for x in (self.pool.view(torch.uint8), self.lens)]
        self.w = b.q_w.cuda(), b.k_w.cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def reset(self):
        self.pool.view(torch.uint8).copy_(self.start[0])
        self.lens.copy_(self.start[1])
        for x in self.inputs:
            for t in x[5:]:
                t.zero_()

    def run(self, between=lambda: None):
        b = self.b
        kw = dict(num_kv_heads=b.hkv, kv_scales=self.scales, status=self.status)
        for qkv, cu, step, pos, ws, q, out, k, v, lse in self.inputs:
            if self.norm:
                k3da.k3da_kv_append_qknorm(self.pool, qkv, self.table, self.lens, cu, pos, *self.w, q_out=q, num_q_heads=b.hq, **kw)
            else:
                k3da.k3da_kv_append(self.pool, qkv, self.table, self.lens, cu, num_q_heads=b.hq, **kw)
            between()
            k3da.k3da_chunk_attn(out, q if self.norm else qkv[:, :b.hq * D], self.pool, self.table, self.lens, cu,
                                 num_q_heads=b.hq, lse=lse, workspace=ws, **kw)
            between()
            k3da.k3da_kv_gather(k, v, self.pool, self.table, self.lens, cu, **kw)
            between()
            self.lens.add_(step)
            between()

    def results(self):
        torch.cuda.synchronize()
        assert int(self.status) == 0
        return [t.clone() for x in self.inputs for t in x[5:]] + [self.pool.view(torch.uint8).clone(), self.lens.clone()]


def server(cache, norm, stride):
    b = Batch([160, 140, 30, 60], [3, 700, 64, 1500], 6, 1, cache, seed=30, stride=stride)
    return Server(b, norm)


@pytest.mark.parametrize("stride", [None, 1300])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_a_server_that_never_waits(cache, norm, stride):
    s = server(cache, norm, stride)
    s.run(between=torch.cuda.synchronize)
    want = s.results()
    for _ in range(10):
        s.reset()
        s.run()
        for a, b in zip(s.results(), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # As one graph.
    s.reset()
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s.run()
    for _ in range(5):
        s.reset()
        graph.replay()
        for a, b in zip(s.results(), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_every_step_against_the_definition(cache):
    """The last step's attention over a cache that the steps before wrote, and
    what the cache then holds."""
    s = server(cache, False, None)
    s.run()
    s.results()
    ctx = [c + sum(step[r] for step in s.chunks[:-1]) for r, c in enumerate(s.b.ctx)]
    last = Batch(s.chunks[-1], ctx, 6, 1, cache, seed=1, stride=s.b.stride)
    last.table, last.pool = s.table.cpu(), s.pool.cpu()
    last.scales = None if s.scales is None else s.scales.view(torch.uint8).cpu().view(torch.float8_e8m0fnu)
    last.qkv = s.inputs[-1][0].cpu()
    check(last, s.inputs[-1][6], s.inputs[-1][9])
    # The new tokens' K as gathered, and as the cache's definition has it.
    for r in range(4):
        want, wv = last.cached(r, ctx[r] + 1)
        assert torch.equal(s.inputs[-1][7][r].double().cpu(), want[ctx[r], 0])
        assert torch.equal(s.inputs[-1][8][r].double().cpu(), wv[ctx[r], 0])


def shifted(t):
    """A copy 16 bytes past a 256-byte boundary."""
    raw = torch.empty(t.numel() * t.element_size() + 16, dtype=torch.uint8, device="cuda")
    assert raw.data_ptr() % 256 == 0
    out = raw[16:].view(t.dtype if t.dtype.itemsize > 1 else torch.uint8).view(t.dtype).view(t.shape)
    out.view(torch.uint8).copy_(t.view(torch.uint8))
    return out


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_tensors_on_16_byte_boundaries(cache):
    """Nothing needs more alignment than the 16 bytes the calls ask for."""
    b = Batch([40, 1, 7], [300, 700, 5], 6, 1, cache, seed=33)
    results = []
    for place in (lambda t: t, shifted):
        pool, scales, qkv, table, lens, cu = dev(b)
        pool, qkv = place(pool), place(qkv)
        scales = None if scales is None else place(scales)
        q, out, k, v = (place(torch.zeros(b.T, n * D, dtype=torch.bfloat16, device="cuda")) for n in (6, 6, 1, 1))
        kw = dict(num_kv_heads=1, kv_scales=scales)
        k3da.k3da_kv_append_qknorm(pool, qkv, table, lens, cu, b.positions.cuda(), b.q_w.cuda(), b.k_w.cuda(), q_out=q,
                                   num_q_heads=6, **kw)
        ws = k3da.alloc_chunk_workspace(b.T, b.R, 6, 1, b.stride)
        k3da.k3da_chunk_attn(out, q, pool, table, lens, cu, num_q_heads=6, workspace=ws, **kw)
        k3da.k3da_kv_gather(k, v, pool, table, lens, cu, **kw)
        results.append([t.contiguous().view(torch.uint8).clone() for t in (pool, q, out, k, v)])
    for x, y in zip(*results):
        assert torch.equal(x, y)
