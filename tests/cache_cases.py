"""Small batches over a paged cache, and the cache operators' definitions in
fp64 on the host: shared by the tests of append, gather and chunk attention."""
import math

import numpy as np
import torch

D, PAGE = 64, 64


def cu_of(new):
    return [0] + list(np.cumsum(new))


class Batch:
    """Requests with `new` tokens behind `ctx` cached ones; page ids are a
    random permutation, table entries no token needs are poisoned; `pad` rows
    behind the last sequence."""

    def __init__(self, new, ctx, hq, hkv, cache="bf16", pad=0, seed=0, stride=None, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.new, self.ctx, self.hq, self.hkv, self.cache, self.pad = list(new), list(ctx), hq, hkv, cache, pad
        self.R, self.rows = len(self.new), sum(self.new)
        self.T = self.rows + pad
        self.cu = cu_of(self.new)
        used = [-(-(c + n) // PAGE) for c, n in zip(self.ctx, self.new)]
        self.stride = stride or max(1, max(used))
        self.pages = max(1, sum(used)) + 2
        order = torch.randperm(self.pages, generator=g).tolist()
        table, at = [], 0
        for n in used:
            table.append(order[at:at + n] + [(-1) if k % 2 else 10 ** 6 for k in range(self.stride - n)])
            at += n
        self.table = torch.tensor(table, dtype=torch.int32)
        self.qkv = (torch.randn(self.T, (hq + 2 * hkv) * D, generator=g) * scale).to(torch.bfloat16)
        pool = (torch.randn(self.pages, 2, hkv, PAGE, D, generator=g)).to(torch.bfloat16)
        self.scales = None
        if cache == "e4m3":
            code, byte = quantise(pool.double())
            pool, self.scales = code, byte.view(torch.float8_e8m0fnu)
        self.pool = pool
        self.q_w = (1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16)
        self.k_w = (1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16)
        pos = [c + i for c, n in zip(self.ctx, self.new) for i in range(n)] + [7] * pad
        self.positions = torch.tensor(pos, dtype=torch.int32)

    @property
    def q(self):
        return self.qkv[:, :self.hq * D]

    def lens(self):
        return torch.tensor(self.ctx, dtype=torch.int32)

    def cu_t(self):
        return torch.tensor(self.cu, dtype=torch.int32)

    def where(self):
        """(row, page, slot) of every new token."""
        for r, n in enumerate(self.new):
            for i in range(n):
                c = self.ctx[r] + i
                yield self.cu[r] + i, int(self.table[r, c // PAGE]), c % PAGE

    def cached(self, r, length):
        """K, V [length, Hkv, 64] in fp64 of request r's first tokens."""
        pages = self.table[r, :-(-length // PAGE)].long()
        if self.scales is None:
            x = self.pool[pages].double()
        else:
            x = dequantise(self.pool.view(torch.uint8)[pages].view(torch.float8_e4m3fn), self.scales.view(torch.uint8)[pages])
        kv = x.permute(1, 0, 3, 2, 4).reshape(2, -1, self.hkv, D)[:, :length]
        return kv[0], kv[1]


def quantise(x):
    """(codes e4m3, scale bytes) of rows of 64 (fp64), by the definition."""
    top = x.abs().amax(-1)
    finite = torch.isfinite(x).all(-1)
    m, ex = torch.frexp(torch.where(finite, top, torch.ones_like(top)))
    e = (ex - 9 + (m > 0.875).int()).clamp(-127, 127)
    e = torch.where(top == 0, torch.full_like(e, -127), e)
    y = torch.where(finite[..., None], x, torch.zeros_like(x)) * torch.exp2(-e.double())[..., None]
    # Nearest e4m3 value, ties to even, in fp64 (fp64 -> fp32 -> e4m3 would round twice).
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    y = torch.round(y / step) * step
    byte = torch.where(finite, e + 127, torch.full_like(e, 255)).to(torch.uint8)
    return y.float().to(torch.float8_e4m3fn), byte


def dequantise(code, byte):
    s = torch.exp2(byte.double() - 127.0)
    s = torch.where(byte == 255, torch.full_like(s, math.nan), s)
    return code.float().double() * s[..., None]


def attend(b, mask, scale=0.125, rows=None):
    """(out, lse, weighted |v|, largest sum |q k| scale) in fp64: out
    [T, Hq, 64], lse [T, Hq]; rows of nobody are NaN."""
    out = torch.full((b.T, b.hq, D), math.nan, dtype=torch.float64)
    lse = torch.full((b.T, b.hq), math.nan, dtype=torch.float64)
    mag = torch.zeros(b.T, b.hq, D, dtype=torch.float64)
    grain = 0.0
    G = b.hq // b.hkv
    for r, n in enumerate(b.new):
        if not n:
            continue
        limit = b.ctx[r] + (0 if mask == "context" else n)
        k, v = b.cached(r, limit)
        for i in range(n):
            t = b.cu[r] + i
            seen = b.ctx[r] + i + 1 if mask == "causal" else limit
            q = b.q[t].double().view(b.hkv, G, D)
            x = torch.einsum("hgd,chd->hgc", q, k[:seen]) * scale
            if seen:
                grain = max(grain, float(torch.einsum("hgd,chd->hgc", q.abs(), k[:seen].abs()).nan_to_num(0, 0, 0).max()) * scale)
                p = torch.softmax(x, -1)
                out[t] = torch.einsum("hgc,chd->hgd", p, v[:seen]).reshape(b.hq, D)
                mag[t] = torch.einsum("hgc,chd->hgd", p, v[:seen].abs()).reshape(b.hq, D)
                lse[t] = torch.logsumexp(x, -1).reshape(b.hq)
            else:
                out[t] = 0
                lse[t] = -math.inf
    return out, lse, mag, grain
