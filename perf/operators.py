"""Cases of the paged-cache operators: appending a chunk's K/V to the cache
(bf16, or e4m3 with one power-of-two scale per token and head), reading
cached tokens back, and attention of ragged chunks of new tokens over the
cache.

``run`` computes a case in its plain form (elementary torch operations in
fp32), or, with ``own`` set, through this package's calls.  ``exact`` gives
the same outputs from the definitions in fp64.

Layouts (D = 64, pages of 64 tokens):
  qkv         [T, (Hq + 2*Hkv)*64] bf16, rows of all requests one after the
              other, request r's at cu_seqlens[r] .. cu_seqlens[r+1]
  pool        [pages, 2, Hkv, 64, 64] bf16 or e4m3
  scales      [pages, 2, Hkv, 64] e8m0, for an e4m3 pool
  page_table  [R, S] int32; cache token c of request r is in slot c % 64 of
              page page_table[r, c // 64]
  ctx_lens    [R] int32, tokens already cached; token i of the chunk is cache
              token ctx_lens[r] + i
"""
import math
import random

import torch

own = False

D = 64
PAGE = 64
EPS = 1e-5
BASE = 10000.0
SCALE = 0.125


# --------------------------------------------------------------- the cases --

def _case(name, op, cache, hq, hkv, requests, tokens, ctx_lo, ctx_hi, lengths, mask="causal", norm=False, pad=0):
    """tokens: new (or read) tokens of the longest request; lengths: what the
    others have ("same", or "ragged": down to a single one, and now and then
    none); ctx_lo .. ctx_hi: tokens cached before; pad: rows behind the last
    sequence."""
    return {"name": name, "op": op, "cache": cache, "hq": hq, "hkv": hkv, "requests": requests, "tokens": tokens,
            "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "lengths": lengths, "mask": mask, "norm": norm, "pad": pad}


def listed():
    return [
        # One request generating its next token: nothing but latency.
        _case("attn token 6/1", "attn", "bf16", 6, 1, 1, 1, 300, 300, "same"),
        # A serving batch, one new token each, over a quantised cache.
        _case("attn decode 64 e4m3", "attn", "e4m3", 24, 4, 64, 1, 16, 8191, "same"),
        # The target's check of 8 draft tokens of 8 long conversations.
        _case("attn verify 8x8 long", "attn", "bf16", 24, 4, 8, 8, 16384, 131072, "same"),
        # A prefill step that mixes chunks of many sizes, rows of padding behind.
        _case("attn prefill mixed", "attn", "bf16", 24, 4, 6, 2041, 0, 4096, "ragged", pad=37),
        # A long prompt's second half over a quantised cache.
        _case("attn prefill 8k e4m3", "attn", "e4m3", 24, 4, 1, 8192, 8192, 8192, "same"),
        # The drafter's blocks over their contexts alone (some still empty),
        # to be merged with the blocks' own part by the returned lse.
        _case("attn context 8x6 6/1", "attn", "bf16", 6, 1, 8, 6, 0, 2041, "same", mask="context"),
        # A block of 8 drafted tokens joins the cache: norm, RoPE and write.
        _case("append block 6/1", "append", "bf16", 6, 1, 1, 8, 300, 300, "same", norm=True),
        # A decode step of a large batch, quantised as it is written.
        _case("append 256 tokens e4m3", "append", "e4m3", 24, 4, 256, 1, 0, 2041, "same", norm=True, pad=5),
        # A prefill step, quantised as it is written.
        _case("append prefill e4m3", "append", "e4m3", 24, 4, 8, 4099, 0, 4096, "ragged", norm=True),
        # A prefill step whose k is normalised and roped already.
        _case("append prefill bf16", "append", "bf16", 24, 4, 4, 8192, 0, 4096, "ragged"),
        # One conversation's cache read back.
        _case("gather 2041 6/1", "gather", "bf16", 6, 1, 1, 2041, 0, 0, "same"),
        # Long conversations read back from a quantised cache.
        _case("gather long e4m3", "gather", "e4m3", 24, 4, 4, 65536, 0, 1000, "ragged"),
    ]


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of its range."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    while True:
        hq, hkv = rng.choice([(6, 1), (24, 4), (24, 4), (12, 2), (8, 8), (16, 2)])
        c = _case("", rng.choice(["attn", "attn", "append", "gather"]), rng.choice(["bf16", "e4m3"]), hq, hkv,
                  _between(rng, 1, 256), 1, 0, _between(rng, 1, 131072), rng.choice(["same", "ragged"]),
                  pad=rng.choice([0, 0, 1, 40]))
        del c["name"]
        c["ctx_lo"] = rng.randrange(c["ctx_hi"] + 1) if rng.random() < 0.5 else 0
        if c["op"] == "attn":
            c["tokens"] = _between(rng, 1, 8192) if rng.random() < 0.6 else rng.randrange(1, 9)
            c["mask"] = rng.choice(["causal", "causal", "causal", "full", "context"])
        else:
            c["tokens"] = _between(rng, 1, 65536)
            c["norm"] = c["op"] == "append" and rng.random() < 0.6
        new, ctx, cu, kv = _lengths(c)
        if kv * c["hkv"] * c["requests"] > 8 * 4 * 131080 or cu[-1] * c["hq"] > 24 * 131072:
            continue
        if c["op"] == "attn" and (c["requests"] * max(new) * kv * hq > 2.5e9 or work(c)["flops"] > 5e11):
            continue
        return c


def _lengths(case):
    """(new tokens, cached tokens, first rows, longest cache) of the requests:
    fixed by the case."""
    g = random.Random("%(requests)d %(tokens)d %(ctx_lo)d %(ctx_hi)d" % case)
    new, ctx = [], []
    for r in range(case["requests"]):
        n = case["tokens"]
        if case["lengths"] == "ragged" and r:
            n = 0 if g.random() < 0.05 else _between(g, 1, n)
        new.append(n)
        ctx.append(g.randint(case["ctx_lo"], case["ctx_hi"]))
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return new, ctx, cu, max(c + n for c, n in zip(ctx, new))


def _pages(case):
    new, ctx, cu, kv = _lengths(case)
    stride = -(-kv // PAGE)
    used = [-(-(c + n) // PAGE) for c, n in zip(ctx, new)]
    return stride, used, sum(used) + 3


# ---------------------------------------------------------------- the work --

def work(case):
    new, ctx, cu, _ = _lengths(case)
    hq, hkv, rows = case["hq"], case["hkv"], cu[-1]
    slot = 2 * D * 2 if case["cache"] == "bf16" else 2 * (D + 1)  # K and V of one token and head
    ids = 4 * sum(_pages(case)[1]) + 4 * (2 * case["requests"] + 1)
    if case["op"] == "attn":
        if case["mask"] == "causal":
            seen, keys = sum(n * c + n * (n + 1) // 2 for n, c in zip(new, ctx)), sum(c + n for n, c in zip(new, ctx) if n)
        elif case["mask"] == "full":
            seen, keys = sum(n * (c + n) for n, c in zip(new, ctx)), sum(c + n for n, c in zip(new, ctx) if n)
        else:
            seen, keys = sum(n * c for n, c in zip(new, ctx)), sum(c for n, c in zip(new, ctx) if n)
        return {"bytes": keys * hkv * slot + rows * hq * (2 * D * 2 + 4) + ids, "flops": 4 * D * hq * seen}
    if case["op"] == "append":
        moved = rows * hkv * (2 * D * 2 + slot)
        if case["norm"]:
            moved += rows * (hq * 2 * D * 2 + 4)
        return {"bytes": moved + ids, "flops": 10 * D * rows * (hkv + (hq + hkv if case["norm"] else 0))}
    return {"bytes": rows * hkv * (slot + 2 * D * 2) + ids, "flops": rows * hkv * 2 * D}


# -------------------------------------------------------------- the inputs --

def _quantise(x):
    """Rows of 64 as e4m3 codes and their scales' exponents + 127: the
    smallest power of two that brings the row's largest magnitude to at most
    448."""
    top, ex = torch.frexp(x.abs().amax(-1))
    e = torch.where(top > 0, ex - 9 + (top > 0.875).int(), -127).clamp(-127, 127)
    code = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn)
    return code, (e + 127).to(torch.uint8)


def prepare(case, seed):
    new, ctx, cu, kv = _lengths(case)
    stride, used, pages = _pages(case)
    R, hq, hkv, T = case["requests"], case["hq"], case["hkv"], cu[-1] + case["pad"]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)

    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).tolist()
    table, at = [], 0
    for n in used:
        table.append(order[at:at + n] + [-1] * (stride - n))
        at += n

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    s = {"case": dict(case), "rows": cu[-1], "new": max(new), "kv": kv, "page_table": ints(table), "ctx_lens": ints(ctx),
         "cu_seqlens": ints(cu), "scales": None}
    pool = normal(pages, 2, hkv, PAGE, D)
    if case["cache"] == "e4m3":
        codes = torch.empty(pool.shape, dtype=torch.float8_e4m3fn, device="cuda")
        scales = torch.empty(pool.shape[:-1], dtype=torch.uint8, device="cuda")
        for a in range(0, pages, 4096):
            codes[a:a + 4096], scales[a:a + 4096] = _quantise(pool[a:a + 4096].float())
        pool, s["scales"] = codes, scales.view(torch.float8_e8m0fnu)
    s["pool"] = pool
    if case["op"] == "attn":
        s["q"] = normal(T, (hq + 2 * hkv) * D)[:, :hq * D]  # the q heads of the chunk's qkv rows
        s["out"] = torch.zeros(T, hq * D, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros(T, hq, dtype=torch.float32, device="cuda")
    elif case["op"] == "append":
        s["qkv"] = normal(T, (hq + 2 * hkv) * D)
        if case["norm"]:
            s["q_w"], s["k_w"] = (1 + 0.1 * normal(2, D).float()).to(torch.bfloat16).unbind(0)
            row = torch.arange(T, device="cuda")
            r = torch.searchsorted(s["cu_seqlens"][1:].long(), row, right=True).clamp(max=R - 1)
            s["positions"] = (s["ctx_lens"][r] + row - s["cu_seqlens"][r]).to(torch.int32)
            s["q"] = torch.zeros(T, hq * D, dtype=torch.bfloat16, device="cuda")
    else:
        s["k"] = torch.zeros(T, hkv * D, dtype=torch.bfloat16, device="cuda")
        s["v"] = torch.zeros(T, hkv * D, dtype=torch.bfloat16, device="cuda")
    if own and case["op"] == "attn":
        import speculative_decoding_drafter_k3_gb300 as k3da
        s["workspace"] = k3da.alloc_chunk_workspace(T, R, hq, hkv, stride)
    return s


# ---------------------------------------------------------- the plain form --

def _where(s):
    """(page, slot) in the pool of every row's cache token."""
    row = torch.arange(s["rows"], device="cuda")
    r = torch.searchsorted(s["cu_seqlens"][1:].long(), row, right=True)
    c = s["ctx_lens"][r].long() + row - s["cu_seqlens"][r]
    return s["page_table"][r, c // PAGE].long(), c % PAGE


def _norm_rope(x, w, turn):
    """RMSNorm over the 64 dims of a head, then NeoX RoPE by the angles."""
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    cos, sin = turn.cos().float()[:, None], turn.sin().float()[:, None]
    a, b = y[..., :D // 2], y[..., D // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(s):
    c, n = s["case"], s["rows"]
    hq, hkv = c["hq"], c["hkv"]
    x = s["qkv"][:n].view(n, hq + 2 * hkv, D)
    k, v = x[:, hq:hq + hkv].float(), x[:, hq + hkv:].float()
    if c["norm"]:
        rate = BASE ** (torch.arange(D // 2, device="cuda", dtype=torch.float64) * (-2 / D))
        turn = s["positions"][:n, None].double() * rate
        s["q"][:n] = _norm_rope(x[:, :hq].float(), s["q_w"], turn).reshape(n, hq * D).to(torch.bfloat16)
        k = _norm_rope(k, s["k_w"], turn)
    page, slot = _where(s)
    if c["cache"] == "bf16":
        s["pool"][page, 0, :, slot] = k.to(torch.bfloat16)
        s["pool"][page, 1, :, slot] = v.to(torch.bfloat16)
    else:
        pool, scales = s["pool"].view(torch.uint8), s["scales"].view(torch.uint8)
        code, e = _quantise(torch.stack([k, v], 1))
        pool[page, :, :, slot] = code.view(torch.uint8)
        scales[page, :, :, slot] = e


def _values(s, page, kv, slot):
    """Cached rows [..., Hkv, 64] in fp32."""
    if s["scales"] is None:
        return s["pool"][page, kv, :, slot].float()
    x = s["pool"].view(torch.uint8)[page, kv, :, slot].view(torch.float8_e4m3fn).float()
    e = s["scales"].view(torch.uint8)[page, kv, :, slot].int() - 127
    return torch.ldexp(x, e[..., None])


def _plain_gather(s):
    n = s["rows"]
    page, slot = _where(s)
    s["k"][:n] = _values(s, page, 0, slot).reshape(n, -1).to(torch.bfloat16)
    s["v"][:n] = _values(s, page, 1, slot).reshape(n, -1).to(torch.bfloat16)


def _plain_attn(s):
    c, L, N = s["case"], s["kv"], s["new"]
    hq, hkv, R = c["hq"], c["hkv"], c["requests"]
    first, ctx = s["cu_seqlens"][:-1].long(), s["ctx_lens"].long()
    n = s["cu_seqlens"][1:].long() - first
    i, j = torch.arange(N, device="cuda"), torch.arange(L, device="cuda")
    row = (first[:, None] + i).clamp(max=s["q"].shape[0] - 1)                   # [R, N]
    q = s["q"][row].view(R, N, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4).float().reshape(R, hkv, -1, D)
    page = s["page_table"][:, j // PAGE].long().clamp(min=0)                    # [R, L]
    k = _values(s, page, 0, (j % PAGE).expand(R, L)).transpose(1, 2)            # [R, Hkv, L, 64]
    x = torch.matmul(q, k.transpose(-1, -2)).view(R, hkv, hq // hkv, N, L).mul_(SCALE)
    del k
    if c["mask"] == "causal":
        seen = j <= (ctx[:, None] + i)[..., None]
    elif c["mask"] == "full":
        seen = j < (ctx + n)[:, None, None].expand(R, N, 1)
    else:
        seen = j < ctx[:, None, None].expand(R, N, 1)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m.clamp(min=-3e38)).exp_()
    total = p.sum(-1)
    v = _values(s, page, 1, (j % PAGE).expand(R, L)).transpose(1, 2)
    o = torch.matmul(p.view(R, hkv, -1, L), v).view(R, hkv, hq // hkv, N, D)
    o = o / total.clamp(min=1e-30)[..., None]
    lse = m[..., 0] + total.log()
    real = i < n[:, None]                                                       # [R, N]
    s["out"][:s["rows"]] = o.permute(0, 3, 1, 2, 4)[real].reshape(-1, hq * D).to(torch.bfloat16)
    s["lse"][:s["rows"]] = lse.permute(0, 3, 1, 2)[real].reshape(-1, hq)


# ------------------------------------------------------ the package's calls --

def _own_append(s):
    import speculative_decoding_drafter_k3_gb300 as k3da
    c = s["case"]
    heads = dict(num_q_heads=c["hq"], num_kv_heads=c["hkv"], kv_scales=s["scales"])
    if c["norm"]:
        k3da.k3da_kv_append_qknorm(s["pool"], s["qkv"], s["page_table"], s["ctx_lens"], s["cu_seqlens"], s["positions"],
                                   s["q_w"], s["k_w"], q_out=s["q"], eps=EPS, rope_base=BASE, **heads)
    else:
        k3da.k3da_kv_append(s["pool"], s["qkv"], s["page_table"], s["ctx_lens"], s["cu_seqlens"], **heads)


def _own_gather(s):
    import speculative_decoding_drafter_k3_gb300 as k3da
    k3da.k3da_kv_gather(s["k"], s["v"], s["pool"], s["page_table"], s["ctx_lens"], s["cu_seqlens"],
                        num_kv_heads=s["case"]["hkv"], kv_scales=s["scales"])


def _own_attn(s):
    import speculative_decoding_drafter_k3_gb300 as k3da
    c = s["case"]
    k3da.k3da_chunk_attn(s["out"], s["q"], s["pool"], s["page_table"], s["ctx_lens"], s["cu_seqlens"],
                         num_q_heads=c["hq"], num_kv_heads=c["hkv"], softmax_scale=SCALE, mask=c["mask"],
                         kv_scales=s["scales"], lse=s["lse"], workspace=s["workspace"])


def run(state):
    op = state["case"]["op"]
    if op == "attn":
        _own_attn(state) if own else _plain_attn(state)
        return {"out": state["out"], "lse": state["lse"]}
    if op == "gather":
        _own_gather(state) if own else _plain_gather(state)
        return {"k": state["k"], "v": state["v"]}
    _own_append(state) if own else _plain_append(state)
    got = {"pool": state["pool"]}
    if state["scales"] is not None:
        got["scales"] = state["scales"]
    if state["case"]["norm"]:
        got["q"] = state["q"]
    return got


# --------------------------------------------- the definitions, in 64 bits --

def _exact_cache(s):
    """The whole pool's values in fp64."""
    x = s["pool"].double()
    if s["scales"] is None:
        return x
    return x * torch.exp2(s["scales"].view(torch.uint8).double() - 127.0)[..., None]


def _exact_rope(x, w, pos):
    """x [tokens, heads, 64] in fp64."""
    x = x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()
    z = torch.complex(x[..., :D // 2], x[..., D // 2:])
    j = torch.arange(D // 2, device=x.device, dtype=torch.float64)
    angle = pos.double()[:, None] * torch.exp(-(2 * j / D) * math.log(BASE))
    z = z * torch.polar(torch.ones_like(angle), angle)[:, None]
    return torch.cat([z.real, z.imag], -1)


def _exact_append(s, new, ctx, cu):
    c = s["case"]
    hq, hkv = c["hq"], c["hkv"]
    quantised = c["cache"] == "e4m3"
    pool = s["pool"].double()
    scales = torch.exp2(s["scales"].view(torch.uint8).double() - 127.0) if quantised else None
    q = s["q"].double() if c["norm"] else None
    for r, n in enumerate(new):
        if not n:
            continue
        x = s["qkv"][cu[r]:cu[r] + n].double().reshape(n, -1, D)
        k, v = x[:, hq:hq + hkv], x[:, hq + hkv:]
        pos = torch.arange(ctx[r], ctx[r] + n, device="cuda")
        if c["norm"]:
            q[cu[r]:cu[r] + n] = _exact_rope(x[:, :hq], s["q_w"], pos).reshape(n, -1)
            k = _exact_rope(k, s["k_w"], pos)
        page = s["page_table"][r].long()[pos // PAGE]
        for kv, y in ((0, k), (1, v)):
            if quantised:
                top = y.abs().amax(-1)
                e = torch.ceil(torch.log2(top / 448.0))
                scales[page, kv, :, pos % PAGE] = torch.exp2(e)
                y = y * torch.exp2(-e)[..., None]
                step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
                y = torch.round(y / step) * step
            pool[page, kv, :, pos % PAGE] = y
    got = {"pool": pool}
    if quantised:
        got["scales"] = scales
    if c["norm"]:
        got["q"] = q
    return got


def _exact_gather(s, new, ctx, cu):
    cache = _exact_cache(s)
    got = {"k": s["k"].double(), "v": s["v"].double()}
    for r, n in enumerate(new):
        pos = torch.arange(ctx[r], ctx[r] + n, device="cuda")
        page = s["page_table"][r].long()[pos // PAGE]
        for kv, name in enumerate("kv"):
            got[name][cu[r]:cu[r] + n] = cache[page, kv, :, pos % PAGE].flatten(1)
    return got


def _exact_attn(s, new, ctx, cu):
    c = s["case"]
    hq, hkv = c["hq"], c["hkv"]
    cache = s["pool"]
    out, lse = s["out"].double(), s["lse"].double()
    for r, n in enumerate(new):
        limit = ctx[r] + (n if c["mask"] != "context" else 0)
        page = s["page_table"][r].long()[:-(-limit // PAGE)]
        mine = cache[page].double()
        if s["scales"] is not None:
            mine = mine * torch.exp2(s["scales"].view(torch.uint8)[page].double() - 127.0)[..., None]
        for h in range(hkv):
            k = mine[:, 0, h].reshape(-1, D)[:limit]
            v = mine[:, 1, h].reshape(-1, D)[:limit]
            for a in range(0, n, 512):
                rows = slice(cu[r] + a, cu[r] + min(n, a + 512))
                q = s["q"][rows].double().reshape(-1, hq, D)[:, h * (hq // hkv):(h + 1) * (hq // hkv)]
                x = torch.einsum("tgd,ld->tgl", q, k) * SCALE
                if c["mask"] == "causal":
                    pos = ctx[r] + a + torch.arange(q.shape[0], device="cuda")
                    x = torch.where(torch.arange(limit, device="cuda") > pos[:, None, None], -math.inf, x)
                got = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
                total = torch.logsumexp(x, -1) if limit else torch.full(x.shape[:2], -math.inf, device="cuda", dtype=torch.float64)
                weights = torch.exp(x - torch.where(total.isinf(), 0.0, total)[..., None])
                lse[rows, got] = total
                out[rows].view(-1, hq, D)[:, got] = torch.einsum("tgl,ld->tgd", weights, v)
    return {"out": out, "lse": lse}


def exact(case, seed):
    new, ctx, cu, _ = _lengths(case)
    if case["op"] == "attn" and work(case)["flops"] > 1.5e12:
        return None
    s = prepare(case, seed)
    return {"append": _exact_append, "gather": _exact_gather, "attn": _exact_attn}[case["op"]](s, new, ctx, cu)
