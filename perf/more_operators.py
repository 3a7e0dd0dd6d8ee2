"""Cases of the operators around a drafter's cache: probabilities of logits,
verification of drafted tokens, and the pages of the cache (taking and giving
back, forking, compacting, copying).

``run`` computes a case in its plain form (elementary torch operations), or,
with ``own`` set, through this package's calls.  ``exact`` gives the same
outputs from the definitions: in fp64, or, for whole numbers, step by step on
the host.

Layouts (pages of 64 tokens):
  rows        packed rows of all requests, request r's at
              cu_seqlens[r] .. cu_seqlens[r+1]; rows behind are nobody's
  logits      [T, V], rows possibly further apart (a padded vocabulary)
  tokens      [T] the rows' tokens: a request's first is known, the others are
              drafts; row i's probabilities are those of the token behind it
  page_table  [R, S] int32, page ids; entries past ceil(lens / 64) are -1
  lens        [R] int32 tokens a row holds pages for
  refs        [P] int32, in how many rows a page is listed; 0: it is free
  copies      [3, N] int32: from page, to page, tokens; from -1: nothing
  pool        [P, 2, Hkv, 64, 64] bf16 or e4m3, scales [P, 2, Hkv, 64] e8m0
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 64
D = 64


# --------------------------------------------------------------- the cases --

def _probs(name, requests, rows, vocab, dtype, lengths="same", greedy=False, pad=0, gap=0):
    """rows: of the longest request; greedy: some requests have temperature 0;
    gap: elements between the vocabulary's end and the next row."""
    return {"name": name, "op": "probs", "requests": requests, "rows": rows, "vocab": vocab, "dtype": dtype,
            "lengths": lengths, "greedy": greedy, "pad": pad, "gap": gap}


def _verify(name, requests, rows, vocab, drafts, lengths="same", wide=False, pad=0, gap=0):
    """drafts: the drafter's probabilities are known (without them its tokens
    count as certain); wide: token ids in 64 bits."""
    return {"name": name, "op": "verify", "requests": requests, "rows": rows, "vocab": vocab, "drafts": drafts,
            "lengths": lengths, "wide": wide, "pad": pad, "gap": gap}


def _book(name, op, requests, stride, pages, ctx_lo, ctx_hi, kind):
    """ctx_lo .. ctx_hi: tokens of a request."""
    return {"name": name, "op": op, "requests": requests, "stride": stride, "pages": pages, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "kind": kind}


def _copy(name, cache, hkv, pages, copies, kind):
    return {"name": name, "op": "copy", "cache": cache, "hkv": hkv, "pages": pages, "copies": copies, "kind": kind}


def listed():
    return [
        # The target's logits over one block of 6: nothing but latency.
        _probs("probs 1x6", 1, 6, 32768, "bf16"),
        # A verification step of a large batch: blocks of up to 8, an odd
        # vocabulary, some requests greedy, rows of padding behind.
        _probs("probs 64x8 odd", 64, 8, 128003, "bf16", "ragged", greedy=True, pad=5),
        # One block of 6 is verified.
        _verify("verify 1x6", 1, 6, 32768, True),
        # The same large batch is verified.
        _verify("verify 64x8 odd", 64, 8, 128003, True, "ragged", pad=5),
        # Eight conversations make room for their next block of 8 drafts.
        _book("resize 8 blocks", "resize", 8, 40, 512, 0, 2041, "block"),
        # A scheduler's step over a thousand: finished requests leave, new
        # prompts enter, some share pages, the others grow or give up drafts.
        _book("resize 1024 mixed", "resize", 1024, 2049, 262144, 1, 131072, "mixed"),
        # Three more samples of one prompt.
        _book("fork 1 to 3", "fork", 8, 40, 512, 2041, 2041, "one"),
        # Long prompts, each sampled four times.
        _book("fork 64 long", "fork", 256, 2049, 262144, 16384, 131072, "each"),
        # A small pool pulled together.
        _book("compact 512", "compact", 8, 40, 512, 0, 2041, "all"),
        # A large pool pulled together.
        _book("compact 262144", "compact", 1024, 2049, 262144, 1, 131072, "all"),
        # Requests that share their last page get pages of their own.
        _copy("copy 8 begun pages", "bf16", 1, 512, 8, "begun"),
        # The data of a large quantised cache moves when it is pulled together.
        _copy("copy 8191 pages e4m3", "e4m3", 4, 24576, 8191, "whole"),
    ]


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of its range."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["probs", "probs", "verify", "verify", "resize", "fork", "compact", "copy"])
    if op in ("probs", "verify"):
        while True:
            requests, rows, vocab = _between(rng, 1, 256), rng.randrange(1, 9), _between(rng, 100, 262144)
            if requests * rows * vocab <= 64 * 8 * 128003:
                break
        how = dict(lengths=rng.choice(["same", "ragged"]), pad=rng.choice([0, 0, 1, 7]), gap=rng.choice([0, 0, 1, 64]))
        if op == "probs":
            c = _probs("", requests, rows, vocab, rng.choice(["bf16", "bf16", "fp16", "fp32"]), greedy=rng.random() < 0.3, **how)
            if c["dtype"] == "fp32" and requests * rows * vocab > 64 * 6 * 128003:
                c["dtype"] = "bf16"
        else:
            c = _verify("", requests, rows, vocab, rng.random() < 0.7, wide=rng.random() < 0.3, **how)
    elif op == "copy":
        hkv, cache = rng.choice([1, 2, 4, 8]), rng.choice(["bf16", "e4m3"])
        most = 8191 * 4 // (hkv * (2 if cache == "bf16" else 1))
        copies = _between(rng, 1, most)
        c = _copy("", cache, hkv, 2 * copies + rng.randrange(1, 1000), copies, rng.choice(["begun", "whole"]))
    else:
        requests, hi = _between(rng, 2, 1024), _between(rng, 1, 131072)
        stride = -(-hi // PAGE) + rng.randrange(1, 4)
        pages = max(32, min(262144, int(requests * stride * rng.uniform(0.3, 1.2))))
        kinds = {"resize": ["block", "mixed", "mixed"], "fork": ["one", "each"], "compact": ["all", "some"]}
        c = _book("", op, requests, stride, pages, rng.randrange(hi + 1) if rng.random() < 0.5 else 0, hi, rng.choice(kinds[op]))
    del c["name"]
    return c


def _rows(case):
    """(rows of each request, first rows): fixed by the case."""
    g = random.Random("%(requests)d %(rows)d %(vocab)d" % case)
    new = []
    for r in range(case["requests"]):
        n = case["rows"]
        if case["lengths"] == "ragged" and r:
            n = 0 if g.random() < 0.05 else g.randint(1, n)
        new.append(n)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return new, cu


def _plan(case):
    """What the requests hold and are to hold: fixed by the case.  `lens` fit
    the pool with a tenth to spare; `same[r]` is the request whose pages r
    shares, or -1."""
    c = case
    g = random.Random("%(op)s %(requests)d %(stride)d %(pages)d %(ctx_lo)d %(ctx_hi)d %(kind)s" % c)
    R, most = c["requests"], c["stride"] * PAGE
    lens, same, room = [], [], c["pages"] - c["pages"] // 10
    parents = 1 if c["kind"] == "one" else -(-R // 4)
    for r in range(R):
        n = min(g.randint(c["ctx_lo"], c["ctx_hi"]), most)
        s = -1
        if c["op"] == "fork":
            n = n if r < parents else 0
        elif c["kind"] in ("mixed", "all", "some"):
            if g.random() < 0.1:
                n = 0
            elif r and g.random() < 0.15 and lens[-1]:
                n, s = lens[-1], (same[-1] if same[-1] >= 0 else r - 1)
        need = 0 if s >= 0 else -(-n // PAGE)
        if need > room:
            n, s, need = 0, -1, 0
        room -= need
        lens.append(n)
        same.append(s)
    new = list(lens)
    if c["op"] == "resize":
        for r in range(R):
            if c["kind"] == "block":
                new[r] = lens[r] + 8
            else:
                x = g.random()
                if not lens[r]:
                    new[r] = g.randint(1, 2041) if x < 0.7 else 0
                elif x < 0.08:
                    new[r] = 0
                elif x < 0.35:
                    new[r] = max(0, lens[r] - g.randint(1, 8))
                elif x < 0.95:
                    new[r] = lens[r] + g.randint(1, 8)
                else:
                    new[r] = -1  # left as it is
            new[r] = min(new[r], most)
    forks = []
    if c["op"] == "fork":
        if c["kind"] == "one":
            forks = [(0, r) for r in range(1, min(R, 4))]
        else:
            forks = [(r % parents, r) for r in range(parents, R)]
    return lens, same, new, forks


def _held(case):
    return sum(-(-n // PAGE) for n in _plan(case)[0])


def _capacity(case):
    return max(1, case["pages"] // (2 if case["kind"] == "all" else 16))


# ---------------------------------------------------------------- the work --

def work(case):
    c, op = case, case["op"]
    if op == "probs":
        n = _rows(c)[1][-1] * c["vocab"]
        return {"bytes": n * ((4 if c["dtype"] == "fp32" else 2) + 4), "flops": 5 * n}
    if op == "verify":
        new, cu = _rows(c)
        # A row of p for each request, and one of q where a draft is rejected.
        n = sum((2 if c["drafts"] and k > 1 else 1) * c["vocab"] for k in new if k)
        return {"bytes": 4 * n + 24 * cu[-1], "flops": 4 * n}
    if op == "copy":
        tile = 2 * c["hkv"] * (PAGE * D * 2 if c["cache"] == "bf16" else PAGE * (D + 1))
        tile = tile // 2 if c["kind"] == "begun" else tile
        return {"bytes": 2 * c["copies"] * tile + 12 * c["copies"], "flops": 0}
    lens, same, new, forks = _plan(c)
    if op == "resize":
        moved = sum(abs(-(-n // PAGE) - -(-m // PAGE)) for m, n in zip(lens, new) if n >= 0)
        return {"bytes": 4 * c["pages"] + 12 * moved + 24 * c["requests"], "flops": c["pages"]}
    if op == "fork":
        n = sum(-(-lens[p] // PAGE) for p, _ in forks)
        return {"bytes": 16 * n, "flops": n}
    live = sum(-(-n // PAGE) for n, s in zip(lens, same) if s < 0)
    moves = min(_capacity(c), int(live * (1 - live / c["pages"])))
    return {"bytes": 4 * c["pages"] + 4 * _held(c) + 24 * moves, "flops": 2 * c["pages"]}


# -------------------------------------------------------------- the inputs --

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _prepare_rows(case, g, s):
    new, cu = _rows(case)
    R, V, T = case["requests"], case["vocab"], cu[-1] + case["pad"]
    s["cu_seqlens"] = _ints(cu)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    wide = V + case["gap"]
    # A few words stand out of the rest in each row, as in a language model.
    x = normal(T, wide) * 2
    x += 9 * (uniform(T, wide) < 8 / V) * uniform(T, 1)
    if case["op"] == "probs":
        x[uniform(T, 1).expand(T, wide) < 0.1 * (normal(wide) > 0.5)] = -math.inf  # words that a grammar forbids here
        x = x.to({"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[case["dtype"]])
        s["logits"] = x[:, :V]
        t = 0.2 + 1.3 * uniform(R)
        if case["greedy"]:
            t[uniform(R) < 0.3] = 0
        s["temperatures"] = t
        s["probs"] = torch.zeros(T, V, device="cuda")
        return
    q = torch.softmax(x[:, :V] + 0.5 * normal(T, V), -1)
    p = torch.empty(T, wide, device="cuda")
    p[:, :V] = torch.softmax(x[:, :V], -1)
    s["target"] = p[:, :V]
    kind = torch.int64 if case["wide"] else torch.int32
    # Row t's token is a draft from the row before it.
    at = (q.cumsum(-1, dtype=torch.float64) < uniform(T, 1).double()).sum(-1).clamp(max=V - 1)
    s["tokens"] = torch.cat([at[:1], at[:-1]]).to(kind)
    s["draft"] = q if case["drafts"] else None
    s["uniforms"] = uniform(T)
    s["out"] = torch.full((T,), -7, dtype=kind, device="cuda")
    s["num_out"] = torch.zeros(R, dtype=torch.int32, device="cuda")


def _parts(case, flat):
    """page_table, lens and refs in one buffer."""
    R, S, P = case["requests"], case["stride"], case["pages"]
    a = -(-R * S // 64) * 64
    b = a + -(-R // 64) * 64
    return flat[:R * S].view(R, S), flat[a:a + R], flat[b:b + P]


def _prepare_book(case, seed, s):
    rng = np.random.default_rng(seed)
    lens, same, new, forks = _plan(case)
    R, S, P = case["requests"], case["stride"], case["pages"]
    ids = rng.permutation(P).astype(np.int32)
    table, refs, at = np.full((R, S), -1, np.int32), np.zeros(P, np.int32), 0
    for r in range(R):
        n = -(-lens[r] // PAGE)
        if same[r] >= 0:
            table[r, :n] = table[same[r], :n]
        else:
            table[r, :n] = ids[at:at + n]
            at += n
        refs[table[r, :n]] += 1
    size = -(-R * S // 64) * 64 + -(-R // 64) * 64 + P
    flat = torch.zeros(size, dtype=torch.int32, device="cuda")
    for part, v in zip(_parts(case, flat), (table, np.array(lens, np.int32), refs)):
        part.copy_(torch.from_numpy(v))
    s["start"], s["now"] = flat, flat.clone()
    if case["op"] == "resize":
        s["new_lens"], s["copies"] = _ints(new), _ints([[-1] * R] * 3)
    elif case["op"] == "fork":
        s["parents"], s["children"] = (_ints(list(v)) for v in zip(*forks)) if forks else (_ints([]), _ints([]))
    else:
        s["copies"], s["num_copies"] = _ints([[-1]] * 3).repeat(1, _capacity(case)), _ints([0])


def _codes(x):
    """Rows of 64 as e4m3 codes and the exponents + 127 of their scales."""
    top = x.abs().amax(-1).clamp(min=1e-6)
    e = torch.ceil(torch.log2(top / 448.0))
    return (x * torch.exp2(-e)[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _prepare_copy(case, g, s):
    P, hkv, n = case["pages"], case["hkv"], case["copies"]
    pool = torch.randn((P, 2, hkv, PAGE, D), generator=g, device="cuda", dtype=torch.bfloat16)
    s["scales"] = None
    if case["cache"] == "e4m3":
        codes = torch.empty(pool.shape, dtype=torch.float8_e4m3fn, device="cuda")
        scales = torch.empty(pool.shape[:-1], dtype=torch.uint8, device="cuda")
        for a in range(0, P, 4096):
            codes[a:a + 4096], scales[a:a + 4096] = _codes(pool[a:a + 4096].float())
        pool, s["scales"] = codes, scales.view(torch.float8_e8m0fnu)
    s["pool"] = pool
    order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    tokens = torch.full((n,), PAGE, dtype=torch.int32, device="cuda")
    if case["kind"] == "begun":
        tokens = torch.randint(1, PAGE, (n,), generator=g, device="cuda", dtype=torch.int32)
    s["copies"] = torch.stack([order[:n], order[n:2 * n], tokens])
    if case["kind"] == "begun" and n > 2:
        s["copies"][0, n // 2] = -1  # this request shares nothing


def prepare(case, seed):
    s = {"case": dict(case)}
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] in ("probs", "verify"):
        _prepare_rows(case, g, s)
    elif case["op"] == "copy":
        _prepare_copy(case, g, s)
    else:
        _prepare_book(case, seed, s)
        if own and case["op"] == "compact":
            import speculative_decoding_drafter_k3_gb300 as k3da
            s["workspace"] = k3da.alloc_compact_workspace(case["pages"])
    return s


# ---------------------------------------------------------- the plain form --

def _plain_probs(s):
    n = _rows(s["case"])[1][-1]
    x = s["logits"][:n].float()
    r = torch.searchsorted(s["cu_seqlens"][1:].long(), torch.arange(n, device="cuda"), right=True)
    t = s["temperatures"][r][:, None]
    m = x.amax(-1, keepdim=True)
    e = torch.where(x == m, 0.0, (x - m) / t.clamp(min=1e-30)).exp_()
    e = torch.where(m == -math.inf, 0.0, e)  # a row that allows nothing
    e = e / e.sum(-1, keepdim=True).clamp(min=1e-30)
    V = x.shape[1]
    word = torch.arange(V, device="cuda")
    first = torch.where(x == m, word, V).amin(-1, keepdim=True)
    s["probs"][:n] = torch.where(t > 0, e, ((word == first) & (m > -math.inf)).float())


def _weights(x):
    """Probabilities as whole multiples of 2^-40."""
    return (x.nan_to_num(0.0).clamp(0, 1).double() * 2.0 ** 40).floor().long()


def _plain_verify(s):
    c, N = s["case"], s["case"]["rows"]
    n_rows, V = _rows(c)[1][-1], c["vocab"]
    first = s["cu_seqlens"][:-1].long()
    n = s["cu_seqlens"][1:].long() - first
    i = torch.arange(N, device="cuda")
    row = (first[:, None] + i).clamp(max=s["tokens"].numel() - 1)                # [R, N]
    draft = s["tokens"][(row + 1).clamp(max=s["tokens"].numel() - 1)].long().clamp(0, V - 1)
    p = s["target"][row, draft].double()
    q = s["draft"][row, draft].double() if s["draft"] is not None else 1.0
    yes = (s["uniforms"][row].double() * q < p) & (i < n[:, None] - 1)
    kept = yes.long().cumprod(-1).sum(-1)                                        # [R] accepted drafts
    last = (first + kept).clamp(max=s["tokens"].numel() - 1)                     # the row the next token comes from
    p = s["target"][last]
    rest = p - s["draft"][last] if s["draft"] is not None else \
        torch.where(torch.arange(V, device="cuda") == draft.gather(1, kept[:, None].clamp(max=N - 1)), 0.0, p)
    whole = _weights(p)
    left = torch.where((kept < n - 1)[:, None], _weights(rest), whole)
    left = torch.where(left.sum(-1, keepdim=True) > 0, left, whole)
    run = left.cumsum(-1)
    total = run[:, -1]
    u = (s["uniforms"][(first + n - 1).clamp(min=0)].double() * 2.0 ** 24).floor().long()
    at = (total >> 24) * u + ((total & (1 << 24) - 1) * u >> 24)
    token = (run <= at[:, None]).sum(-1)
    token = torch.where(total > 0, token, -1)
    out = torch.where(i < kept[:, None], draft, torch.where(i == kept[:, None], token[:, None], -1))
    s["out"][:n_rows] = out[i < n[:, None]].to(s["out"].dtype)
    s["num_out"].copy_(torch.where(n > 0, kept + 1, 0))


def _plain_resize(s):
    c = s["case"]
    table, lens, refs = _parts(c, s["start"].clone())
    S, P = c["stride"], c["pages"]
    new = torch.where((s["new_lens"] < 0) | (s["new_lens"] > S * PAGE), lens, s["new_lens"]).long()
    old = lens.long()
    held, want = (old + PAGE - 1) // PAGE, (new + PAGE - 1) // PAGE
    j = torch.arange(S, device="cuda")
    ids = table.long().clamp(min=0)
    gone = (j >= want[:, None]) & (j < held[:, None])
    refs.scatter_add_(0, ids.flatten(), -gone.int().flatten())
    table.masked_fill_(gone, -1)
    grows = new > old
    last = ids.gather(1, (old // PAGE).clamp(max=S - 1)[:, None])[:, 0]
    shared = grows & (old % PAGE > 0) & (refs[last] > 1)
    alike = (last[:, None] == last) & shared & shared[:, None]
    keeps = (alike.sum(-1) == refs[last]) & ((alike.long().cumsum(-1) * alike).amax(-1) == alike.sum(-1)) & \
        (torch.where(alike, torch.arange(len(old), device="cuda"), len(old)).amin(-1) == torch.arange(len(old), device="cuda"))
    moves = shared & ~keeps
    need = torch.where(grows, want - held, 0) + moves
    until = need.cumsum(0)
    free = refs == 0
    rank = free.long().cumsum(0)
    enough = until[-1] <= rank[-1]
    kth = torch.zeros(P + 1, dtype=torch.long, device="cuda")
    kth.scatter_(0, torch.where(free, rank - 1, P), torch.arange(P, device="cuda"))
    moves = moves & enough
    start = until - need
    own_page = kth[start.clamp(max=P)]
    fresh = (j >= held[:, None]) & (j < want[:, None]) & enough
    taken = kth[(start[:, None] + moves[:, None] + (j - held[:, None])).clamp(0, P)]
    table.copy_(torch.where(fresh, taken.int(), table))
    at = (old // PAGE).clamp(max=S - 1)[:, None]
    table.scatter_(1, at, torch.where(moves, own_page, table.gather(1, at)[:, 0].long()).int()[:, None])
    refs += (free & (rank - 1 < until[-1]) & enough).int()
    refs.scatter_add_(0, last, -moves.int())
    lens.copy_(torch.where(grows & ~enough, old, new))
    copies = torch.where(moves, torch.stack([last, own_page, old % PAGE]), -1).int()
    return {"page_table": table, "lens": lens, "refs": refs, "copies": copies}


def _plain_fork(s):
    c = s["case"]
    table, lens, refs = _parts(c, s["start"].clone())
    p, k = s["parents"].long(), s["children"].long()
    table[k] = table[p]
    lens[k] = lens[p]
    held = torch.arange(c["stride"], device="cuda") < ((lens[p] + PAGE - 1) // PAGE)[:, None]
    refs.scatter_add_(0, table[p].long().clamp(min=0).flatten(), held.int().flatten())
    return {"page_table": table, "lens": lens, "refs": refs}


def _plain_compact(s):
    c = s["case"]
    P, room = c["pages"], s["copies"].shape[1]
    table, lens, refs = _parts(c, s["start"].clone())
    live = refs > 0
    total = live.long().sum()
    page = torch.arange(P, device="cuda")
    high, low = live & (page >= total), ~live & (page < total)
    moves = high.long().sum().clamp(max=room)
    from_top = high.flip(0).long().cumsum(0).flip(0) - 1   # the k-th highest
    from_below = low.long().cumsum(0) - 1
    source = torch.full((P + 1,), -1, dtype=torch.long, device="cuda")
    target = source.clone()
    source.scatter_(0, torch.where(high, from_top, P), page)
    target.scatter_(0, torch.where(low, from_below, P), page)
    to = torch.where(high & (from_top < moves), target[from_top.clamp(min=0)], page)
    k = torch.arange(room, device="cuda")
    ours = k < moves
    s["copies"].copy_(torch.where(ours, torch.stack([source[k], target[k], torch.full_like(k, PAGE)]), s["copies"]).int())
    moved = torch.zeros_like(refs).scatter_add_(0, to, refs)
    held = torch.arange(c["stride"], device="cuda") < ((lens + PAGE - 1) // PAGE)[:, None]
    table = torch.where(held, to[table.long().clamp(min=0)].int(), table)
    s["num_copies"].copy_(moves)
    return {"page_table": table, "refs": moved, "copies": s["copies"], "num_copies": s["num_copies"]}


def _plain_copy(s):
    src, dst, tokens = s["copies"].long()
    ours = (torch.arange(PAGE, device="cuda") < tokens[:, None]) & (src >= 0)[:, None]
    src, dst = src.clamp(min=0), dst.clamp(min=0)

    def move(x):
        m = ours.view(len(src), 1, 1, PAGE, *[1] * (x.dim() - 4))
        x[dst] = torch.where(m, x[src], x[dst])

    if s["scales"] is None:
        move(s["pool"].view(torch.int16))
    else:
        move(s["pool"].view(torch.uint8))
        move(s["scales"].view(torch.uint8))


# ------------------------------------------------------ the package's calls --

def _own_run(s):
    import speculative_decoding_drafter_k3_gb300 as k3da
    op = s["case"]["op"]
    if op == "probs":
        k3da.k3da_token_probs(s["probs"], s["logits"], s["cu_seqlens"], temperatures=s["temperatures"])
        return {"probs": s["probs"]}
    if op == "verify":
        k3da.k3da_verify(s["out"], s["num_out"], s["tokens"], s["target"], s["uniforms"], s["cu_seqlens"], draft_probs=s["draft"])
        return {"out": s["out"], "num_out": s["num_out"]}
    if op == "copy":
        k3da.k3da_kv_copy(s["pool"], s["copies"], kv_scales=s["scales"])
        return {"pool": s["pool"]} if s["scales"] is None else {"pool": s["pool"], "scales": s["scales"]}
    s["now"].copy_(s["start"])  # the calls change the pages in place: each pass starts from the same
    table, lens, refs = _parts(s["case"], s["now"])
    if op == "resize":
        k3da.k3da_pages_resize(table, lens, refs, s["new_lens"], s["copies"])
        return {"page_table": table, "lens": lens, "refs": refs, "copies": s["copies"]}
    if op == "fork":
        k3da.k3da_pages_fork(table, lens, refs, s["parents"], s["children"])
        return {"page_table": table, "lens": lens, "refs": refs}
    k3da.k3da_pages_compact(table, lens, refs, s["copies"], s["num_copies"], workspace=s["workspace"])
    return {"page_table": table, "refs": refs, "copies": s["copies"], "num_copies": s["num_copies"]}


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op == "probs":
        _plain_probs(state)
        return {"probs": state["probs"]}
    if op == "verify":
        _plain_verify(state)
        return {"out": state["out"], "num_out": state["num_out"]}
    if op == "copy":
        _plain_copy(state)
        return {"pool": state["pool"]} if state["scales"] is None else {"pool": state["pool"], "scales": state["scales"]}
    return {"resize": _plain_resize, "fork": _plain_fork, "compact": _plain_compact}[op](state)


# ------------------------------------------------------------ the definitions --

def _exact_probs(s):
    out = s["probs"].double()
    new, cu = _rows(s["case"])
    for r, n in enumerate(new):
        t = float(s["temperatures"][r])
        for row in range(cu[r], cu[r] + n):
            x = s["logits"][row].double()
            if t > 0:
                total = torch.logsumexp(x / t, 0)
                out[row] = torch.exp(x / t - total) if total > -math.inf else 0.0
            else:
                out[row] = 0.0
                best = x.max()
                if best > -math.inf:
                    out[row, torch.nonzero(x == best)[0, 0]] = 1.0
    return {"probs": out}


def _exact_verify(s):
    new, cu = _rows(s["case"])
    out, num = s["out"].cpu().numpy().copy(), s["num_out"].cpu().numpy().copy()
    tokens, u = s["tokens"].cpu().numpy(), s["uniforms"].cpu().numpy().astype(np.float64)
    for r, n in enumerate(new):
        if not n:
            num[r] = 0
            continue
        a, i = cu[r], 0
        out[a:a + n] = -1
        while i < n - 1:
            d = int(tokens[a + i + 1])
            q = float(s["draft"][a + i, d]) if s["draft"] is not None else 1.0
            if not u[a + i] * q < float(s["target"][a + i, d]):
                break
            out[a + i] = d
            i += 1
        p = s["target"][a + i].cpu().numpy()
        w = p
        if i < n - 1:
            w = p.copy()
            if s["draft"] is not None:
                w -= s["draft"][a + i].cpu().numpy()
            else:
                w[int(tokens[a + i + 1])] = 0
        for x in (w, p):
            run = np.cumsum(np.floor(np.ldexp(np.clip(x, 0, 1).astype(np.float64), 40)).astype(np.int64))
            if run[-1]:
                break
        at = int(run[-1]) * int(u[a + n - 1] * 2 ** 24) >> 24
        out[a + i] = np.searchsorted(run, at, side="right") if run[-1] else -1
        num[r] = i + 1
    return {"out": out, "num_out": num}


def _exact_resize(case, table, lens, refs, new_lens):
    R, limit = len(lens), case["stride"] * PAGE
    copies = np.full((3, R), -1, np.int32)
    new = [int(lens[r]) if not 0 <= n <= limit else n for r, n in enumerate(new_lens)]
    for r in range(R):
        for j in range(-(-new[r] // PAGE), -(-int(lens[r]) // PAGE)):
            refs[table[r, j]] -= 1
            table[r, j] = -1
    growing = [r for r in range(R) if new[r] > lens[r]]
    begun = {}  # last pages that are written into next, and by whom
    for r in growing:
        if lens[r] % PAGE:
            begun.setdefault(int(table[r, lens[r] // PAGE]), []).append(r)
    copying = set()
    for page, who in begun.items():
        if refs[page] > 1:
            copying.update(who[1:] if refs[page] == len(who) else who)
    free = np.flatnonzero(refs == 0)
    need = sum(-(-new[r] // PAGE) - -(-int(lens[r]) // PAGE) for r in growing) + len(copying)
    if need > len(free):
        for r in range(R):
            lens[r] = min(lens[r], new[r])
        return copies
    give = iter(free)
    for r in growing:
        if r in copying:
            page, j = next(give), lens[r] // PAGE
            copies[:, r] = table[r, j], page, lens[r] % PAGE
            refs[table[r, j]] -= 1
            refs[page] = 1
            table[r, j] = page
        for j in range(-(-int(lens[r]) // PAGE), -(-new[r] // PAGE)):
            table[r, j] = next(give)
            refs[table[r, j]] = 1
    lens[:] = new
    return copies


def _exact_compact(case, table, lens, refs, copies):
    live = np.flatnonzero(refs)
    high = live[live >= len(live)][::-1][:copies.shape[1]]
    low = np.flatnonzero(refs == 0)[:len(high)]
    to = np.arange(len(refs), dtype=np.int32)
    for k, (x, y) in enumerate(zip(high, low)):
        copies[:, k] = x, y, PAGE
        to[x], refs[y], refs[x] = y, refs[x], 0
    for r, n in enumerate(lens):
        held = -(-int(n) // PAGE)
        table[r, :held] = to[table[r, :held]]
    return len(high)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "probs":
        return _exact_probs(s)
    if op == "verify":
        return _exact_verify(s)
    if op == "copy":
        pool, scales = s["pool"].double(), None if s["scales"] is None else s["scales"].clone()
        for x, y, n in s["copies"].T.tolist():
            if x >= 0:
                pool[y, :, :, :n] = pool[x, :, :, :n]
                if scales is not None:
                    scales.view(torch.uint8)[y, :, :, :n] = scales.view(torch.uint8)[x, :, :, :n]
        return {"pool": pool} if scales is None else {"pool": pool, "scales": torch.exp2(scales.view(torch.uint8).double() - 127)}
    table, lens, refs = (x.cpu().numpy().copy() for x in _parts(case, s["start"]))
    if op == "resize":
        copies = _exact_resize(case, table, lens, refs, s["new_lens"].tolist())
        return {"page_table": table, "lens": lens, "refs": refs, "copies": copies}
    if op == "fork":
        for p, k in zip(s["parents"].tolist(), s["children"].tolist()):
            n = -(-int(lens[p]) // PAGE)
            table[k, :n], lens[k] = table[p, :n], lens[p]
            refs[table[p, :n]] += 1
        return {"page_table": table, "lens": lens, "refs": refs}
    copies = s["copies"].cpu().numpy().copy()
    moves = _exact_compact(case, table, lens, refs, copies)
    return {"page_table": table, "refs": refs, "copies": copies, "num_copies": np.array([moves], np.int32)}
