"""What stands around the paged cache, as it is measured: rotary positions for the rows that go
into it, its pages' sharing, freeing and moving, and the attention of requests that share a prefix.

Head layouts, context lengths and block widths are those of the package's own workloads (32 query /
8 KV heads of 128, 24 / 2 of 256, 16 / 16 of 128, 4 / 2 of 64; contexts of 512..8192 and 4096..32768
tokens, blocks of up to 16, prompts of 4096).

Pages.  block_table [n, max_pages] holds the page ids of each request, used [n] how many of them, and
refs [pages] how many table entries hold a page (0: free).
  resize: request i ends with ceil(length[i] / page) pages.  Pages taken away lose one reference;
          then the free pages with the lowest ids go to the growing requests in order, while all that
          was asked so far fits.
  fork:   request dst[f], which holds nothing, takes the first length[f] tokens of src[f]: whole pages are
          shared, the part of a page at the end is copied to a page of its own (the lowest free ones in
          the forks' order).
  compact: with L pages in use, the k-th of those with ids >= L moves to the k-th free id < L.

8-bit rows: a (token, head) row of d elements is held as e4m3 codes and one exponent byte b; an
element is code * 2^(b - 127), and 2^(b - 127) is the smallest power of two that takes the row's
largest magnitude to 448 or less (b >= 15).
"""
import math
import random

import torch

own = False

HEADS = {"tiny": (4, 2, 64), "even": (16, 16, 128), "main": (32, 8, 128), "wide": (24, 2, 256)}
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


def listed():
    return [
        # one new token of each of 8 requests: q rotated, k rotated and stored with v in 8 bits
        dict(name="rotate token e4m3", op="rotate", heads="main", kv="e4m3", new="bf16", page=16, rot=128, pairs="half",
             base=10000.0, way="none", factor=1.0, n=8, rows=1, full=True, long_n=0, long_rows=0, ctx_lo=512,
             ctx_hi=8192, pad=0, mix=1),
        # 64 requests' candidate blocks before a verification, which takes keys as rows: half of each head
        # rotated in interleaved pairs, frequencies stretched for long contexts
        dict(name="rotate blocks rows", op="rotate", heads="main", kv="none", new="bf16", page=16, rot=64, pairs="inter",
             base=500000.0, way="yarn", factor=8.0, n=64, rows=16, full=False, long_n=0, long_rows=0, ctx_lo=4096,
             ctx_hi=32768, pad=11, mix=2),
        # prompts of up to 8192 tokens next to requests that add a block, into a bf16 cache
        dict(name="rotate prompts bf16", op="rotate", heads="main", kv="bf16", new="bf16", page=16, rot=128, pairs="half",
             base=10000.0, way="linear", factor=4.0, n=12, rows=16, full=False, long_n=4, long_rows=8192, ctx_lo=0,
             ctx_hi=700, pad=0, mix=3),
        # one decode step of 64 requests: most need a page or none, some give back what was not accepted
        dict(name="resize step", op="resize", page=16, n=64, pages=16384, ctx_lo=512, ctx_hi=2048, move=16, gone=0.0,
             shared=0.25, mix=4),
        # requests leave and others come with long prompts
        dict(name="resize churn", op="resize", page=16, n=256, pages=262144, ctx_lo=512, ctx_hi=16384, move=4096, gone=0.4,
             shared=0.5, mix=5),
        # 8 samples from one prompt of 700 tokens
        dict(name="fork samples", op="fork", heads="main", kv="bf16", page=16, layers=1, n=16, parents=1, forks=8, ctx_lo=700,
             ctx_hi=700, spare=64, mix=6),
        # 56 children of 8 long requests in the cache of four layers, 8-bit rows
        dict(name="fork long e4m3", op="fork", heads="main", kv="e4m3", page=64, layers=4, n=64, parents=8, forks=56,
             ctx_lo=4096, ctx_hi=32768, spare=256, mix=7),
        # a small pool after a few requests have left
        dict(name="compact small", op="compact", heads="main", kv="bf16", page=16, layers=1, n=16, pages=1024, ctx_lo=64,
             ctx_hi=700, mix=8),
        # a large one: one page in six moves
        dict(name="compact large", op="compact", heads="main", kv="bf16", page=16, layers=2, n=64, pages=16384, ctx_lo=512,
             ctx_hi=4096, mix=9),
        # 8 samples of one prompt, one token each: the latency of such a decode call
        dict(name="attend samples bf16", op="attend", heads="main", kv="bf16", page=16, n=8, groups=1, alone=0, rows=1,
             full=True, pre_lo=4096, pre_hi=4096, ctx_lo=16, ctx_hi=256, pad=0, mix=10),
        # four long prompts with 16 samples each, 8-bit cache
        dict(name="attend samples e4m3", op="attend", heads="main", kv="e4m3", page=16, n=64, groups=4, alone=0, rows=1,
             full=True, pre_lo=8192, pre_hi=32768, ctx_lo=16, ctx_hi=1024, pad=0, mix=11),
        # candidate blocks of 60 requests behind two common beginnings, four others alone
        dict(name="attend blocks bf16", op="attend", heads="main", kv="bf16", page=16, n=64, groups=2, alone=4, rows=16,
             full=False, pre_lo=4096, pre_hi=16384, ctx_lo=64, ctx_hi=2048, pad=9, mix=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rotate", "resize", "fork", "compact", "attend", "attend"])
    heads, mix = rng.choice(list(HEADS)), rng.randrange(1 << 20)
    page = rng.choice([16, 16, 32, 64, 128])
    d = HEADS[heads][2]
    if op == "rotate":
        long_n = rng.choice([0, 0, 1, 2])
        kv = rng.choice(["none", "bf16", "e4m3"])
        hi = _log(rng, 1, 32768)
        return dict(op=op, heads=heads, kv=kv, new="bf16" if kv == "bf16" else rng.choice(["bf16", "f32"]), page=page,
                    rot=rng.choice([d, d, d // 2, d // 4 + 2, 2 * rng.randint(1, d // 2)]), pairs=rng.choice(["half", "inter"]),
                    base=rng.choice([10000.0, 500000.0, 1000000.0]), way=rng.choice(["none", "linear", "ntk", "yarn"]),
                    factor=rng.choice([1.5, 4.0, 8.0, 32.0]), n=max(long_n, _log(rng, 1, 64)), rows=rng.randint(1, 16),
                    full=rng.random() < 0.3, long_n=long_n, long_rows=_log(rng, 17, 6000) if long_n else 0, ctx_lo=hi // 16,
                    ctx_hi=hi, pad=rng.randrange(12), mix=mix)
    if op == "resize":
        hi = _log(rng, 16, 8192)
        n = _log(rng, 1, 200)
        return dict(op=op, page=page, n=n, pages=2 * n * (-(-(hi + 600) // page)) + rng.randint(3, 5000), ctx_lo=hi // 8,
                    ctx_hi=hi, move=_log(rng, 1, 600), gone=rng.choice([0.0, 0.1, 0.5]), shared=rng.choice([0.0, 0.3, 0.7]), mix=mix)
    if op == "fork":
        parents = _log(rng, 1, 8)
        forks = _log(rng, 1, 56)
        hi = _log(rng, 1, 16384)
        return dict(op=op, heads=heads, kv=rng.choice(["bf16", "e4m3"]), page=page, layers=rng.randint(1, 3),
                    n=parents + forks + rng.randrange(4), parents=parents, forks=forks, ctx_lo=max(1, hi // 8), ctx_hi=hi,
                    spare=rng.randint(60, 300), mix=mix)
    if op == "compact":
        hi = _log(rng, 16, 2048)
        n = _log(rng, 2, 48)
        return dict(op=op, heads=heads, kv=rng.choice(["bf16", "e4m3"]), page=page, layers=rng.randint(1, 2), n=n,
                    pages=n * (-(-hi // page)) + rng.randint(0, 500), ctx_lo=max(1, hi // 8), ctx_hi=hi, mix=mix)
    groups = rng.randint(1, 4)
    alone = rng.randrange(4)
    pre, hi = _log(rng, 16, 16384), _log(rng, 1, 2048)
    rows = rng.choice([1, 1, 7, 16])
    return dict(op=op, heads=heads, kv=rng.choice(["bf16", "e4m3"]), page=page, n=groups + alone + _log(rng, 1, 48), groups=groups,
                alone=alone, rows=rows, full=rows == 1 or rng.random() < 0.3, pre_lo=max(1, pre // 4), pre_hi=pre,
                ctx_lo=hi // 8, ctx_hi=hi, pad=rng.randrange(12), mix=mix)


# ------------------------------------------------------------------ sizes, from the case alone
def _sizes(case):
    """(rows, cached tokens before them) of each request of a rotate case."""
    r = random.Random(case["mix"])
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["n"])]
    rows = [case["rows"] if case["full"] else r.randint(1, case["rows"]) for _ in range(case["n"])]
    for i in range(case["long_n"]):
        rows[i] = case["long_rows"] if case["long_n"] == 1 else r.randint(case["long_rows"] // 2, case["long_rows"])
    return rows, ctx


def _groups(case):
    """(first request of each group and the end of the last, tokens that each group shares, rows, cached tokens)."""
    r = random.Random(case["mix"])
    members = case["n"] - case["alone"]
    cuts = sorted(r.sample(range(1, members), case["groups"] - 1)) if case["groups"] > 1 else []
    first = [0] + cuts + [members]
    whole = [max(1, r.randint(case["pre_lo"], case["pre_hi"]) // case["page"]) * case["page"] for _ in range(case["groups"])]
    rows = [case["rows"] if case["full"] else r.randint(1, case["rows"]) for _ in range(case["n"])]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["n"])]
    for g in range(case["groups"]):
        for i in range(first[g], first[g + 1]):
            ctx[i] += whole[g]
    return first, whole, rows, ctx


def _plan(case):
    """A resize case: (tokens held, tokens wanted, requests that share their first pages, and of whom)."""
    r = random.Random(case["mix"])
    n, page = case["n"], case["page"]
    held = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)]
    length = []
    for h in held:
        if r.random() < case["gone"]:
            length.append(0)
        else:
            length.append(max(0, h + r.randint(-case["move"] // 2, case["move"])) if r.random() < 0.9 else h)
    parent = [r.randrange(i) if i and r.random() < case["shared"] else -1 for i in range(n)]
    # what is kept in part of a page is its request's own: a request that shrinks into shared pages ends with a whole one
    common = [0] * n
    for i in range(n):
        if parent[i] >= 0:
            common[i] = min(held[i], held[parent[i]]) // (2 * page)
    deepest = list(common)
    for i in range(n):
        if parent[i] >= 0:
            deepest[parent[i]] = max(deepest[parent[i]], common[i])
    for i in range(n):
        if length[i] < held[i] and length[i] // page < deepest[i]:
            length[i] = length[i] // page * page
    return held, length, parent, common


def _pages(case, tokens):
    return -(-tokens // case["page"])


def _forks(case):
    """A fork case: (tokens of the parents, source, destination and tokens of each fork)."""
    r = random.Random(case["mix"])
    held = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["parents"])]
    src = [r.randrange(case["parents"]) for _ in range(case["forks"])]
    dst = r.sample(range(case["parents"], case["n"]), case["forks"])
    length = [held[s] if r.random() < 0.7 else r.randint(1, held[s]) for s in src]
    return held, src, dst, length


def _live(case):
    """A compact case: tokens of each request (0: it has left)."""
    r = random.Random(case["mix"])
    t = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["n"])]
    left = [r.random() < 0.3 for _ in t]
    return t, [0 if x else y for x, y in zip(left, t)]


def _token_bytes(case):
    hq, hkv, d = HEADS[case["heads"]]
    return 2 * hkv * (d + 1 if case["kv"] == "e4m3" else d * TYPES[case["kv"]].itemsize)


def work(case):
    op = case["op"]
    if op == "rotate":
        hq, hkv, d = HEADS[case["heads"]]
        m, size = sum(_sizes(case)[0]), TYPES[case["new"]].itemsize
        read = (hq + (1 if case["kv"] == "none" else 2) * hkv) * d * size
        written = hq * d * size + (hkv * d * size if case["kv"] == "none" else _token_bytes(case))
        return {"bytes": m * (read + written), "flops": 3 * m * (hq + hkv) * case["rot"]}
    if op == "resize":
        held, length, _, _ = _plan(case)
        moved = sum(abs(_pages(case, a) - _pages(case, b)) for a, b in zip(held, length))
        return {"bytes": 12 * case["n"] + 12 * moved + 4 * moved, "flops": 0}
    if op == "fork":
        held, src, dst, length = _forks(case)
        tail = sum(x % case["page"] for x in length)
        return {"bytes": 2 * case["layers"] * tail * _token_bytes(case) + sum(16 * _pages(case, x) for x in length), "flops": 0}
    if op == "compact":
        used = sum(_pages(case, x) for x in _live(case)[1])
        total = max(case["pages"], 1)
        moved = used * max(0, total - used) // total      # about: which pages are free is the seed's affair
        return {"bytes": 4 * total + 4 * used + 2 * case["layers"] * moved * case["page"] * _token_bytes(case), "flops": 0}
    hq, hkv, d = HEADS[case["heads"]]
    first, whole, rows, ctx = _groups(case)
    keys = sum(whole) + sum(c + k for c, k in zip(ctx, rows))
    for g in range(case["groups"]):
        keys -= (first[g + 1] - first[g]) * whole[g]
    seen = sum(k * c + k * (k + 1) // 2 for k, c in zip(rows, ctx))
    return {"bytes": keys * _token_bytes(case) + sum(rows) * hq * (4 * d + 4), "flops": 4 * d * hq * seen}


# ------------------------------------------------------------------ 8-bit rows
def _pack(x):
    """Rows x [..., d] in fp32 as (e4m3 codes, exponent bytes)."""
    mant, power = torch.frexp(x.abs().amax(-1))        # largest magnitude = mant * 2^power, mant in [0.5, 1)
    e = torch.where(mant > 0.875, power - 8, power - 9)  # 448 = 0.875 * 2^9
    e = torch.where(mant == 0, torch.full_like(e, -112), e).clamp_min(-112)
    inverse = ((127 - e) << 23).to(torch.int32).view(torch.float32)   # 2^-e, made from its bits: exact
    return (x * inverse[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _unpack(codes, exps):
    return codes.float() * (exps.to(torch.int32) << 23).view(torch.float32)[..., None]


# ------------------------------------------------------------------ inputs
def _pools(case, pages, g, live=True):
    """K and V pools [layers, pages, hkv, page, d] (and their exponent bytes); keys have a few channels of
    larger magnitude, tokens differ in size."""
    hq, hkv, d = HEADS[case["heads"]]
    shape = (case.get("layers", 1), pages, hkv, case["page"])
    loud = 1.0 + 5.0 * (torch.arange(d, device="cuda") % 29 == 3)
    out = []
    for key in (True, False):
        x = torch.randn(*shape, d, generator=g, device="cuda", dtype=torch.bfloat16)
        x *= torch.exp(0.3 * torch.randn(*shape, 1, generator=g, device="cuda")).to(torch.bfloat16)
        if key:
            x *= loud.to(torch.bfloat16)
        out.append(_pack(x.float()) if case["kv"] == "e4m3" else (x, None))
        del x
    return out


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _offsets(count):
    return _ints([0] + [sum(count[:i + 1]) for i in range(len(count))])


def _frequencies(case):
    """Radians per position of each pair, in 64 bits."""
    r, base, f = case["rot"], case["base"], case["factor"]
    t = torch.arange(r // 2, dtype=torch.float64)
    if case["way"] == "ntk" and r > 2:
        base = base * f ** (r / (r - 2))
    freq = base ** (-2.0 * t / r)
    if case["way"] == "linear":
        freq = freq / f
    if case["way"] == "yarn":
        # pairs that turn more than 32 times in the original 4096 tokens stay, those that turn less than once
        # are stretched, and a straight line joins them
        edge = [r * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), r - 1)
        ramp = ((t - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        freq = freq * (1.0 - ramp) + freq / f * ramp
    return freq


def _tables(need, pages, width, g):
    """Block tables of requests with `need` pages each, scattered over the pool."""
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(need), max(width, 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k]
        at += k
    return table


def _meta(s, table, used, pages):
    """The three arrays of the pages' state in one buffer, with what they hold before the call beside it."""
    n, width = table.shape
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    ids = table[table >= 0].long()
    refs.index_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))
    s["before"] = torch.cat([refs, table.reshape(-1), used])
    now = s["now"] = s["before"].clone()
    s["refs"], s["table"], s["used"] = now[:pages], now[pages:pages + n * width].view(n, width), now[pages + n * width:]


def prepare(case, seed):
    op = case["op"]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=case)
    if op == "rotate":
        hq, hkv, d = HEADS[case["heads"]]
        rows, ctx = _sizes(case)
        m = s["live"] = sum(rows)
        s["rows"], s["ctx"] = rows, ctx
        s["ctx_len"], s["cu"] = _ints(ctx), _offsets(rows)
        # the fused projection's rows of this step
        qkv = torch.randn(m + case["pad"], hq + 2 * hkv, d, generator=g, device="cuda")
        qkv *= torch.exp(0.3 * torch.randn(m + case["pad"], hq + 2 * hkv, 1, generator=g, device="cuda"))
        qkv = qkv.to(TYPES[case["new"]])
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_out"] = torch.zeros(m + case["pad"], hq, d, dtype=qkv.dtype, device="cuda")
        s["rad"] = _frequencies(case).cuda()
        if case["kv"] == "none":
            s["k_out"] = torch.zeros(m + case["pad"], hkv, d, dtype=qkv.dtype, device="cuda")
        else:
            need = [_pages(case, c + k) for c, k in zip(ctx, rows)]
            pages = sum(need) + 3
            s["table"] = _tables(need, pages, max(need), g)
            s["pools"] = [torch.zeros(pages, hkv, case["page"], d, dtype=TYPES[case["kv"]], device="cuda") for _ in range(2)]
            s["exps"] = [torch.full((pages, hkv, case["page"]), 127, dtype=torch.uint8, device="cuda") for _ in range(2)] \
                if case["kv"] == "e4m3" else [None, None]
            if case["kv"] == "e4m3":
                s["back"] = [torch.zeros(m, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    elif op == "resize":
        held, length, parent, common = _plan(case)
        need = [_pages(case, h) for h in held]
        width = max(need + [_pages(case, x) for x in length])
        table = _tables(need, case["pages"], width, g)
        for i in range(case["n"]):
            if common[i]:
                table[i, :common[i]] = table[parent[i], :common[i]]
        _meta(s, table, _ints(need), case["pages"])
        s["length"] = _ints(length)
    elif op == "fork":
        held, src, dst, length = _forks(case)
        need = [_pages(case, h) for h in held] + [0] * (case["n"] - case["parents"])
        pages = sum(need) + case["spare"]
        _meta(s, _tables(need, pages, max(need), g), _ints(need), pages)
        s["src"], s["dst"], s["length"] = _ints(src), _ints(dst), _ints(length)
    elif op == "compact":
        held, kept = _live(case)
        need = [_pages(case, h) for h in held]
        pages = max(case["pages"], sum(need))
        table = _tables(need, pages, max(need), g)
        for i in range(case["n"]):
            if not kept[i]:
                table[i] = -1
        _meta(s, table, _ints([k if x else 0 for k, x in zip(need, kept)]), pages)
    else:
        hq, hkv, d = HEADS[case["heads"]]
        first, whole, rows, ctx = _groups(case)
        s["rows"], s["ctx"], s["live"] = rows, ctx, sum(rows)
        s["ctx_len"], s["cu"] = _ints(ctx), _offsets(rows)
        s["cu_groups"], s["prefix"] = _ints(first), _ints(whole)
        need = [_pages(case, c + k) for c, k in zip(ctx, rows)]
        common = [0] * case["n"]
        for j in range(case["groups"]):
            for i in range(first[j], first[j + 1]):
                common[i] = whole[j] // case["page"]
        # the groups' pages, then each request's own
        part = [w // case["page"] for w in whole] + [k - c for k, c in zip(need, common)]
        pages = sum(part) + 3
        ids = _tables(part, pages, max(part), g)
        s["table"] = torch.full((case["n"], max(need)), -1, dtype=torch.int32, device="cuda")
        for j in range(case["groups"]):
            s["table"][first[j]:first[j + 1], :part[j]] = ids[j, :part[j]]
        for i in range(case["n"]):
            s["table"][i, common[i]:need[i]] = ids[case["groups"] + i, :need[i] - common[i]]
        (k, ke), (v, ve) = _pools(case, pages, g)
        s["pools"], s["exps"] = [k[0], v[0]], [None if x is None else x[0] for x in (ke, ve)]
        m = s["live"] + case["pad"]
        s["q"] = torch.randn(m, hq, d, generator=g, device="cuda").to(torch.bfloat16)
        s["out"] = torch.zeros(m, hq, d, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros(m, hq, dtype=torch.float32, device="cuda")
    if op in ("fork", "compact"):
        (k, ke), (v, ve) = _pools(case, pages, g)
        s["pools"], s["exps"] = [k, v], [ke, ve]
    if own:
        import speculative_decoding_verification_packed_gb300 as svp
        s["svp"] = svp
        if op == "rotate":
            s["freq"] = svp.rope_frequencies(case["rot"], base=case["base"], scaling=case["way"], factor=case["factor"],
                                             original=4096, device="cuda")
        if op in ("resize", "fork", "compact"):
            s["pages"] = svp.make_pages(s["table"], s["used"], s["refs"], page_size=case["page"])
        if "pools" in s:
            layers = range(case["layers"]) if op in ("fork", "compact") else [None]
            s["caches"] = [svp.make_cache(s["pools"][0] if x is None else s["pools"][0][x], s["pools"][1] if x is None else s["pools"][1][x],
                                          s["table"], **({} if s["exps"][0] is None else
                                                         {"k_exp": s["exps"][0] if x is None else s["exps"][0][x],
                                                          "v_exp": s["exps"][1] if x is None else s["exps"][1][x]})) for x in layers]
    return s


# ------------------------------------------------------------------ plain forms
def _rows_of(s, count):
    """Request, row within it and cache position of packed rows 0..count-1."""
    row = torch.arange(count, device=s["cu"].device, dtype=torch.int32)
    req = torch.searchsorted(s["cu"], row, right=True) - 1
    j = row - s["cu"][req]
    return req, s["ctx_len"][req] + j


def _turned(x, cos, sin, pairs):
    """fp32 rows x [m, heads, d] with their first 2 t elements rotated by cos, sin [m, 1, t]."""
    r = 2 * cos.shape[-1]
    head, rest = x[..., :r], x[..., r:]
    if pairs == "half":
        a, b = head[..., :r // 2], head[..., r // 2:]
        head = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([head, rest], -1)


def _rotate(s):
    m, case = s["live"], s["case"]
    req, pos = _rows_of(s, m)
    angle = (pos.double()[:, None] * s["rad"])[:, None]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    s["q_out"][:m] = _turned(s["q"][:m].float(), cos, sin, case["pairs"]).to(s["q_out"].dtype)
    k = _turned(s["k"][:m].float(), cos, sin, case["pairs"])
    if case["kv"] == "none":
        s["k_out"][:m] = k.to(s["k_out"].dtype)
        return
    pg, tok = s["table"][req, pos // case["page"]].long(), (pos % case["page"]).long()
    if case["kv"] == "bf16":
        s["pools"][0][pg, :, tok] = k.to(torch.bfloat16)
        s["pools"][1][pg, :, tok] = s["v"][:m].to(torch.bfloat16)
        return
    packed = _pack(k), _pack(s["v"][:m].float())
    s["pools"][0].view(torch.uint8)[pg, :, tok] = packed[0][0].view(torch.uint8)
    s["pools"][1].view(torch.uint8)[pg, :, tok] = packed[1][0].view(torch.uint8)
    s["exps"][0][pg, :, tok] = packed[0][1]
    s["exps"][1][pg, :, tok] = packed[1][1]
    s["back"][0].copy_(_unpack(s["pools"][0].view(torch.uint8)[pg, :, tok].view(torch.float8_e4m3fn), s["exps"][0][pg, :, tok]))
    s["back"][1].copy_(_unpack(s["pools"][1].view(torch.uint8)[pg, :, tok].view(torch.float8_e4m3fn), s["exps"][1][pg, :, tok]))


def _resize(s):
    page, table, used, refs = s["case"]["page"], s["table"], s["used"], s["refs"]
    want = (s["length"] + page - 1) // page
    at = torch.arange(table.shape[1], device=table.device)[None]
    drop = (at >= want[:, None]) & (at < used[:, None])
    ids = table[drop].long()
    refs.index_add_(0, ids, torch.full_like(ids, -1, dtype=torch.int32))
    table[drop] = -1
    free = (refs == 0).nonzero()[:, 0].to(torch.int32)
    need = (want - used).clamp_min(0)
    end = need.cumsum(0)
    fits = end <= free.numel()
    grow = (at >= used[:, None]) & (at < want[:, None]) & fits[:, None]
    new = free[((end - need - used)[:, None] + at)[grow]]
    table[grow] = new
    refs[new.long()] = 1
    used.copy_(torch.where(fits | (want < used), want, used))


def _fork(s):
    page, table, used, refs = s["case"]["page"], s["table"], s["used"], s["refs"]
    src, dst, length = s["src"].long(), s["dst"].long(), s["length"]
    whole, part = length // page, length % page
    at = torch.arange(table.shape[1], device=table.device)[None]
    shared = at < whole[:, None]
    rows = torch.where(shared, table[src], torch.full_like(table[src], -1))
    free = (refs == 0).nonzero()[:, 0]
    ids = rows[shared].long()
    refs.index_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))
    tails = (part > 0).nonzero()[:, 0]
    to = free[:tails.numel()]
    origin = table[src[tails], whole[tails].long()].long()
    rows[tails, whole[tails].long()] = to.to(torch.int32)
    refs[to] = 1
    table[dst] = rows
    used[dst] = whole + (part > 0).to(torch.int32)
    keep = torch.arange(page, device=table.device)[None] < part[tails][:, None]      # [tails, tokens]
    for pool, exps in zip(s["pools"], s["exps"]):
        raw = pool.view(torch.uint8) if exps is not None else pool
        raw[:, to] = torch.where(keep[None, :, None, :, None], raw[:, origin], raw[:, to])
        if exps is not None:
            exps[:, to] = torch.where(keep[None, :, None, :], exps[:, origin], exps[:, to])


def _compact(s):
    table, refs = s["table"], s["refs"]
    live = refs > 0
    ids = torch.arange(refs.numel(), device=refs.device)
    count = live.sum()
    movers, holes = (live & (ids >= count)).nonzero()[:, 0], (~live & (ids < count)).nonzero()[:, 0]
    for pool, exps in zip(s["pools"], s["exps"]):
        raw = pool.view(torch.uint8) if exps is not None else pool
        raw[:, holes] = raw[:, movers]
        if exps is not None:
            exps[:, holes] = exps[:, movers]
    where = ids.to(torch.int32)
    where[movers] = holes.to(torch.int32)
    table.copy_(torch.where(table >= 0, where[table.clamp_min(0).long()], table))
    refs[holes] = refs[movers]
    refs[movers] = 0


def _attend_one(s, i):
    """softmax(q k^T / sqrt(d)) v of request i's rows, and the logarithm of the softmax's sum."""
    k, c, page = s["rows"][i], s["ctx"][i], s["case"]["page"]
    first = sum(s["rows"][:i])
    q = s["q"][first:first + k].float()
    hq, d = q.shape[1:]
    hkv = s["pools"][0].shape[1]
    pos = torch.arange(c + k, device=q.device)
    pg, tok = s["table"][i][pos // page].long(), pos % page
    kv = [pool[pg, :, tok].float() if exps is None else
          _unpack(pool.view(torch.uint8)[pg, :, tok].view(torch.float8_e4m3fn), exps[pg, :, tok])
          for pool, exps in zip(s["pools"], s["exps"])]
    grp = hq // hkv
    qh = q.view(k, hkv, grp, d).permute(1, 0, 2, 3).reshape(hkv, k * grp, d)
    scores = (qh @ kv[0].permute(1, 2, 0)).view(hkv, k, grp, c + k) * (1.0 / math.sqrt(d))
    hidden = pos[None, :] > c + torch.arange(k, device=q.device)[:, None]
    scores.masked_fill_(hidden[None, :, None, :], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    o = (p.view(hkv, k * grp, c + k) @ kv[1].permute(1, 0, 2)).view(hkv, k, grp, d) / total
    lse = (top + torch.log(total)).squeeze(-1)
    return o.permute(1, 0, 2, 3).reshape(k, hq, d), lse.permute(1, 0, 2).reshape(k, hq)


def run(state):
    s = state
    case, op = s["case"], s["case"]["op"]
    if op == "rotate":
        if own:
            turn = dict(freq=s["freq"], interleaved=case["pairs"] == "inter", q_out=s["q_out"])
            if case["kv"] == "none":
                s["svp"].rope(s["q"], s["k"], s["ctx_len"], s["cu"], k_out=s["k_out"], **turn)
            else:
                s["svp"].rope_cache_write(s["q"], s["k"], s["v"], s["ctx_len"], s["cu"], cache=s["caches"][0], **turn)
                if case["kv"] == "e4m3":
                    s["svp"].cache_read(s["ctx_len"], s["cu"], cache=s["caches"][0], k_out=s["back"][0], v_out=s["back"][1])
        else:
            _rotate(s)
        # (what is held in 8 bits comes back as the values it stands for: this step's rows, read from the cache)
        return [s["q_out"], s["k_out"]] if case["kv"] == "none" else [s["q_out"]] + (s["back"] if case["kv"] == "e4m3" else s["pools"])
    if op == "attend":
        if own:
            s["svp"].prefix_attn(s["q"], s["ctx_len"], s["cu"], s["cu_groups"], s["prefix"], cache=s["caches"][0],
                                 w=case["rows"], out=s["out"], lse=s["lse"])
        else:
            parts = [_attend_one(s, i) for i in range(len(s["rows"]))]
            s["out"][:s["live"]] = torch.cat([o for o, _ in parts]).to(torch.bfloat16)
            s["lse"][:s["live"]] = torch.cat([t for _, t in parts])
        return [s["out"], s["lse"]]
    # this step's tables, which the call then changes
    s["now"].copy_(s["before"])
    if op == "resize":
        if own:
            s["svp"].pages_resize(s["pages"], s["length"])
        else:
            _resize(s)
        return [s["table"], s["used"], s["refs"]]
    if op == "fork":
        if own:
            s["svp"].pages_fork(s["pages"], s["src"], s["dst"], s["length"], caches=s["caches"])
        else:
            _fork(s)
    else:
        if own:
            s["svp"].pages_compact(s["pages"], caches=s["caches"])
        else:
            _compact(s)
    return [s["table"], s["used"], s["refs"]] + s["pools"] + [x for x in s["exps"] if x is not None]


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _cached(s, i, count, which):
    at = torch.arange(count, device=s["table"].device)
    pg, tok = s["table"][i][torch.div(at, s["case"]["page"], rounding_mode="floor")].long(), at.remainder(s["case"]["page"])
    pool, exps = s["pools"][which], s["exps"][which]
    if exps is None:
        return pool[pg, :, tok].double()
    two = ((exps[pg, :, tok].to(torch.int64) - 127 + 1023) << 52).view(torch.float64)
    return pool.view(torch.uint8)[pg, :, tok].view(torch.float8_e4m3fn).double() * two[..., None]


def exact(case, seed):
    op = case["op"]
    if op in ("resize", "fork", "compact"):
        return None                     # whole numbers and copies
    s = prepare(case, seed)
    hq, hkv, d = HEADS[case["heads"]]
    if op == "rotate":
        pos = torch.cat([torch.arange(c, c + k) for c, k in zip(s["ctx"], s["rows"])]).double().cuda()
        r = case["rot"]
        one, other = (lambda t: t, lambda t: t + r // 2) if case["pairs"] == "half" else (lambda t: 2 * t, lambda t: 2 * t + 1)
        got = []
        for x in (s["q"], s["k"]):
            y = x[:s["live"]].double()
            z = y.clone()
            for t in range(r // 2):
                turn = torch.exp(1j * (pos * s["rad"][t]))[:, None] * torch.complex(y[..., one(t)], y[..., other(t)])
                z[..., one(t)], z[..., other(t)] = turn.real, turn.imag
            got.append(z)
        q, k = s["q_out"].double(), got[1]
        q[:s["live"]] = got[0]
        if case["kv"] == "none":
            keys = s["k_out"].double()
            keys[:s["live"]] = k
            return [q, keys]
        if case["kv"] == "e4m3":
            return [q, None, None]      # what 8 bits hold of a row has no value of its own
        pools = [x.double() for x in s["pools"]]
        first = 0
        for i, (c, n) in enumerate(zip(s["ctx"], s["rows"])):
            at = torch.arange(c, c + n, device="cuda")
            pg, tok = s["table"][i][torch.div(at, case["page"], rounding_mode="floor")].long(), at.remainder(case["page"])
            pools[0][pg, :, tok] = k[first:first + n]
            pools[1][pg, :, tok] = s["v"][first:first + n].double()
            first += n
        return [q] + pools
    out, lse = s["out"].double(), s["lse"].double()
    first = 0
    for i, (c, n) in enumerate(zip(s["ctx"], s["rows"])):
        keys, vals = _cached(s, i, c + n, 0), _cached(s, i, c + n, 1)
        seen = c + torch.arange(n, device=keys.device)
        late = torch.arange(c + n, device=keys.device)[None] > seen[:, None]
        for h in range(hq):
            z = s["q"][first:first + n, h].double() @ keys[:, h // (hq // hkv)].T / math.sqrt(d)
            z = torch.where(late, torch.full_like(z, -math.inf), z)
            lse[first:first + n, h] = torch.logsumexp(z, -1)
            out[first:first + n, h] = torch.softmax(z, -1) @ vals[:, h // (hq // hkv)]
        first += n
    return [out, lse]
