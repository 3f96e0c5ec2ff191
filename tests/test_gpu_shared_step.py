"""The calls around the cache as a generation with parallel samples uses them: one prompt, forks of it, steps of
resize -> rope_cache_write -> prefix_attn -> accept -> resize, a sample that ends, a compaction, more steps.  Beside it
the same rows go through a cache without any sharing, by rope, cache_write and chunk_attn."""
import pytest
import torch

import speculative_decoding_verification_packed_gb300 as svp
from test_gpu_cache import BF16, E4M3, i32, packed

pytestmark = pytest.mark.gpu

N, HQ, HKV, D, PAGE, W, VOCAB, LAYERS = 7, 8, 2, 128, 16, 4, 32, 2


def pools(kind, pages):
    out = []
    for _ in range(LAYERS):
        x = [torch.zeros(pages, HKV, PAGE, D, dtype=kind, device="cuda") for _ in range(2)]
        e = [torch.full((pages, HKV, PAGE), 127, dtype=torch.uint8, device="cuda") for _ in range(2)] if kind == E4M3 else [None] * 2
        out.append((x, e))
    return out


def caches(pool, table):
    return [svp.make_cache(x[0], x[1], table, k_exp=e[0], v_exp=e[1]) for x, e in pool]


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("prompt", [150, 160])
@pytest.mark.parametrize("captured", [False, True])
def test_samples_of_one_prompt(kind, prompt, captured):
    g = torch.Generator(device="cuda").manual_seed(5)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)
    freq = svp.rope_frequencies(D, base=500000.0, scaling="yarn", factor=4.0, original=4096)
    cols = 20
    # shared: 44 pages for what would be 6 x 13 apart; request 6 is another prompt's, alone
    table = torch.full((N, cols), -1, dtype=torch.int32, device="cuda")
    used, refs = torch.zeros(N, dtype=torch.int32, device="cuda"), torch.zeros(60, dtype=torch.int32, device="cuda")
    pages = svp.make_pages(table, used, refs, page_size=PAGE)
    pool = pools(kind, 60)
    cache = caches(pool, table)
    # apart: every request has its own pages from the start
    own_table = torch.arange(N * cols, dtype=torch.int32, device="cuda").view(N, cols).contiguous()
    own_pool = pools(kind, N * cols)
    own = caches(own_pool, own_table)
    other = 37
    ctx = i32([0] * N)
    cu_p = i32([0] + [prompt] * 6 + [prompt + other])
    svp.pages_resize(pages, i32([prompt] + [0] * 5 + [other]))
    for layer in range(LAYERS):
        q, k, v = randn(prompt + other, HQ, D), randn(prompt + other, HKV, D), randn(prompt + other, HKV, D)
        turned = svp.rope_cache_write(q, k, v, ctx, cu_p, cache=cache[layer], freq=freq)
        qr, kr = svp.rope(q, k, ctx, cu_p, freq=freq)
        assert torch.equal(turned, qr)
        # the plain cache: every one of the six samples writes the prompt itself
        kk = torch.cat([kr[:prompt]] * 6 + [kr[prompt:]])
        vv = torch.cat([v[:prompt]] * 6 + [v[prompt:]])
        if kind == E4M3:        # one rounding from fp32 to 8 bits, as the fused call's
            _, kf = svp.rope(None, k.float(), ctx, cu_p, freq=freq)
            kk = torch.cat([kf[:prompt]] * 6 + [kf[prompt:]])
            vv = vv.float()
        svp.cache_write(kk, vv, ctx, i32(packed([prompt] * 6 + [other])), cache=own[layer])
    svp.pages_fork(pages, i32([0] * 5), i32([1, 2, 3, 4, 5]), i32([prompt] * 5), caches=cache)
    assert pages.ws.read_status() == 0
    whole = prompt // PAGE
    assert refs[table[0, :whole].long()].tolist() == [6] * whole
    ctx = i32([prompt] * 6 + [other])
    rows = i32([W] * N)
    cu_groups, prefix_len = i32([0, 6]), i32([prompt])
    bufs = [randn(N * W, HQ, D), randn(N * W, HKV, D), randn(N * W, HKV, D), randn(N * W, VOCAB)]
    tokens = torch.zeros(N * W, dtype=torch.int32, device="cuda")
    cu = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
    qo = [torch.zeros(N * W, HQ, D, dtype=BF16, device="cuda") for _ in range(LAYERS)]
    out = [torch.zeros(N * W, HQ, D, dtype=BF16, device="cuda") for _ in range(LAYERS)]
    lse = [torch.zeros(N * W, HQ, device="cuda") for _ in range(LAYERS)]
    acc, nxt = i32([0] * N), i32([0] * N)
    before = i32([0] * N)

    def step():
        """(rows of requests that have ended: 0)"""
        before.copy_(ctx)
        cu[1:].copy_(rows.cumsum(0))
        svp.pages_resize(pages, torch.where(rows > 0, ctx + rows, -1).int())
        for layer in range(LAYERS):
            svp.rope_cache_write(bufs[0], bufs[1], bufs[2], ctx, cu, cache=cache[layer], freq=freq, q_out=qo[layer])
            svp.prefix_attn(qo[layer], ctx, cu, cu_groups, prefix_len, cache=cache[layer], w=W, out=out[layer], lse=lse[layer])
        svp.margin_accept(bufs[3], tokens, cu, outs=margin + (acc, nxt), ws=mws)
        ctx.add_(acc)
        svp.pages_resize(pages, torch.where(rows > 0, ctx, -1).int())

    margin = tuple(torch.zeros(N * W, dtype=t, device="cuda") for t in (torch.int32,) + (torch.float32,) * 3)
    mws = svp.Workspace(svp.margin_accept_workspace_size(N, N * W, VOCAB))

    def feed():
        for b in bufs:
            b.copy_(randn(*b.shape))
        top = bufs[3].float().argmax(-1).int()
        tokens.copy_(torch.randint(0, VOCAB, tokens.shape, generator=g, device="cuda"))
        keep = torch.rand(N * W, generator=g, device="cuda") < 0.6
        tokens[1:] = torch.where(keep[1:], top[:-1], tokens[1:])

    def plain():
        """The same rows through the cache without sharing; the kept ones are those that were accepted."""
        live = int(cu[-1])
        lens = ctx.tolist()
        for layer in range(LAYERS):
            qr, kr = svp.rope(bufs[0], bufs[1], before, cu, freq=freq)
            assert torch.equal(qr[:live], qo[layer][:live])
            v = bufs[2]
            if kind == E4M3:
                _, kr = svp.rope(None, bufs[1].float(), before, cu, freq=freq)
                v = v.float()
            svp.cache_write(kr, v, before, cu, cache=own[layer])
            o, l = svp.chunk_attn(qr, before, cu, cache=own[layer], w=W)
            cu_c = packed([x if r else 0 for x, r in zip(lens, rows.tolist())])
            a = svp.cache_read(None, i32(cu_c), cache=cache[layer], rows=cu_c[-1])
            b = svp.cache_read(None, i32(cu_c), cache=own[layer], rows=cu_c[-1])
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])       # every kept position of every request
            # two kernels over the same values: each probability and each output is off by half a bf16 step in both
            size = float(max(b[1].float().abs().max(), bufs[2].float().abs().max()))
            assert ((out[layer][:live].float() - o[:live].float()).abs() <= 4 * 2.0 ** -8 * size).all()
            # 8-bit scores are products with the query in fp16 (2^-11 of its elements), whichever kernel takes them
            assert ((lse[layer][:live] - l[:live]).abs() <= 2.0 ** -8).all()

    graph = None
    if captured:
        keep = [t.clone() for t in (ctx, table, used, refs)]
        state = [[t.clone() for t in x + [y for y in e if y is not None]] for x, e in pool]
        feed()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for t, s in zip((ctx, table, used, refs), keep):
            t.copy_(s)
        for (x, e), s in zip(pool, state):
            for t, u in zip(x + [y for y in e if y is not None], s):
                t.copy_(u)
    for turn in range(9):
        feed()
        if turn == 3:                     # sample 2 has ended, and so has the prompt's first request
            rows.copy_(i32([0, W, 0, W, W, W, W]))
            svp.pages_resize(pages, i32([0, -1, 0, -1, -1, -1, -1]))
        if turn == 5:
            live = i32([0])
            svp.pages_compact(pages, caches=cache, live=live)
            assert int(refs[int(live):].abs().sum()) == 0 and (refs[:int(live)] > 0).all()
        graph.replay() if graph else step()
        torch.cuda.synchronize()
        assert pages.ws.read_status() == 0
        plain()
    assert acc.max() > 1                  # (some drafts were accepted)
    # all end: every page is free again
    svp.pages_resize(pages, i32([0] * N))
    assert (refs == 0).all() and (table == -1).all() and (used == 0).all() and pages.ws.read_status() == 0
