"""The scratch of prefix_attn calls that bring no workspace: it takes no place from chunk_attn's, and that of a call of
many rows is not kept."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_packed_gb300 as svp
from test_gpu_cache import BF16, i32, packed
from test_gpu_prefix import Shared, attend_exact

pytestmark = pytest.mark.gpu


def setup(rows, ctx, groups, hq, hkv, d, m_cap, seed=5):
    pool = Shared(rows, ctx, groups, hkv, d, 16, BF16, seed=seed)
    q = torch.randn(m_cap, hq, d, generator=torch.Generator().manual_seed(seed)).to(BF16).cuda()
    return pool, pool.cuda(), q, i32(ctx), i32(packed(rows)), i32([0, len(rows)]), i32([groups[0][2]])


def test_chunk_attn_keeps_its_own():
    pool, cache, q, ctx, cu, groups, length = setup([1, 2], [70, 80], [(0, 2, 64)], 4, 2, 64, 3)
    streams = [torch.cuda.Stream() for _ in range(16)]
    torch.cuda.synchronize()
    want = svp.prefix_attn(q, ctx, cu, groups, length, cache=cache)
    svp._chunk_ws.clear()
    for s in streams:
        svp.chunk_attn(q, ctx, cu, cache=cache, stream=s)
    kept = list(svp._chunk_ws.values())
    assert len(kept) == 16
    outs = [svp.prefix_attn(q, ctx, cu, groups, length, cache=cache, stream=s) for s in streams + streams]
    torch.cuda.synchronize()
    assert all(a is b for a, b in zip(kept, svp._chunk_ws.values())) and len(svp._chunk_ws) == 16
    assert all(torch.equal(a, want[0]) and torch.equal(b, want[1]) for a, b in outs)


def test_the_scratch_of_many_rows_is_not_kept():
    """8 bytes for each of 5000 x 32 x 128 elements; two calls in a row on one stream, and calls of few rows between."""
    rows, ctx, m_cap = [3, 1], [200, 210], 5000
    pool, cache, q, *args = setup(rows, ctx, [(0, 2, 192)], 32, 8, 128, m_cap)
    size = svp.prefix_attn_workspace_size(32, 8, 128, m_cap)
    assert size > 128 << 20 >= svp.prefix_attn_workspace_size(32, 8, 128, 4)
    few = svp.prefix_attn(q[:4], *args, cache=cache, w=3)            # (what is kept stands already)
    before = torch.cuda.memory_allocated()
    outs = []
    for _ in range(2):
        outs.append(svp.prefix_attn(q, *args, cache=cache, w=3))
        outs.append(svp.prefix_attn(q[:4], *args, cache=cache, w=3))
    torch.cuda.synchronize()
    made = sum(-(-x.numel() * x.element_size() // 512) * 512 for pair in outs for x in pair)
    assert torch.cuda.memory_allocated() - before <= made + (8 << 20) < made + size - (47 << 20)
    # (the joining kernel adds a row's parts in another order where the call has many rows, as one or eight half warps take
    # them: bits are compared between calls of one size, and either size with the bound in 64 bits, which holds any order)
    o, l, tol, ltol = attend_exact(pool, q[:4], rows, ctx, 1 / math.sqrt(128))
    for i, (out, lse) in enumerate(outs):
        like = outs[0] if i % 2 == 0 else few
        assert torch.equal(out, like[0]) and torch.equal(lse, like[1])
        assert not out[4:].any() and not lse[4:].any()
        assert (np.abs(out[:4].double().cpu().numpy() - o) <= tol).all()
        assert (np.abs(lse[:4].double().cpu().numpy() - l) <= ltol).all()
