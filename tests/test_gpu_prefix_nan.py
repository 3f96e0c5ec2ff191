"""A key of NaN that only the last row of one request sees, by every type of page: the rows of other requests keep their
bits, the rows of its own request keep their values."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_packed_gb300 as svp
from test_gpu_cache import BF16, E4M3, F32, i32, packed
from test_gpu_prefix import Shared, attend_exact

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [BF16, E4M3, F32])
@pytest.mark.parametrize("hq,hkv,d,rows,ctx,tokens", [(4, 2, 128, [2, 1, 1], [300, 310, 290], 288),
                                                      (16, 2, 64, [3, 5, 1], [140, 131, 170], 128),
                                                      (8, 2, 256, [4, 2, 2], [300, 400, 290], 272),
                                                      (8, 1, 128, [40, 33, 2], [600, 520, 513], 512)])
def test_rows_beside_a_nan_key(hq, hkv, d, rows, ctx, tokens, kind):
    qt = F32 if kind == F32 else BF16
    pool = Shared(rows, ctx, [(0, 3, tokens)], hkv, d, 16, kind, seed=hq + d)
    cache = pool.cuda()
    q = torch.randn(sum(rows), hq, d, generator=torch.Generator().manual_seed(d)).to(qt).cuda()
    args = (q, i32(ctx), i32(packed(rows)), i32([0, 3]), i32([tokens]))
    want, wl = svp.prefix_attn(*args, cache=cache)
    x = torch.full((1, hkv, d), float("nan"), device="cuda", dtype=qt)
    last = rows[0] - 1
    svp.cache_write(x, torch.ones_like(x), i32([ctx[0] + last, 0, 0]), i32([0, 1, 1, 1]), cache=cache)
    out, lse = svp.prefix_attn(*args, cache=cache)
    assert torch.isnan(out[last]).all() and torch.isnan(lse[last]).all()
    others = slice(rows[0], None)
    assert torch.equal(out[others], want[others]) and torch.equal(lse[others], wl[others])
    o, l, tol, ltol = attend_exact(pool, q, rows, ctx, 1 / math.sqrt(d))     # (the pool's values without the NaN)
    assert (np.abs(out[:last].double().cpu().numpy() - o[:last]) <= tol[:last]).all()
    assert (np.abs(lse[:last].double().cpu().numpy() - l[:last]) <= ltol[:last]).all()
