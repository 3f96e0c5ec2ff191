"""prefix_attn on the GPU against softmax attention in 64 bits, with the bounds of chunk_attn's tests: a row's two
parts are joined in fp32, one product and one sum more for each, which the bounds' 64 steps of 2^-23 hold."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_packed_gb300 as svp
from test_gpu_cache import BF16, E4M3, F32, Pool, i32, pack_rows, packed, picked_rows

pytestmark = pytest.mark.gpu


def attend_exact(pool, q, rows, ctx, scale, picks=None):
    """test_gpu_cache.attend_exact (the same values and bounds), all heads of a row at once."""
    hq, d = q.shape[1:]
    G = hq // pool.hkv
    half = 2.0 ** -24 if pool.kind == F32 else 2.0 ** -8
    o, lse, tol, ltol = [], [], [], []
    q = q.double().cpu().numpy()
    first = 0
    for i, r in enumerate(rows):
        take = range(r) if picks is None else sorted({j for j in picks if j < r} | {r - 1} if r else set())
        if len(take):
            K, V = (np.ascontiguousarray(pool.rows(w, i, 0, ctx[i] + r).transpose(1, 0, 2)) for w in range(2))   # [hkv, T, d]
        for j in take:
            T = ctx[i] + j + 1
            k, v = K[:, :T], V[:, :T]
            x = q[first + j].reshape(pool.hkv, G, d)
            s = x @ k.transpose(0, 2, 1) * scale                                                                 # [hkv, G, T]
            ds = (d + 2) * 2.0 ** -23 * (np.abs(x) @ np.abs(k).transpose(0, 2, 1)).max(-1, keepdims=True) * scale
            top = s.max(-1, keepdims=True)
            p = np.exp(s - top)
            l = p.sum(-1, keepdims=True)
            y, A = p @ v / l, p @ np.abs(v) / l
            rel = (0 if pool.kind == F32 else half) + 2 * ds + (T / 32 + 64) * 2.0 ** -23
            o.append(y)
            tol.append(rel * A + half * np.abs(y) + 1e-30)
            lse.append(top + np.log(l))
            ltol.append(ds + (T / 32 + 64) * 2.0 ** -23 + np.abs(lse[-1]) * 2.0 ** -22)
        first += r
    return (np.array(o).reshape(-1, hq, d), np.array(lse).reshape(-1, hq), np.array(tol).reshape(-1, hq, d),
            np.array(ltol).reshape(-1, hq))


class Shared(Pool):
    """A pool whose groups (first request, end, tokens) have their first whole pages in common: the pages of the first
    request that has rows; the others have pages of their own for the rest only."""

    def __init__(self, rows, ctx, groups, hkv, d, page, *args, **kw):
        n = len(rows)
        total = [a + b if a else 0 for a, b in zip(rows, ctx)]
        lead, common = list(range(n)), [0] * n
        for lo, hi, tokens in groups:
            live = [i for i in range(lo, hi) if rows[i]]
            for i in live[1:]:
                lead[i], common[i] = live[0], max(tokens, 0) // page
        super().__init__(n, [t - c * page for t, c in zip(total, common)], hkv, d, page, *args, **kw)
        own = self.table
        self.table = torch.full((n, max([-(-t // page) for t in total] + [1])), -1, dtype=torch.int32)
        for i in range(n):
            k = -(-total[i] // page) - common[i]
            self.table[i, :common[i]] = own[lead[i], :common[i]]
            self.table[i, common[i]:common[i] + k] = own[i, :k]
        self.lens = total


def group_tensors(groups, n):
    """cu_groups and prefix_len of groups in order; what lies between two is a group of its own, with no prefix."""
    cu, length = [groups[0][0] if groups else 0], []
    for lo, hi, tokens in groups:
        if lo > cu[-1]:
            cu.append(lo)
            length.append(0)
        cu.append(hi)
        length.append(tokens)
    return i32(cu), i32(length)


def check_prefix(rows, ctx, groups, *, hq=4, hkv=2, d=128, page=16, kind=BF16, layout="head", picks=None, seed=0, std=1.0,
                 scale=0.0, pad=3, fused=False, ws=None, pool=None):
    n = len(rows)
    pool = pool or Shared(rows, ctx, groups, hkv, d, page, kind, layout, seed=seed, std=std)
    cache = pool.cuda()
    cu = packed(rows)
    g = torch.Generator().manual_seed(seed + 1)
    qt = F32 if kind == F32 else BF16
    q = torch.randn(cu[-1] + pad, hq + (2 * hkv if fused else 0), d, generator=g).to(qt).cuda()[:, :hq]
    out = torch.full((cu[-1] + pad, hq, d), -7.0, dtype=qt, device="cuda")
    lse = torch.full((cu[-1] + pad, hq), -7.0, device="cuda")
    ws = ws or svp.Workspace(svp.prefix_attn_workspace_size(hq, hkv, d, cu[-1] + pad, qt), zeroed=256)
    svp.prefix_attn(q, i32(ctx), i32(cu), *group_tensors(groups, n), cache=cache, w=max(rows + [1]), out=out, lse=lse,
                    scale=scale, ws=ws)
    torch.cuda.synchronize()
    assert ws.read_status() == 0
    o, l, tol, ltol = attend_exact(pool, q, rows, ctx, scale or 1 / math.sqrt(d), picks)
    at = picked_rows(rows, picks)
    got = out.double().cpu().numpy()
    assert np.isfinite(got[:cu[-1]]).all()
    assert (got[cu[-1]:] == -7).all() and (lse[cu[-1]:] == -7).all()
    err = np.abs(got[at] - o)
    assert (err <= tol).all(), (float((err / tol).max()), np.argwhere(err > tol)[:5].tolist())
    lerr = np.abs(lse.double().cpu().numpy()[at] - l)
    assert (lerr <= ltol).all(), (float((lerr / ltol).max()), np.argwhere(lerr > ltol)[:5].tolist())
    return out, lse


CASES = [
    # rows, tokens before them, groups (first, end, shared tokens)
    ([1, 1], [16, 16], [(0, 2, 16)]),                                       # nothing but the new token itself
    ([1, 1], [17, 40], [(0, 2, 16)]),
    ([1] * 8, [4100 + 13 * i for i in range(8)], [(0, 8, 4096)]),
    ([1] * 5, [300, 130, 131, 150, 1000], [(1, 4, 128)]),                   # others alone before and behind
    ([2, 7, 1, 16, 3, 5], [600, 513, 700, 1025, 1024, 1100], [(0, 3, 512), (3, 6, 1024)]),
    ([0, 0, 3, 0, 4, 0], [0, 9, 200, 3, 222, 0], [(0, 6, 199)]),            # first one without rows; part of a page
    ([1, 1, 1], [250, 255, 260], [(0, 3, 250)]),
    ([40, 50, 90], [300, 280, 299], [(0, 3, 272)]),                         # several query tiles and blocks
    ([200, 1, 1, 3], [140, 129, 140, 128], [(0, 4, 128)]),
    ([257, 256], [40, 48], [(0, 2, 32)]),                                   # fill their own blocks: not shared
    ([5, 5], [9, 7], [(0, 2, 7)]),                                          # no whole page
    ([5, 6, 7], [90, 80, 70], [(0, 1, 64), (1, 2, 64), (2, 3, 48)]),        # groups of one
    ([3] * 12, [200 + i for i in range(12)], [(0, 4, 192), (4, 5, 0), (5, 9, 96), (9, 12, 192)])]


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("rows,ctx,groups", CASES)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_groups(rows, ctx, groups, d, kind):
    check_prefix(rows, ctx, groups, d=d, kind=kind, picks=(0, 1, 31, 32, 63, 64, 127, 128, 200))


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (12, 1), (24, 2), (8, 8), (128, 1), (5, 1), (48, 3)])
def test_head_layouts(hq, hkv, kind):
    check_prefix([1, 9, 1, 30], [300, 258, 257, 270], [(0, 4, 256)], hq=hq, hkv=hkv, kind=kind, page=32, picks=(0, 8, 29),
                 fused=True, seed=4)


@pytest.mark.parametrize("kind", [BF16, E4M3, F32])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("layout", ["head", "token"])
def test_pages_and_strides(page, layout, kind):
    check_prefix([1, 20, 7, 2], [211, 400, 390, 1100], [(1, 4, 389)], page=page, layout=layout, kind=kind, fused=True, seed=7)


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_long_prefixes_and_long_rests(d, kind):
    """Either part split over many blocks, and both."""
    check_prefix([1, 1], [9001, 9100], [(0, 2, 8992)], hq=2, hkv=1, d=d, kind=kind, seed=8)
    check_prefix([3, 1], [6000, 4095], [(0, 2, 32)], hq=6, hkv=2, d=d, kind=kind, seed=9, std=2.0)
    check_prefix([2, 1, 4], [9000, 4600, 5095], [(0, 3, 4592)], hq=2, hkv=2, d=d, kind=kind, seed=10)


@pytest.mark.parametrize("kind", [BF16, E4M3])
def test_many_groups(kind):
    n = 300
    rows = [1 + i % 3 for i in range(n)]
    groups = [(i, i + 3, 16 * (1 + i % 5)) for i in range(0, n, 3)]
    ctx = [16 * (1 + (i - i % 3) % 5) + (7 * i) % 60 for i in range(n)]
    check_prefix(rows, ctx, groups, hq=2, hkv=1, d=64, kind=kind, seed=11)


def crowd(n, rows, shared, rest, seed):
    """n requests of up to `rows` rows (some none) in groups of different sizes, some alone."""
    r = np.random.default_rng(seed)
    k = r.integers(0, rows + 1, n).tolist()
    ctx, groups, at = [0] * n, [], 0
    while at < n:
        size = int(r.integers(1, 30))
        hi = min(n, at + size)
        tokens = int(r.integers(0, shared)) if r.random() < 0.8 else 0
        for i in range(at, hi):
            ctx[i] = tokens + int(r.integers(0, rest))
        groups.append((at, hi, tokens))
        at = hi
    return k, ctx, groups


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("hq,hkv,rows", [(4, 4, 1), (8, 8, 8), (16, 4, 2), (12, 4, 5), (32, 8, 4), (16, 16, 16), (20, 4, 3),
                                         (64, 4, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_crowds_of_few_rows(hq, hkv, rows, d, kind):
    """Requests of up to 16 rows a KV head, more than 300 of them times their heads: a kernel of their own."""
    n = 320 // hkv + 9
    k, ctx, groups = crowd(n, rows, 600, 300, hq + rows + d)
    check_prefix(k, ctx, groups, hq=hq, hkv=hkv, d=d, kind=kind, seed=hq, page=32 if rows > 4 else 16, fused=True)


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("layout", ["head", "token"])
def test_crowds_over_any_pages(page, layout, kind):
    k, ctx, groups = crowd(80, 2, 700, 500, page)
    check_prefix(k, ctx, groups, hq=8, hkv=4, kind=kind, page=page, layout=layout, seed=3)


@pytest.mark.parametrize("kind", [BF16, E4M3])
def test_crowds_with_long_rests_and_wide_scores(kind):
    """Own keys that are split over blocks, and scores far apart."""
    n = 80
    ctx = [64 + (9000 if i % 40 == 7 else 17 * i % 90) for i in range(n)]
    check_prefix([1 + i % 2 for i in range(n)], ctx, [(0, 30, 64), (30, 80, 48)], hq=8, hkv=4, kind=kind, seed=5, picks=(0, 1))
    check_prefix([1] * n, [700 + i for i in range(n)], [(0, n, 640)], hq=4, hkv=4, kind=kind, scale=2.0, std=4.0, seed=6)


@pytest.mark.parametrize("kind", [BF16, E4M3])
def test_crowds_keep_their_neighbours_nan_out(kind):
    """A key of NaN that one row of a crowd sees, another that is behind every row of its request."""
    n, hkv, d = 80, 4, 128
    rows, ctx, groups = [2] * n, [130 + i for i in range(n)], [(0, n, 128)]
    pool = Shared(rows, ctx, groups, hkv, d, 16, kind, seed=7)
    cache = pool.cuda()
    q = torch.randn(2 * n, 8, d, device="cuda").to(BF16)
    args = (i32(ctx), i32(packed(rows)), i32([0, n]), i32([128]))
    before = svp.prefix_attn(q, *args, cache=cache, w=2)
    x = torch.full((1, hkv, d), float("nan"), device="cuda", dtype=BF16)
    at = [0] * n
    at[5] = ctx[5] + 1                     # the last row's own
    cu = [0] * 6 + [1] * (n - 5)
    svp.cache_write(x, torch.ones_like(x), i32(at), i32(cu), cache=cache)
    out, lse = svp.prefix_attn(q, *args, cache=cache, w=2)
    assert torch.isnan(out[11]).all() and torch.isnan(lse[11]).all()
    keep = [r for r in range(2 * n) if r not in (10, 11)]
    assert torch.equal(out[keep], before[0][keep]) and torch.equal(lse[keep], before[1][keep])
    assert torch.isfinite(out[10]).all() and torch.isfinite(lse[10]).all()
    ws = svp.Workspace(svp.prefix_attn_workspace_size(8, hkv, d, 2 * n), zeroed=256)
    ws.buf[256:] = 255
    for c, bit in (([130 + i if i != 9 else -1 for i in range(n)], svp.DEV_BAD_CONTEXT), (ctx, 0)):
        out, lse = torch.full((2 * n, 8, d), -7.0, dtype=BF16, device="cuda"), torch.full((2 * n, 8), -7.0, device="cuda")
        svp.prefix_attn(q, i32(c), *args[1:], cache=cache, w=2, out=out, lse=lse, ws=ws)
        assert ws.read_status() == bit
        assert bool((out[18:20] == -7).all()) == bool(bit) and not (out[:18] == -7).all(-1).any()


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_the_most_requests_and_groups(d, kind):
    """1024 requests in one group, and in 1024 groups; most of them without rows."""
    rows, ctx = [0] * 1024, [0] * 1024
    for i, (r, c) in {3: (1, 140), 500: (150, 160), 900: (2, 129), 1023: (70, 131)}.items():
        rows[i], ctx[i] = r, c
    check_prefix(rows, ctx, [(0, 1024, 128)], hq=4, hkv=1, d=d, kind=kind, seed=19, picks=(0, 1, 69, 149))
    check_prefix(rows, ctx, [(i, i + 1, 16) for i in range(1024)], hq=4, hkv=1, d=d, kind=kind, seed=19, picks=(0, 1, 69, 149))
    check_prefix([1] * 1024, [48 + i % 20 for i in range(1024)], [(0, 1024, 48)], hq=2, hkv=1, d=d, kind=kind, seed=20,
                 page=32)


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("at,high", [(3, 40.0), (3, 416.0), (300, 40.0), (300, 416.0), (520, 40.0), (520, 416.0)])
def test_one_part_outweighs_the_other(at, high, kind):
    """A key far above the others (2^60 and 2^600 in probability) in the common part's first tile, a later one of
    its, and in one request's own: the other rows keep their own weights."""
    d, hkv, page, rows = 64, 2, 16, [1, 2, 1]
    ctx, groups = [530, 560, 700], [(0, 3, 512)]
    pool = Shared(rows, ctx, groups, hkv, d, page, kind, seed=32)
    row = np.zeros(d)
    row[0] = high                          # (bf16 and e4m3 values)
    pg = int(pool.table[0, at // page])
    pool.vals[0][pg, :, at % page] = row
    codes, b = pack_rows(row)
    if kind == E4M3:
        pool.raw[0][pg, :, at % page] = torch.from_numpy(codes)
        pool.exps[0][pg, :, at % page] = int(b)
    else:
        pool.raw[0][pg, :, at % page] = torch.from_numpy(row).to(BF16)
    cache = pool.cuda()
    q = torch.randn(4, hkv, d, generator=torch.Generator().manual_seed(33)).to(BF16)
    q[..., 0] = 8.0                        # the scale is 1 / 8
    q = q.cuda()
    out, lse = svp.prefix_attn(q, i32(ctx), i32(packed(rows)), i32([0, 3]), i32([512]), cache=cache)
    o, l, tol, ltol = attend_exact(pool, q, rows, ctx, 1 / math.sqrt(d))
    assert (np.abs(out.double().cpu().numpy() - o) <= tol).all()
    assert (np.abs(lse.double().cpu().numpy() - l) <= ltol).all()


@pytest.mark.parametrize("kind", [BF16, E4M3])
def test_wide_scores(kind):
    check_prefix([3, 40, 1], [700, 900, 640], [(0, 3, 640)], kind=kind, scale=2.0, std=4.0, seed=10, picks=(0, 1, 39))


@pytest.mark.parametrize("kind", [BF16, E4M3, F32])
def test_nan_keys_reach_the_rows_that_see_them(kind):
    rows, ctx, groups = [2, 1, 1], [300, 310, 290], [(0, 2, 288)]
    qt = F32 if kind == F32 else BF16
    pool = Shared(rows, ctx, groups, 2, 128, 16, kind, seed=14)
    cache = pool.cuda()
    x = torch.full((1, 2, 128), float("nan"), device="cuda", dtype=qt)
    y = torch.ones(1, 2, 128, device="cuda", dtype=qt)
    q = torch.randn(4, 4, 128, device="cuda").to(qt)
    cu, c, gr, ln = i32(packed(rows)), i32(ctx), i32([0, 2]), i32([288])
    want = svp.prefix_attn(q, c, cu, gr, ln, cache=cache)
    svp.cache_write(x, y, i32([301, 0, 0]), i32([0, 1, 1, 1]), cache=cache)      # the last row's own key of request 0
    out, lse = svp.prefix_attn(q, c, cu, gr, ln, cache=cache)
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    if kind != E4M3:                       # (an 8-bit tile's scale leaves NaN rows out, its other digits may move)
        assert torch.equal(out[[0, 2, 3]], want[0][[0, 2, 3]])
    assert torch.isfinite(out[[0, 2, 3]]).all() and torch.isfinite(lse[[0, 2, 3]]).all()
    svp.cache_write(x, y, i32([100, 0, 0]), i32([0, 1, 1, 1]), cache=cache)      # a common one
    out, lse = svp.prefix_attn(q, c, cu, gr, ln, cache=cache)
    assert torch.isnan(out[:3]).all() and torch.isnan(lse[:3]).all() and torch.isfinite(out[3]).all()


def test_one_workspace_for_any_call():
    nb = max(svp.prefix_attn_workspace_size(8, 2, d, 400) for d in (64, 128, 256))
    ws = svp.Workspace(nb, zeroed=256)
    ws.buf[256:] = 255                     # (NaN bits: nothing may rest on what is there)
    for d in (64, 256, 128, 64):
        for kind in (BF16, E4M3):
            for rows, ctx, groups in (([1, 1], [4000, 4010], [(0, 2, 3984)]), ([70, 3, 200], [300, 2000, 260], [(0, 3, 256)]),
                                      ([1] * 40, [257] * 40, [(3, 30, 256)])):
                check_prefix(rows, ctx, groups, hq=8, hkv=2, d=d, kind=kind, ws=ws, picks=(0, 2, 63, 64), seed=29)


@pytest.mark.parametrize("kind", [BF16, E4M3])
def test_same_inputs_give_the_same_bits_and_no_groups_those_of_chunk_attn(kind):
    rows, ctx, groups = [1, 129, 1, 2], [4000, 4001, 4100, 3999], [(0, 4, 3984)]
    pool = Shared(rows, ctx, groups, 2, 128, 16, kind, seed=12)
    cache = pool.cuda()
    q = torch.randn(133, 8, 128, device="cuda").to(BF16)
    cu, c = i32(packed(rows)), i32(ctx)
    first = svp.prefix_attn(q, c, cu, i32([0, 4]), i32([3984]), cache=cache)
    for _ in range(5):
        again = svp.prefix_attn(q, c, cu, i32([0, 4]), i32([3984]), cache=cache)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    plain = svp.chunk_attn(q, c, cu, cache=cache)
    for gr, ln in (([0], []), ([0, 4], [0]), ([2, 3], [3984]), ([0, 4], [15])):
        got = svp.prefix_attn(q, c, cu, i32(gr), i32(ln), cache=cache)
        assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])
    out, none = svp.prefix_attn(q, c, cu, i32([0, 4]), i32([3984]), cache=cache, want_lse=False)
    assert none is None and torch.equal(out, first[0])


def test_broken_descriptions():
    rows, ctx, groups = [2, 2, 2, 2], [100, 90, 85, 120], [(0, 4, 80)]
    pool = Shared(rows, ctx, groups, 2, 64, 16, BF16, seed=3)
    cache = pool.cuda()
    q = torch.randn(8, 4, 64, device="cuda").to(BF16)
    ws = svp.Workspace(svp.prefix_attn_workspace_size(4, 2, 64, 8), zeroed=256)
    want, wl = svp.chunk_attn(q, i32(ctx), i32(packed(rows)), cache=cache, w=2)
    scale = float(np.nanmax(np.abs(pool.vals[1])))

    def run(cu=packed(rows), c=ctx, gr=(0, 4), ln=(80,), w=2):
        out, lse = torch.full((8, 4, 64), -7.0, dtype=BF16, device="cuda"), torch.full((8, 4), -7.0, device="cuda")
        svp.prefix_attn(q, i32(c), i32(cu), i32(list(gr)), i32(list(ln)), cache=cache, w=w, out=out, lse=lse, ws=ws)
        return out, lse, ws.read_status()

    def same(out, lse, rows_):
        # two splits of the same sums: half a bf16 step of each probability and of the output in both
        assert ((out[rows_].float() - want[rows_].float()).abs() <= 4 * 2.0 ** -8 * scale).all()
        assert ((lse[rows_] - wl[rows_]).abs() <= 2.0 ** -16 * (1 + wl[rows_].abs())).all()

    every = list(range(8))
    out, lse, st = run()
    assert st == 0
    same(out, lse, every)
    for cu in ([0, 2, 1, 6, 8], [-1, 2, 4, 6, 8], [0, 2, 4, 6, 9], [0, 20, 4, 6, 8]):      # the whole call
        out, lse, st = run(cu=cu)
        assert st == svp.DEV_BAD_SLOTS and (out == -7).all() and (lse == -7).all()
    for gr, ln in (([0, 3, 1, 4], [80, 80, 80]), ([0, 5], [80]), ([-1, 4], [80])):         # no group at all
        out, lse, st = run(gr=gr, ln=ln)
        assert st == svp.DEV_BAD_SLOTS
        same(out, lse, every)
    for gr, ln in (([0, 4], [-5]), ([0, 4], [86]), ([0, 4], [2 ** 31 - 1]), ([0, 4], [-2 ** 31])):   # one group, not shared
        out, lse, st = run(gr=gr, ln=ln)
        assert st == svp.DEV_BAD_CONTEXT
        same(out, lse, every)
    for c, bit in (([100, -1, 85, 120], svp.DEV_BAD_CONTEXT), ([100, 10 ** 6, 85, 120], svp.DEV_BAD_CONTEXT)):
        out, lse, st = run(c=c)                                                             # one request is skipped
        assert st == bit and (out[2:4] == -7).all() and (lse[2:4] == -7).all()
        same(out, lse, [0, 1, 4, 5, 6, 7])
    out, lse, st = run(cu=[0, 1, 5, 6, 8], w=2)                                             # more rows than w
    assert st == svp.DEV_BAD_SLOTS and (out[1:5] == -7).all() and (out[[0, 5, 6, 7]] != -7).any(-1).all()


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("bad", [-1, 1 << 30, -2 ** 31])
def test_bad_pages_of_a_prefix_read_as_zeros(kind, bad):
    rows, ctx, groups, hq, hkv, d = [1, 2], [100, 120], [(0, 2, 96)], 4, 2, 128
    pool = Shared(rows, ctx, groups, hkv, d, 16, kind, seed=13)
    good = pool.table.clone()
    pool.table[:, 3] = bad
    cache = pool.cuda()
    q = torch.randn(3, hq, d, device="cuda").to(BF16)
    ws = svp.Workspace(svp.prefix_attn_workspace_size(hq, hkv, d, 3), zeroed=256)
    out, lse = svp.prefix_attn(q, i32(ctx), i32([0, 1, 3]), i32([0, 2]), i32([96]), cache=cache, ws=ws)
    assert ws.read_status() == svp.DEV_BAD_CONTEXT
    pool.table = good
    kept = [[pool.rows(w, i, 0, ctx[i] + rows[i]).copy() for i in range(2)] for w in range(2)]
    for per in kept:
        for z in per:
            z[48:64] = 0.0
    pool.rows = lambda which, i, lo, hi: kept[which][i][lo:hi]
    o, l, tol, ltol = attend_exact(pool, q, rows, ctx, 1 / math.sqrt(d))
    assert (np.abs(out.double().cpu().numpy() - o) <= tol).all()
    assert (np.abs(lse.double().cpu().numpy() - l) <= ltol).all()


def test_output_on_a_16_byte_boundary():
    rows, ctx, groups = [1, 30], [300, 270], [(0, 2, 256)]
    pool = Shared(rows, ctx, groups, 2, 128, 16, BF16, seed=26)
    cache = pool.cuda()
    q = torch.randn(31, 16, 128, device="cuda").to(BF16)
    args = (i32(ctx), i32(packed(rows)), i32([0, 2]), i32([256]))
    want, _ = svp.prefix_attn(q, *args, cache=cache)
    buf = torch.full((31 * 16 * 128 + 16,), -7.0, device="cuda", dtype=BF16)
    out = buf[8:-8].view(31, 16, 128)
    svp.prefix_attn(q, *args, cache=cache, out=out)
    assert torch.equal(out, want) and (buf[:8] == -7).all() and (buf[-8:] == -7).all()


def test_streams_and_graphs_at_once():
    rows, ctx, groups = [1] * 6, [3000 + 20 * i for i in range(6)], [(0, 4, 2992), (4, 6, 3072)]
    pool = Shared(rows, ctx, groups, 2, 128, 16, E4M3, seed=28)
    cache = pool.cuda()
    args = (i32(ctx), i32(packed(rows)), i32([0, 4, 6]), i32([2992, 3072]))
    qs = [torch.randn(6, 8, 128, device="cuda").to(BF16) for _ in range(2)]
    want = [svp.prefix_attn(q, *args, cache=cache, w=1) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(8):
        for s in streams:
            got.append(svp.prefix_attn(qs[0], *args, cache=cache, w=1, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want[0][0]) and torch.equal(b, want[0][1]) for a, b in got)
    graphs, outs = [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(svp.prefix_attn(q, *args, cache=cache, w=1))
        graphs.append(g)
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) for a, b in zip(outs, want))
    # lengths change on the device between replays
    args[3].copy_(i32([16, 3072]))
    args[0].copy_(i32([2990, 3000, 20, 3050, 3080, 3073]))
    for o in outs:
        o[0].zero_()
    graphs[0].replay()
    torch.cuda.synchronize()
    again = svp.prefix_attn(qs[0], *args, cache=cache, w=1)
    assert torch.equal(outs[0][0], again[0]) and torch.equal(outs[0][1], again[1])


def test_calls_of_growing_and_shrinking_rows_without_a_workspace():
    for m in (3, 900, 2):
        rows, ctx = [m, 1], [200, 210]
        pool = Shared(rows, ctx, [(0, 2, 192)], 2, 64, 16, BF16, seed=m)
        cache = pool.cuda()
        q = torch.randn(m + 1, 4, 64, device="cuda").to(BF16)
        out, lse = svp.prefix_attn(q, i32(ctx), i32(packed(rows)), i32([0, 2]), i32([192]), cache=cache)
        o, l, tol, ltol = attend_exact(pool, q, rows, ctx, 1 / 8, (0, 500))
        at = picked_rows(rows, (0, 500))
        assert (np.abs(out.double().cpu().numpy()[at] - o) <= tol).all()


def test_empty_calls_and_refusals():
    pool = Pool(2, [16, 16], 2, 64, 16, BF16)
    cache = pool.cuda()
    q = torch.zeros(0, 4, 64, device="cuda", dtype=BF16)
    out, lse = svp.prefix_attn(q, i32([0, 0]), i32([0, 0, 0]), i32([0, 2]), i32([16]), cache=cache)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    q = torch.ones(3, 4, 64, device="cuda", dtype=BF16)
    out = torch.full_like(q, -7)
    svp.prefix_attn(q, i32([]), i32([0]), i32([0, 0]), i32([16]), cache=cache, out=out)          # no request
    svp.prefix_attn(q, i32([5, 5]), i32([0, 0, 0]), i32([0, 2]), i32([0]), cache=cache, out=out)  # no rows
    assert (out == -7).all()
    c, cu = i32([1, 1]), i32([0, 1, 2])
    with pytest.raises(ValueError):
        svp.prefix_attn(q, c, cu, i32([]), i32([]), cache=cache)
    with pytest.raises(ValueError):
        svp.prefix_attn(q, c, cu, i32([0, 2]), i32([]), cache=cache)
    with pytest.raises(ValueError):
        svp.prefix_attn(q, c, cu, i32([0, 2]).long(), i32([0]), cache=cache)
    with pytest.raises(ValueError):
        svp.prefix_attn(q, c, cu, i32([0, 2]), i32([0]), cache=cache, out=out.float())
    with pytest.raises(ValueError):
        svp.prefix_attn(q[:, :3], c, cu, i32([0, 2]), i32([0]), cache=cache)
    with pytest.raises(svp.SvpError):
        svp.prefix_attn(q, c, cu, i32([0, 2]), i32([0]), cache=cache, ws=svp.Workspace(256))
