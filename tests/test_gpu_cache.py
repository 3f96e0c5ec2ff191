"""The paged cache's calls on the GPU: cache_write and cache_read bit for bit, chunk_attn
against softmax attention in 64 bits with error bounds from the roundings it makes.

A rounding to nearest is off by eps / 2 relative: bf16 2^-8, fp32 2^-24."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_packed_gb300 as svp

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


# ------------------------------------------------------------------ plain 64-bit forms
def e4m3_values(codes):
    """Values of e4m3 codes (uint8) in 64 bits, from the format: bias 7, 3 mantissa bits, the
    last code of each sign NaN."""
    c = codes.astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where(c & 127 == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def pack_rows(x):
    """(codes uint8, bytes uint8) of rows x [..., d] (64-bit): the smallest power of two that
    takes the largest magnitude to 448 or less, elements to the nearest code, ties to even."""
    fine = np.isfinite(x).all(-1)
    x = np.where(fine[..., None], x, 0.0)
    top = np.abs(x).max(-1)
    e = np.full(top.shape, -112, np.int64)
    for k in range(-112, 121):
        e = np.where(top > 448.0 * 2.0 ** (k - 1), np.maximum(k, -112), e)
    e = np.where(top <= 448.0 * 2.0 ** -112, -112, e)
    y = np.abs(x) / 2.0 ** e[..., None].astype(np.float64)
    p = np.maximum(np.frexp(y)[1] - 1, -6)
    v = np.round(y / 2.0 ** (p - 3.0)) * 2.0 ** (p - 3.0)
    grid = e4m3_values(np.arange(127, dtype=np.uint8))
    codes = np.searchsorted(grid, v).astype(np.uint8)
    assert (grid[codes] == v).all()
    codes = codes | (np.signbit(x).astype(np.uint8) << 7)
    codes = np.where(fine[..., None], codes, 0).astype(np.uint8)
    return codes, np.where(fine, e + 127, 255).astype(np.uint8)


class Pool:
    """Page pools of one cache on the CPU, with every position's 64-bit values beside them."""

    def __init__(self, n, lens, hkv, d, page, kind, layout="head", seed=0, spare=2, max_pages=None,
                 std=1.0, stale="nan"):
        g = torch.Generator().manual_seed(seed)
        need = [-(-x // page) for x in lens]
        self.n, self.lens, self.hkv, self.d, self.page, self.kind = n, lens, hkv, d, page, kind
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=g).tolist()
        cols = max_pages or max(need + [1])
        self.table = torch.full((n, cols), -1, dtype=torch.int32)
        for i in range(n):
            for b in range(need[i]):
                self.table[i, b] = order.pop()
        shape = (pages, hkv, page, d)
        vals = []
        for which in range(2):
            x = torch.randn(shape, generator=g, dtype=torch.float64) * std
            x = x.to(F32 if kind == F32 else BF16).double().numpy()
            vals.append(x)
        self.exps = [None, None]
        self.raw = []
        for which, x in enumerate(vals):
            if kind == E4M3:
                codes, b = pack_rows(x)
                self.raw.append(torch.from_numpy(codes))
                self.exps[which] = torch.from_numpy(b)
                vals[which] = e4m3_values(codes) * 2.0 ** (b.astype(np.float64) - 127)[..., None]
            else:
                self.raw.append(torch.from_numpy(x).to(kind))
        self.vals = vals
        if stale == "nan":        # positions that belong to no request
            used = torch.zeros(pages, page, dtype=torch.bool)
            for i in range(n):
                for t in range(lens[i]):
                    used[int(self.table[i, t // page]), t % page] = True
            hole = (~used)[:, None, :].expand(pages, hkv, page)
            for which in range(2):
                if kind == E4M3:
                    self.raw[which][hole] = 0x7f
                    self.exps[which][hole] = 255
                else:
                    self.raw[which][hole] = float("nan")
        self.layout = layout

    def cuda(self):
        pools = []
        for x in self.raw:
            x = x.cuda()
            x = x.view(E4M3) if self.kind == E4M3 else x
            if self.layout == "token":   # [pages, page, hkv, d] storage
                x = x.transpose(1, 2).contiguous().transpose(1, 2)
            pools.append(x)
        self.dev_table = self.table.cuda()
        self.dev_exps = [None if e is None else e.cuda() for e in self.exps]
        self.dev = pools
        return svp.make_cache(pools[0], pools[1], self.dev_table, k_exp=self.dev_exps[0], v_exp=self.dev_exps[1])

    def rows(self, which, i, lo, hi):
        """64-bit values [hi - lo, hkv, d] of request i's positions."""
        pos = np.arange(lo, hi)
        return self.vals[which][self.table[i].numpy()[pos // self.page], :, pos % self.page]


def bytes_of(t):
    return t.cpu().contiguous().view(torch.uint8)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def packed(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(int).tolist()


# ------------------------------------------------------------------ write
def special_rows(d, kind):
    """Rows at the quantisation's borders."""
    rows = [torch.zeros(d), torch.full((d,), -0.0), torch.full((d,), 448.0), torch.full((d,), 450.0)]
    r = torch.linspace(-448, 448, d); rows.append(r)
    rows.append(r * 2.0 ** -20)
    rows.append(torch.where(torch.arange(d) == 5, torch.tensor(3.3e38), torch.tensor(1.0)))
    rows.append(torch.where(torch.arange(d) == 7, torch.tensor(float("nan")), torch.tensor(1.0)))
    rows.append(torch.where(torch.arange(d) == d - 1, torch.tensor(-float("inf")), torch.tensor(1.0)))
    rows.append(torch.full((d,), 1e-38))
    rows.append(torch.where(torch.arange(d) % 2 == 0, torch.tensor(448.0), torch.tensor(0.0009765625)))
    ties = torch.tensor([1.0, 1.0625, 1.1875, 1.3125, 1.9375, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 448.0])
    rows.append(ties.repeat(d // 10 + 1)[:d])
    return torch.stack(rows).to(kind)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", [BF16, F32])
def test_write_8_bit_rows_at_the_borders(d, kind):
    x = special_rows(d, kind)
    m, hkv = x.shape[0], 2
    k = torch.stack([x, x.flip(0)], 1).cuda()
    v = torch.stack([x.flip(0), -x], 1).cuda()
    pool = Pool(1, [m], hkv, d, 16, E4M3, stale="keep")
    cache = pool.cuda()
    ws = svp.Workspace(256)
    svp.cache_write(k, v, i32([0]), i32([0, m]), cache=cache, ws=ws)
    assert ws.read_status() == 0
    for which, src in ((0, k), (1, v)):
        codes, b = pack_rows(src.double().cpu().numpy())
        pos = np.arange(m)
        pg = pool.table[0].numpy()[pos // 16]
        got = bytes_of(pool.dev[which]).numpy()[pg, :, pos % 16]
        gb = pool.dev_exps[which].cpu().numpy()[pg, :, pos % 16]
        assert (gb == b).all()
        assert (got == codes).all()


@pytest.mark.parametrize("rows,ctx,page", [
    ([1], [0], 16), ([1, 1, 1], [15, 16, 17], 16), ([5, 0, 37, 1, 16], [0, 9, 100, 63, 1], 32),
    ([300, 2, 0, 129], [7, 127, 0, 500], 128), ([1] * 300, [3] * 300, 64), ([4000], [11], 16)])
@pytest.mark.parametrize("new,kind", [(BF16, BF16), (F32, F32), (BF16, E4M3), (F32, E4M3), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("layout", ["head", "token"])
def test_write_places_and_leaves_the_rest(rows, ctx, page, new, kind, layout):
    n, hkv, d = len(rows), 3, 64
    lens = [c + r for c, r in zip(ctx, rows)]
    pool = Pool(n, lens, hkv, d, page, kind, layout, seed=3)
    cache = pool.cuda()
    cu = packed(rows)
    g = torch.Generator().manual_seed(1)
    hq, pad = 6, 5
    qkv = torch.randn(cu[-1] + pad, hq + 2 * hkv, d, generator=g).to(new).cuda()   # a fused projection
    k, v = qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    take = [max(0, r - 1 - i % 3) if i % 2 else r + i for i, r in enumerate(rows)]
    for tk in (None, i32(take)):
        for x, e, raw, ex in zip(pool.dev, pool.dev_exps, pool.raw, pool.exps):
            x.view(torch.uint8).copy_(raw.contiguous().view(torch.uint8).cuda() if kind == E4M3 else raw.view(torch.uint8).cuda())
            if e is not None:
                e.copy_(ex)
        ws = svp.Workspace(256)
        svp.cache_write(k, v, i32(ctx), i32(cu), cache=cache, take=tk, ws=ws)
        assert ws.read_status() == 0
        for which, src in ((0, k), (1, v)):
            want, want_e = pool.raw[which].clone(), None if kind != E4M3 else pool.exps[which].clone()
            s = src.cpu()
            for i in range(n):
                r = rows[i] if tk is None else min(rows[i], max(take[i], 0))
                pos = np.arange(ctx[i], ctx[i] + r)
                pg, tok = pool.table[i][pos // page].long(), torch.from_numpy(pos % page)
                if kind == E4M3:
                    codes, b = pack_rows(s[cu[i]:cu[i] + r].double().numpy())
                    want[pg, :, tok] = torch.from_numpy(codes)
                    want_e[pg, :, tok] = torch.from_numpy(b)
                else:
                    want[pg, :, tok] = s[cu[i]:cu[i] + r].to(kind)
            assert torch.equal(bytes_of(pool.dev[which]), want.view(torch.uint8))
            if want_e is not None:
                assert torch.equal(pool.dev_exps[which].cpu(), want_e)


# ------------------------------------------------------------------ read
@pytest.mark.parametrize("kind", [BF16, F32, E4M3])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("rows,start,page,d", [
    ([1], [0], 16, 128), ([3, 0, 40, 1], [13, 0, 5, 127], 16, 64), ([700, 65], [0, 63], 64, 256),
    ([2500], [9], 128, 64), ([1] * 280, [2] * 280, 32, 64)])
def test_read_back(kind, out, rows, start, page, d):
    n, hkv = len(rows), 2
    pool = Pool(n, [a + b for a, b in zip(rows, start)], hkv, d, page, kind, "token", seed=5)
    cache = pool.cuda()
    cu = packed(rows)
    ks = torch.full((cu[-1] + 3, hkv, d), -7.0, dtype=out, device="cuda")
    vs = torch.full_like(ks, -7.0)
    ws = svp.Workspace(256)
    svp.cache_read(i32(start), i32(cu), cache=cache, k_out=ks, v_out=vs, ws=ws)
    assert ws.read_status() == 0
    for which, got in ((0, ks), (1, vs)):
        want = np.concatenate([pool.rows(which, i, start[i], start[i] + rows[i]) for i in range(n)])
        assert torch.equal(got[:cu[-1]].cpu(), torch.from_numpy(want).to(out))    # one rounding at most, exact for 8 bits
        assert (got[cu[-1]:] == -7.0).all()


def test_read_every_code_and_byte():
    """All 256 codes under every exponent byte the write makes, and the NaN row."""
    d, page = 256, 16
    bytes_ = list(range(15, 248)) + [255]
    pages = -(-len(bytes_) // page)
    raw = torch.arange(256, dtype=torch.uint8).expand(pages, 1, page, 256).contiguous()
    exps = torch.full((pages, 1, page), 255, dtype=torch.uint8)
    for t, b in enumerate(bytes_):
        exps[t // page, 0, t % page] = b
    dev = raw.cuda().view(E4M3)
    cache = svp.make_cache(dev, dev.clone(), torch.arange(pages, dtype=torch.int32)[None].cuda(),
                           k_exp=exps.cuda(), v_exp=exps.cuda())
    k, _ = svp.cache_read(None, i32([0, len(bytes_)]), cache=cache, rows=len(bytes_), dtype=F32)
    k = k.cpu().double().numpy()[:, 0]
    assert np.isnan(k[-1]).all()
    vals = e4m3_values(np.arange(256, dtype=np.uint8))
    want = vals[None] * 2.0 ** (np.array(bytes_[:-1], np.float64) - 127)[:, None]
    with np.errstate(over="ignore"):
        want = want.astype(np.float32)
    assert np.array_equal(k[:-1].astype(np.float32), want, equal_nan=True)


# ------------------------------------------------------------------ attention
def attend_exact(pool, q, rows, ctx, scale, picks=None):
    """(o, lse, bound) in 64 bits for the picked packed rows: bound is the largest error that
    the kernel's roundings allow.  A = sum p |v| / l;  each probability is off by half a bf16
    step (0 in fp32) and by the error of its score: fp32 sums of d products, d * 2^-23 relative
    to sum |q k|, and a few steps more in exp and in the sums over the keys."""
    hq, d = q.shape[1:]
    G = hq // pool.hkv
    half = 2.0 ** -24 if pool.kind == F32 else 2.0 ** -8
    o, lse, tol, ltol = [], [], [], []
    first = 0
    for i, r in enumerate(rows):
        take = range(r) if picks is None else sorted({j for j in picks if j < r} | {r - 1} if r else set())
        if len(take):
            K, V = pool.rows(0, i, 0, ctx[i] + r), pool.rows(1, i, 0, ctx[i] + r)
            x = q[first:first + r].double().cpu().numpy()
        for j in take:
            T = ctx[i] + j + 1
            for h in range(hq):
                k, v = K[:T, h // G], V[:T, h // G]
                s = k @ x[j, h] * scale
                ds = (d + 2) * 2.0 ** -23 * (np.abs(k) @ np.abs(x[j, h])).max() * scale
                top = s.max()
                p = np.exp(s - top)
                l = p.sum()
                y = p @ v / l
                A = p @ np.abs(v) / l
                rel = (0 if pool.kind == F32 else half) + 2 * ds + (T / 32 + 64) * 2.0 ** -23
                o.append(y)
                tol.append(rel * A + half * np.abs(y) + 1e-30)
                lse.append(top + np.log(l))
                ltol.append(ds + (T / 32 + 64) * 2.0 ** -23 + abs(lse[-1]) * 2.0 ** -22)
        first += r
    shape = (-1, hq, d)
    return (np.array(o).reshape(shape), np.array(lse).reshape(-1, hq), np.array(tol).reshape(shape),
            np.array(ltol).reshape(-1, hq))


def picked_rows(rows, picks):
    out, first = [], 0
    for r in rows:
        take = range(r) if picks is None else sorted({j for j in picks if j < r} | {r - 1} if r else set())
        out += [first + j for j in take]
        first += r
    return out


def check_attend(rows, ctx, *, hq=4, hkv=2, d=128, page=16, kind=BF16, layout="head", picks=None, seed=0,
                 std=1.0, scale=0.0, w=None, pad=3, fused=False, ws=None, stream=None):
    n = len(rows)
    pool = Pool(n, [a + b for a, b in zip(rows, ctx)], hkv, d, page, kind, layout, seed=seed, std=std)
    cache = pool.cuda()
    cu = packed(rows)
    g = torch.Generator().manual_seed(seed + 1)
    qt = F32 if kind == F32 else BF16
    wide = torch.randn(cu[-1] + pad, hq + (2 * hkv if fused else 0), d, generator=g).to(qt).cuda()
    q = wide[:, :hq]
    out = torch.full((cu[-1] + pad, hq, d), -7.0, dtype=qt, device="cuda")
    lse = torch.full((cu[-1] + pad, hq), -7.0, device="cuda")
    own = ws is None
    ws = ws or svp.Workspace(svp.chunk_attn_workspace_size(hq, hkv, d, qt))
    svp.chunk_attn(q, i32(ctx), i32(cu), cache=cache, w=w or max(rows + [1]), out=out, lse=lse, scale=scale, ws=ws)
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


ATTEND = [
    ([1], [0]), ([1], [1]), ([1, 1], [127, 128]), ([1, 1, 1], [126, 500, 2000]),
    ([2, 0, 7, 1], [15, 40, 122, 255]), ([16, 3], [1000, 0]), ([33, 64, 1], [3, 300, 777]),
    ([130], [0]), ([257, 5, 128], [10, 0, 129]), ([0, 0, 1], [0, 5, 63])]


@pytest.mark.parametrize("kind", [BF16, E4M3, F32])
@pytest.mark.parametrize("rows,ctx", ATTEND)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_lengths(rows, ctx, d, kind):
    check_attend(rows, ctx, d=d, kind=kind, picks=(0, 1, 31, 32, 63, 64, 127, 128, 200))


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (12, 1), (24, 2), (8, 8), (128, 1), (5, 1), (48, 3)])
def test_attend_head_layouts(hq, hkv, kind):
    check_attend([1, 9, 70], [300, 130, 17], hq=hq, hkv=hkv, kind=kind, page=32, picks=(0, 8, 33), fused=True, seed=4)


@pytest.mark.parametrize("kind", [BF16, E4M3, F32])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("layout", ["head", "token"])
def test_attend_pages_and_strides(page, layout, kind):
    check_attend([1, 20, 7], [211, 0, 1100], page=page, layout=layout, kind=kind, fused=True, seed=7)


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_long_split_contexts(d, kind):
    """One and two requests whose keys are split over many blocks and joined."""
    check_attend([1], [9001], hq=2, hkv=1, d=d, kind=kind, seed=8)
    check_attend([5, 1], [6000, 4095], hq=6, hkv=2, d=d, kind=kind, seed=9, std=2.0)


@pytest.mark.parametrize("kind", [BF16, E4M3])
def test_attend_scores_that_grow(kind):
    """Scores far apart (a wide softmax scale): the running reference has to move."""
    check_attend([3, 40], [700, 900], kind=kind, scale=2.0, std=4.0, seed=10, picks=(0, 1, 39))


@pytest.mark.parametrize("kind", [BF16, E4M3])
def test_attend_many_requests(kind):
    rows = [i % 4 for i in range(300)]
    check_attend(rows, [(37 * i) % 190 for i in range(300)], hq=2, hkv=1, d=64, kind=kind, seed=11)


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_the_most_requests(d, kind):
    """1024 requests, most of them empty, among them rows of several query tiles."""
    rows, ctx = [0] * 1024, [0] * 1024
    for i, (r, c) in {3: (1, 40), 500: (150, 60), 900: (2, 129), 1023: (70, 1)}.items():
        rows[i], ctx[i] = r, c
    check_attend(rows, ctx, hq=4, hkv=1, d=d, kind=kind, seed=19, picks=(0, 1, 69, 149))


def test_one_workspace_serves_any_size_twice():
    ws = svp.Workspace(svp.chunk_attn_workspace_size(8, 2, 128))
    for rows, ctx in (([1], [5000]), ([200, 1], [100, 3000]), ([1], [5000]), ([3] * 40, [257] * 40)):
        check_attend(rows, ctx, hq=8, hkv=2, ws=ws, picks=(0, 1, 100))


@pytest.mark.parametrize("kind", [BF16, E4M3])
def test_same_inputs_give_the_same_bits(kind):
    pool = Pool(3, [4001, 700, 260], 2, 128, 16, kind, seed=12)
    cache = pool.cuda()
    q = torch.randn(132, 8, 128, device="cuda").to(BF16)
    cu, ctx = i32([0, 1, 130, 131]), i32([4000, 571, 259])
    first = svp.chunk_attn(q, ctx, cu, cache=cache)
    for _ in range(5):
        again = svp.chunk_attn(q, ctx, cu, cache=cache)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


# ------------------------------------------------------------------ errors on the device
def test_bad_requests_are_skipped():
    pool = Pool(3, [40, 40, 40], 2, 64, 16, BF16, stale="keep")
    cache = pool.cuda()
    k = torch.ones(12, 2, 64, device="cuda", dtype=BF16)
    q = torch.ones(12, 4, 64, device="cuda", dtype=BF16)
    size = svp.chunk_attn_workspace_size(4, 2, 64)
    for cu, ctx, bit, skipped in (
            ([0, 4, 2, 6], [30, 30, 30], svp.DEV_BAD_SLOTS, [1]),          # runs backwards
            ([0, 4, 8, 13], [30, 30, 30], svp.DEV_BAD_SLOTS, [2]),         # leaves the buffer
            ([0, 4, 8, 12], [30, -1, 30], svp.DEV_BAD_CONTEXT, [1]),
            ([0, 4, 8, 12], [30, 30, 45], svp.DEV_BAD_CONTEXT, [2])):      # past the block table
        ws, wa = svp.Workspace(256), svp.Workspace(size)
        before = [x.clone() for x in pool.dev]
        svp.cache_write(k, k, i32(ctx), i32(cu), cache=cache, ws=ws)
        assert ws.read_status() == bit
        for i in skipped:
            for x, y in zip(pool.dev, before):
                pg = pool.table[i].long().cuda()
                assert torch.equal(x[pg], y[pg])
        out = torch.full((12, 4, 64), -7.0, device="cuda", dtype=BF16)
        svp.chunk_attn(q, i32(ctx), i32(cu), cache=cache, w=8, out=out, ws=wa)
        assert wa.read_status() == bit
        own = {r for i in range(3) if i not in skipped for r in range(cu[i], cu[i + 1])}
        for r in range(12):
            assert bool((out[r] == -7).all()) == (r not in own)
    # more rows than w
    wa = svp.Workspace(size)
    out = torch.full((12, 4, 64), -7.0, device="cuda", dtype=BF16)
    svp.chunk_attn(q, i32([30, 30, 30]), i32([0, 4, 9, 12]), cache=cache, w=4, out=out, ws=wa)
    assert wa.read_status() == svp.DEV_BAD_SLOTS
    assert (out[4:9] == -7).all() and (out[:4] != -7).any() and (out[9:] != -7).any()


@pytest.mark.parametrize("kind", [BF16, E4M3, F32])
@pytest.mark.parametrize("bad", [-1, 1 << 30])
def test_bad_pages_read_as_zeros_and_are_not_written(kind, bad):
    rows, ctx, hq, hkv, d = [2], [100], 4, 2, 128
    pool = Pool(1, [102], hkv, d, 16, kind, seed=13)
    pool.table[0, 3] = bad
    cache = pool.cuda()
    qt = F32 if kind == F32 else BF16
    q = torch.randn(2, hq, d, device="cuda").to(qt)
    wa = svp.Workspace(svp.chunk_attn_workspace_size(hq, hkv, d, qt))
    out, lse = svp.chunk_attn(q, i32(ctx), i32([0, 2]), cache=cache, ws=wa)
    assert wa.read_status() == svp.DEV_BAD_CONTEXT
    hole = np.arange(48, 64)
    table = pool.table.clone()
    table[0, 3] = 0
    pool.table = table
    zero = [pool.rows(w, 0, 0, 102).copy() for w in range(2)]
    for z in zero:
        z[hole] = 0.0
    pool.rows = lambda which, i, lo, hi: zero[which][lo:hi]
    o, l, tol, ltol = attend_exact(pool, q, rows, ctx, 1 / math.sqrt(d))
    assert (np.abs(out.double().cpu().numpy() - o) <= tol).all()
    assert (np.abs(lse.double().cpu().numpy() - l) <= ltol).all()
    # the write and the read skip rows on such a page
    before = [bytes_of(x) for x in pool.dev]
    ws = svp.Workspace(256)
    x = torch.ones(3, hkv, d, device="cuda", dtype=qt)
    svp.cache_write(x, x, i32([50]), i32([0, 3]), cache=cache, ws=ws)
    assert ws.read_status() == svp.DEV_BAD_CONTEXT
    assert all(torch.equal(bytes_of(x), y) for x, y in zip(pool.dev, before))
    ko, vo = (torch.full((102, hkv, d), -7.0, device="cuda", dtype=qt) for _ in range(2))
    svp.cache_read(None, i32([0, 102]), cache=cache, k_out=ko, v_out=vo, ws=ws)
    assert ws.read_status() == svp.DEV_BAD_CONTEXT
    assert (ko[48:64] == -7).all() and (ko[:48] != -7).any() and (ko[64:] != -7).any()


def test_nan_rows_reach_the_rows_that_see_them():
    for kind in (BF16, E4M3):
        pool = Pool(2, [300, 300], 2, 128, 16, kind, seed=14)
        cache = pool.cuda()
        k = torch.randn(2, 2, 128, device="cuda").to(BF16)
        k[0, 1, 5] = float("nan")
        svp.cache_write(k, k, i32([200, 200]), i32([0, 1, 2]), cache=cache)
        q = torch.randn(4, 4, 128, device="cuda").to(BF16)
        out, lse = svp.chunk_attn(q, i32([298, 298]), i32([0, 2, 4]), cache=cache)
        assert torch.isnan(out[:2, 2:]).all() and torch.isnan(lse[:2, 2:]).all()
        assert torch.isfinite(out[:2, :2]).all() and torch.isfinite(out[2:]).all()
        early, _ = svp.chunk_attn(q, i32([126, 298]), i32([0, 2, 4]), cache=cache)   # position 200 is not seen
        assert torch.isfinite(early).all()


@pytest.mark.parametrize("kind", [BF16, E4M3, F32])
@pytest.mark.parametrize("rows,ctx", [(3, 200), (50, 100), (130, 130)])
def test_a_nan_key_that_only_the_last_row_sees(rows, ctx, kind):
    hq, hkv, d = 4, 2, 128
    pool = Pool(1, [ctx + rows], hkv, d, 16, kind, seed=34)
    cache = pool.cuda()
    qt = F32 if kind == F32 else BF16
    x = torch.full((1, hkv, d), float("nan"), device="cuda", dtype=qt)
    q = torch.randn(rows, hq, d, generator=torch.Generator().manual_seed(35)).to(qt).cuda()
    last = ctx + rows - 1
    v = torch.from_numpy(pool.rows(1, 0, last, last + 1)).to(qt).cuda()
    svp.cache_write(x, v, i32([last]), i32([0, 1]), cache=cache)
    out, lse = svp.chunk_attn(q, i32([ctx]), i32([0, rows]), cache=cache)
    assert torch.isnan(out[-1]).all() and torch.isnan(lse[-1]).all()
    o, l, tol, ltol = attend_exact(pool, q[:-1], [rows - 1], [ctx], 1 / math.sqrt(d), picks=(0, 1, 31, 32, 48, 100))
    at = picked_rows([rows - 1], (0, 1, 31, 32, 48, 100))
    assert (np.abs(out.double().cpu().numpy()[at] - o) <= tol).all()
    assert (np.abs(lse.double().cpu().numpy()[at] - l) <= ltol).all()


# ------------------------------------------------------------------ as they are used
@pytest.mark.parametrize("kind", [BF16, E4M3])
def test_a_generation_step_captured_and_replayed(kind):
    """Prompt chunks, then steps of write -> attend -> accept -> commit, one of them a graph that
    is replayed while lengths change on the device; against the same steps run eagerly, and the
    cache's contents against a verification over the rows read back."""
    n, hq, hkv, d, w, page, vocab = 3, 8, 2, 128, 6, 16, 64
    g = torch.Generator(device="cuda").manual_seed(15)
    prompt = [150, 33, 1]
    cap = [p + 8 * w for p in prompt]

    def fresh():
        return Pool(n, cap, hkv, d, page, kind, seed=16)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(BF16)

    cu_p = packed(prompt)
    pq, pk, pv = randn(cu_p[-1], hq, d), randn(cu_p[-1], hkv, d), randn(cu_p[-1], hkv, d)
    cu_w = i32(packed([w] * n))
    steps = [(randn(n * w, hq, d), randn(n * w, hkv, d), randn(n * w, hkv, d), randn(n * w, vocab),
              torch.randint(0, vocab, (n * w,), generator=g, device="cuda", dtype=torch.int32)) for _ in range(4)]
    for s in steps:     # make most drafts match
        top = s[3].float().argmax(-1).int()
        keep = torch.rand(n * w, generator=g, device="cuda") < 0.7
        s[4][1:] = torch.where(keep[1:], top[:-1], s[4][1:])

    def run(captured):
        pool = fresh()
        cache = pool.cuda()
        ctx = i32([0] * n)
        svp.cache_write(pk, pv, ctx, i32(cu_p), cache=cache)
        outs = [svp.chunk_attn(pq, ctx, i32(cu_p), cache=cache)[0].clone()]
        ctx += i32(prompt)
        bufs = [t.clone() for t in steps[0]]
        out = torch.zeros(n * w, hq, d, dtype=BF16, device="cuda")
        lse = torch.zeros(n * w, hq, device="cuda")
        acc, nxt = i32([0] * n), i32([0] * n)

        def step():
            q, k, v, logits, tokens = bufs
            svp.cache_write(k, v, ctx, cu_w, cache=cache)
            svp.chunk_attn(q, ctx, cu_w, cache=cache, w=w, out=out, lse=lse)
            top = svp.draft_margin(logits)[0]
            svp.greedy_accept(top, tokens, cu_w, outs=(acc, nxt))
            ctx.add_(acc)

        graph = None
        if captured:
            keep = ctx.clone()
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                step()
            side.synchronize()
            ctx.copy_(keep)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            ctx.copy_(keep)
        for s in steps:
            for b, x in zip(bufs, s):
                b.copy_(x)
            graph.replay() if graph else step()
            outs += [out.clone(), lse.clone(), acc.clone(), ctx.clone()]
        torch.cuda.synchronize()
        return pool, cache, outs

    pool, cache, eager = run(False)
    _, _, replayed = run(True)
    assert all(torch.equal(a, b) for a, b in zip(eager, replayed))
    # the last step again as a verification over the committed context read back to rows
    ctx = eager[-1] - eager[-2]
    lens = ctx.tolist()
    cu_c = packed(lens)
    kc, vc = svp.cache_read(None, i32(cu_c), cache=cache, rows=cu_c[-1])
    q, k, v = steps[-1][:3]
    kr, vr = svp.cache_read(ctx, cu_w, cache=cache, rows=n * w)     # the candidates as the cache holds them
    if kind == BF16:
        assert torch.equal(kr, k) and torch.equal(vr, v)
    ref, rl = svp.verify_attn_packed(q, kr, vr, ctx, cu_w, w=w, k_ctx=kc, v_ctx=vc,
                                     cu_ctx=torch.tensor(cu_c, dtype=torch.int64, device="cuda"))
    # two kernels over the same values: each probability and each output is off by half a bf16 step in both
    size = float(vc.float().abs().max())
    assert (ref.float() - eager[-4].float()).abs().max() <= 4 * 2.0 ** -8 * size
    assert (rl - eager[-3]).abs().max() <= 2.0 ** -8 + 1e-4


def test_committing_accepted_rows_only():
    """verify_attn_packed over the cache, then the accepted prefix goes into it."""
    n, hkv, d, w = 4, 2, 128, 5
    pool = Pool(n, [64] * n, hkv, d, 16, BF16, seed=17)
    cache = pool.cuda()
    k, v = torch.randn(n * w, hkv, d, device="cuda").to(BF16), torch.randn(n * w, hkv, d, device="cuda").to(BF16)
    ctx, cu, acc = [20, 0, 31, 47], packed([w] * n), [1, 5, 3, 0]
    before = [x.clone() for x in pool.dev]
    svp.cache_write(k, v, i32(ctx), i32(cu), cache=cache, take=i32(acc))
    for x, y, src in zip(pool.dev, before, (k, v)):
        for i in range(n):
            for t in range(64):
                pg = int(pool.table[i, t // 16])
                want = src[cu[i] + t - ctx[i]] if 0 <= t - ctx[i] < acc[i] else y[pg, :, t % 16]
                assert torch.equal(x[pg, :, t % 16].view(torch.int16), want.view(torch.int16))


def test_two_streams_at_once_and_own_workspaces():
    pool = Pool(2, [3000, 2500], 2, 128, 16, BF16, seed=18)
    cache = pool.cuda()
    q = torch.randn(2, 8, 128, device="cuda").to(BF16)
    ctx, cu = i32([2999, 2499]), i32([0, 1, 2])
    want = svp.chunk_attn(q, ctx, cu, cache=cache)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(svp.chunk_attn(q, ctx, cu, cache=cache))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want[0]) and torch.equal(b, want[1]) for a, b in got)


def test_empty_calls():
    pool = Pool(1, [16], 2, 64, 16, BF16)
    cache = pool.cuda()
    q = torch.zeros(0, 4, 64, device="cuda", dtype=BF16)
    out, lse = svp.chunk_attn(q, i32([0]), i32([0, 0]), cache=cache)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    svp.cache_write(q[:, :2], q[:, :2], i32([0]), i32([0, 0]), cache=cache)
    k, v = svp.cache_read(None, i32([0, 0]), cache=cache, rows=0)
    assert k.shape == (0, 2, 64)
    q = torch.ones(3, 4, 64, device="cuda", dtype=BF16)
    out = torch.full_like(q, -7)
    svp.chunk_attn(q, i32([]), i32([0]), cache=cache, out=out)       # no request
    assert (out == -7).all()


# ------------------------------------------------------------------ borders of the attention's kernels
@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,rows", [(2, 2, 16), (2, 2, 17), (4, 2, 8), (4, 2, 9), (16, 1, 1), (17, 1, 1),
                                         (8, 1, 1), (9, 1, 1), (3, 1, 3)])
def test_attend_rows_around_the_short_kernel(hq, hkv, rows, d, kind):
    """16 query rows of a KV head and one more, 8 and one more; requests of fewer rows among them."""
    check_attend([rows, 1, rows, 0, max(1, rows - 1)], [700, 40, 0, 9, 255], hq=hq, hkv=hkv, d=d, kind=kind, seed=21)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("w", [1, 20])
def test_every_code_and_exponent_through_one_key(d, w):
    """A row that sees one key gets its value row, bit for bit: the probability is 1 (2^y with |y| below
    2^-12, which fp16 rounds to 1 and which moves a code's 4 bits of mantissa by no bf16 step)."""
    few = w == 1 and d < 256          # the kernel for few rows holds every byte that is written, the other 2^-60 up
    parts = 256 // d
    cases = [(b, x) for b in range(15 if few else 67, 247) for x in range(parts)]
    n, page = len(cases), 16
    codes = torch.zeros(n, 1, page, d, dtype=torch.uint8)
    exps = torch.full((n, 1, page), 127, dtype=torch.uint8)
    for i, (b, x) in enumerate(cases):
        row = torch.arange(x * d, (x + 1) * d, dtype=torch.uint8)
        codes[i, 0, 0] = torch.where((row & 127) == 127, torch.zeros_like(row), row)
        exps[i, 0, 0] = b
    kc = torch.randint(0, 120, codes.shape, generator=torch.Generator().manual_seed(22)).to(torch.uint8)
    ke = torch.full_like(exps, 119)
    cache = svp.make_cache(kc.cuda().view(E4M3), codes.cuda().view(E4M3),
                           torch.arange(n, dtype=torch.int32)[:, None].cuda(), k_exp=ke.cuda(), v_exp=exps.cuda())
    q = torch.randn(n, 1, d, generator=torch.Generator().manual_seed(23)).to(BF16).cuda()
    out, _ = svp.chunk_attn(q, i32([0] * n), i32(list(range(n + 1))), cache=cache, w=w)
    want = e4m3_values(codes[:, 0, 0].numpy()) * 2.0 ** (exps[:, 0, 0].numpy().astype(np.float64) - 127)[:, None]
    assert (out[:, 0].double().cpu().numpy() == want).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 40])
def test_rows_of_very_different_sizes_in_one_tile(d, rows):
    """Value rows 2^24 apart and key rows 2^6 apart, position by position.  An element is held to 2^-25 of
    its tile's largest power of two 2^E, which the bound adds: 2^-24 2^E for V, and for a score 2^-24 2^E
    of K times the sum of |q|."""
    ctx, hq, hkv, page = 500, 4, 2, 16
    T = ctx + rows
    pool = Pool(1, [T], hkv, d, page, E4M3, seed=24)
    g = torch.Generator().manual_seed(25)
    for which, lo, hi in ((0, 116, 123), (1, 107, 132)):
        e = torch.randint(lo, hi, pool.exps[which].shape, generator=g).to(torch.uint8)
        live = pool.exps[which] != 255
        pool.exps[which] = torch.where(live, e, pool.exps[which])
        pool.vals[which] = e4m3_values(pool.raw[which].numpy()) * 2.0 ** (pool.exps[which].double().numpy() - 127)[..., None]
    cache = pool.cuda()
    q = torch.randn(rows, hq, d, generator=g).to(BF16).cuda() * 2.0 ** -6
    out, lse = svp.chunk_attn(q, i32([ctx]), i32([0, rows]), cache=cache)
    scale = 1 / math.sqrt(d)
    o, l, tol, ltol = attend_exact(pool, q, [rows], [ctx], scale)
    dsum = q.double().abs().sum(-1).cpu().numpy() * scale * 2.0 ** -24 * 2.0 ** -5     # score: K's E is 2^(122 - 127)
    big = np.abs(pool.vals[1][np.isfinite(pool.vals[1])]).max()
    extra = 2.0 ** -24 * 2.0 ** 4 + 2 * dsum[..., None] * big
    assert (np.abs(out.double().cpu().numpy() - o) <= tol + extra).all()
    assert (np.abs(lse.double().cpu().numpy() - l) <= ltol + dsum).all()


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("rows", [1, 40, 140])
def test_scores_that_jump_between_tiles(rows, kind):
    """Keys 40, 120 and 416 above the others in score (2^600 in probability) in later tiles, in either
    half of one, and a first tile at -416: more heads than CTAs, so that most see all tiles in one piece."""
    d, hkv, ctx, page = 64, 200, 900, 64
    pool = Pool(1, [ctx + rows], hkv, d, page, kind, seed=32)
    at = {t: -416.0 for t in range(128)} | {300: 40.0, 470: 120.0, 660: 416.0}
    for t, x in at.items():
        row = np.zeros(d)
        row[0] = x                        # (bf16 and e4m3 values)
        pg = int(pool.table[0, t // page])
        pool.vals[0][pg, :, t % page] = row
        codes, b = pack_rows(row)
        if kind == E4M3:
            pool.raw[0][pg, :, t % page] = torch.from_numpy(codes)
            pool.exps[0][pg, :, t % page] = int(b)
        else:
            pool.raw[0][pg, :, t % page] = torch.from_numpy(row).to(BF16)
    for upto in (300, 470, 660, ctx):     # the last jump that is seen
        q = torch.randn(rows, hkv, d, generator=torch.Generator().manual_seed(33)).to(BF16)
        q[..., 0] = 8.0                   # the scale is 1 / 8
        q = q.cuda()
        ws = svp.Workspace(svp.chunk_attn_workspace_size(hkv, hkv, d))
        cache = pool.cuda()
        out, lse = svp.chunk_attn(q, i32([upto]), i32([0, rows]), cache=cache, ws=ws)
        assert ws.read_status() == 0
        picks = (0, 39, 100)
        o, l, tol, ltol = attend_exact(pool, q, [rows], [upto], 1 / math.sqrt(d), picks)
        r = picked_rows([rows], picks)
        assert (np.abs(out.double().cpu().numpy()[r] - o) <= tol).all()
        assert (np.abs(lse.double().cpu().numpy()[r] - l) <= ltol).all()


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("rows", [1, 40])
def test_a_tail_under_one_large_score(rows, kind):
    """The first key is 2^26 times as probable as each of the others and its value is zero: what comes
    out is the others'.  A probability over 8-bit pages is off by 2^-11 relative, or below 2^-21 of the
    largest by 2^-32 of it, here 2^-6 of the others' own; over bf16 pages by 2^-8.  More heads than
    CTAs, so that most of them see all their keys in one piece."""
    T, d, page, hkv, hq = 3000, 64, 128, 304, 608
    pages = -(-T // page)
    g = torch.Generator(device="cuda").manual_seed(31)
    k = torch.zeros(pages, hkv, page, d, device="cuda", dtype=BF16)
    v = torch.randint(1, 4, (pages, hkv, page, d), device="cuda", generator=g).to(BF16)
    k[0, :, 0, 0] = 26.0                  # (an e4m3 value)
    v[0, :, 0] = 0
    table = torch.arange(pages, device="cuda", dtype=torch.int32)[None].contiguous()
    if kind == E4M3:
        exps = torch.full((pages, hkv, page), 127, dtype=torch.uint8, device="cuda")
        cache = svp.make_cache(k.to(E4M3), v.to(E4M3), table, k_exp=exps, v_exp=exps.clone())
    else:
        cache = svp.make_cache(k, v, table)
    q = torch.zeros(rows, hq, d, device="cuda", dtype=BF16)
    q[..., 0] = 1.0                       # with this scale, a score of 26 is a factor of 2^26
    out, lse = svp.chunk_attn(q, i32([T - rows]), i32([0, rows]), cache=cache, scale=math.log(2.0))
    values = v.double().transpose(0, 1).reshape(hkv, pages * page, d)
    for j in sorted({0, rows - 1}):
        n = T - rows + j + 1
        l = 1.0 + (n - 1) * 2.0 ** -26
        y = (values[:, 1:n].sum(1) * 2.0 ** -26 / l).repeat_interleave(hq // hkv, 0)
        steps = 26 * 2.0 ** -22 + (n / 32 + 64) * 2.0 ** -23
        rel = (2.0 ** -8 if kind == BF16 else 2.0 ** -6 + 2.0 ** -11) + steps + 2.0 ** -8
        assert ((out[j].double() - y).abs() <= rel * y).all(), float(((out[j].double() - y).abs() / y).max())
        assert (lse[j].double() - (26 * math.log(2.0) + math.log(l))).abs().max() <= steps + 18.1 * 2.0 ** -22


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("rows", [1, 50])
def test_output_on_a_16_byte_boundary(kind, rows):
    pool = Pool(1, [300], 2, 128, 16, kind, seed=26)
    cache = pool.cuda()
    q = torch.randn(rows, 16, 128, device="cuda").to(BF16)
    ctx, cu = i32([300 - rows]), i32([0, rows])
    want, _ = svp.chunk_attn(q, ctx, cu, cache=cache)
    buf = torch.full((rows * 16 * 128 + 16,), -7.0, device="cuda", dtype=BF16)
    out = buf[8:-8].view(rows, 16, 128)
    assert out.data_ptr() % 32 == 16
    svp.chunk_attn(q, ctx, cu, cache=cache, out=out)
    assert torch.equal(out, want) and (buf[:8] == -7).all() and (buf[-8:] == -7).all()


def test_a_stream_that_is_not_the_current_one():
    """Outputs made by the call are cleared on the stream that the call runs on."""
    pool = Pool(1, [260], 2, 128, 16, BF16, seed=27)
    cache = pool.cuda()
    q = torch.randn(200, 8, 128, device="cuda").to(BF16)
    ctx, cu = i32([60]), i32([0, 200])
    want = svp.chunk_attn(q, ctx, cu, cache=cache)
    kw, vw = svp.cache_read(None, i32([0, 260]), cache=cache, rows=260)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    load = torch.randn(4096, 4096, device="cuda")
    for _ in range(3):
        for _ in range(8):
            load = load @ load * 1e-4          # the current stream is busy when the calls are made
        got = svp.chunk_attn(q, ctx, cu, cache=cache, stream=side)
        k, v = svp.cache_read(None, i32([0, 260]), cache=cache, rows=260, stream=side.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(k, kw) and torch.equal(v, vw)


def test_two_graphs_replayed_at_once():
    pool = Pool(2, [3000, 2500], 2, 128, 16, E4M3, seed=28)
    cache = pool.cuda()
    cu, ctx = i32([0, 5, 10]), i32([2900, 2400])
    qs = [torch.randn(10, 8, 128, device="cuda").to(BF16) for _ in range(2)]
    want = [svp.chunk_attn(q, ctx, cu, cache=cache, w=5)[0] for q in qs]
    graphs, outs = [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(svp.chunk_attn(q, ctx, cu, cache=cache, w=5)[0])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_one_workspace_for_every_head_layout_and_size():
    nb = max(svp.chunk_attn_workspace_size(hq, hkv, d) for hq, hkv, d in ((8, 2, 64), (8, 2, 128), (8, 2, 256)))
    ws = svp.Workspace(nb, zeroed=256)
    ws.buf[256:] = 255                # (NaN bits: nothing may rest on what is there)
    for d in (64, 256, 128, 64):
        for kind in (BF16, E4M3):
            for rows, ctx in (([1], [4000]), ([70, 3], [300, 2000])):
                check_attend(rows, ctx, hq=8, hkv=2, d=d, kind=kind, ws=ws, picks=(0, 2, 63, 64), seed=29)


def test_take_outside_its_range():
    pool = Pool(3, [40, 40, 40], 2, 64, 16, BF16, seed=30, stale="keep")
    cache = pool.cuda()
    before = [x.clone() for x in pool.dev]
    k = torch.randn(12, 2, 64, device="cuda").to(BF16)
    svp.cache_write(k, k, i32([5, 6, 7]), i32([0, 4, 8, 12]), cache=cache, take=i32([-3, 1 << 30, -(1 << 31)]))
    for x, y in zip(pool.dev, before):
        pg = pool.table.long().cuda()
        assert torch.equal(x[pg[0]], y[pg[0]]) and torch.equal(x[pg[2]], y[pg[2]])
        assert torch.equal(x[int(pool.table[1, 0]), :, 6:10], k[4:8].transpose(0, 1))
