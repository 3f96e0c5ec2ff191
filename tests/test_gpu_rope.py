"""Rotary positions on the GPU against 64 bits: rope, and rope_cache_write with what the cache then holds.

Error of an element x cos - y sin, rounded once to its type (eps / 2 relative): the angle's upper 32 bits are
off by at most 2^-32 of a turn and are rounded to 24 bits (2^-24 of half a turn at most), so the angle is off by
pi (2^-31 + 2^-24); sincospif is off by 2 ulp (2^-23 of 1), the scale's product, the products and their sum by
four times 2^-24.  Together, of |x| + |y|: pi 2^-23.9 + 2^-22.9 + 2^-22 < 2^-20.9; 2^-20 is taken."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_packed_gb300 as svp
from test_gpu_cache import Pool, BF16, F32, E4M3, bytes_of, e4m3_values, i32, packed

pytestmark = pytest.mark.gpu

FP32_PART = 2.0 ** -20


def positions(ctx, rows):
    return np.concatenate([np.arange(c, c + k) for c, k in zip(ctx, rows)] + [np.zeros(0)]).astype(np.int64)


def rotated(x, pos, freq, interleaved, scale):
    """x [m, h, d] (64-bit) rotated at pos [m], and |x| + |y| of each element's pair (0 where nothing turns)."""
    turns = [(int(f) & (2 ** 64 - 1)) for f in freq.cpu().tolist()]
    half = len(turns)
    out, size = x.copy(), np.zeros_like(x)
    # angles from whole numbers: position times turns modulo one, exact
    frac = np.array([[((int(p) * f) % 2 ** 64) / 2.0 ** 64 for f in turns] for p in pos]).reshape(len(pos), half)
    c, s = np.cos(2 * math.pi * frac)[:, None] * scale, np.sin(2 * math.pi * frac)[:, None] * scale
    a, b = (np.arange(half), np.arange(half) + half) if not interleaved else (2 * np.arange(half), 2 * np.arange(half) + 1)
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., a] * s + x[..., b] * c
    size[..., a] = size[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(scale)
    return out, size


def check(got, want, size):
    eps = torch.finfo(got.dtype).eps / 2
    got = got.double().cpu().numpy()
    bound = eps * np.abs(want) + (1 + eps) * FP32_PART * size + 2.0 ** -133
    bad = np.abs(got - want) > bound
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


def fused(m, hq, hkv, d, kind, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, hq + 2 * hkv + pad, d, generator=g).to(kind).cuda()
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:hq + 2 * hkv]


CASES = [([1], [0]), ([1, 1, 1], [15, 4096, 1048575]), ([5, 0, 37, 1, 16], [0, 9, 100, 2 ** 31 - 2, 1]),
         ([300, 2, 0, 129], [7, 127, 0, 500]), ([1] * 300, [3] * 300), ([2900], [11])]


@pytest.mark.parametrize("rows,ctx", CASES)
@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hkv,d,rot", [(4, 2, 64, 64), (32, 8, 128, 128), (3, 1, 256, 64), (5, 5, 128, 18), (2, 2, 64, 2),
                                          (24, 2, 256, 256), (1, 1, 128, 112)])
def test_rows(rows, ctx, kind, interleaved, hq, hkv, d, rot):
    m, extra = sum(rows), 3
    q, k, _ = fused(m + extra, hq, hkv, d, kind, seed=m + rot)
    freq = svp.rope_frequencies(rot, base=500000.0)
    q_out = torch.full_like(q.contiguous(), 7.0)
    k_out = torch.full_like(k.contiguous(), -7.0)
    ws = svp.Workspace(256)
    svp.rope(q, k, i32(ctx), i32(packed(rows)), freq=freq, interleaved=interleaved, scale=1.25, q_out=q_out, k_out=k_out, ws=ws)
    assert ws.read_status() == 0
    pos = positions(ctx, rows)
    for x, y, fill in ((q, q_out, 7.0), (k, k_out, -7.0)):
        want, size = rotated(x[:m].double().cpu().numpy(), pos, freq, interleaved, 1.25)
        check(y[:m], want, size)
        assert (y[:m, :, rot:] == x[:m, :, rot:]).all()           # bits of what does not turn
        assert (y[m:] == fill).all()


@pytest.mark.parametrize("interleaved,rot", [(False, 128), (False, 18), (False, 96), (True, 128), (True, 6)])
@pytest.mark.parametrize("kind", [BF16, F32])
def test_in_place_equals_out_of_place_and_turns_back(kind, interleaved, rot):
    rows, ctx = [16, 1, 0, 700], [5, 100000, 3, 0]
    m = sum(rows)
    q, k, v = fused(m, 6, 2, 128, kind, seed=3)
    before = [x.clone() for x in (q, k, v)]
    freq = svp.rope_frequencies(rot, scaling="linear", factor=2.0)
    cu = i32(packed(rows))
    a, b = svp.rope(q, k, i32(ctx), cu, freq=freq, interleaved=interleaved)
    qq, kk = svp.rope(q, k, i32(ctx), cu, freq=freq, interleaved=interleaved, q_out=q, k_out=k)
    assert qq.data_ptr() == q.data_ptr() and torch.equal(a, q) and torch.equal(b, k)
    assert torch.equal(v, before[2])                              # what lies between is not touched
    back = -torch.from_numpy(positions(ctx, rows)).to(torch.int32).cuda()
    svp.rope(q, k, None, cu, freq=freq, interleaved=interleaved, pos=back, q_out=q, k_out=k)
    eps = torch.finfo(kind).eps / 2
    for x, y in ((q, before[0]), (k, before[1])):
        # two roundings of elements no larger than the pair's |x| + |y| <= 2 max, through products with cos and sin
        worst = y.double().abs().amax() * 2
        assert ((x.double() - y.double()).abs() <= (2 * eps * 2 + 2 * 2 * FP32_PART) * worst).all()


def test_given_positions_and_single_inputs():
    m = 40
    q, k, _ = fused(m, 4, 2, 64, F32, seed=8)
    freq = svp.rope_frequencies(64)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (m,), dtype=torch.int64, generator=torch.Generator().manual_seed(1))
    dev = pos.to(torch.int32).cuda()
    cu = i32([0, 17, 17, m])
    both = svp.rope(q, k, None, cu, freq=freq, pos=dev)
    alone_q, none = svp.rope(q, None, None, cu, freq=freq, pos=dev)
    none2, alone_k = svp.rope(None, k, None, cu, freq=freq, pos=dev)
    assert none is None and none2 is None and torch.equal(both[0], alone_q) and torch.equal(both[1], alone_k)
    for x, y in ((q, both[0]), (k, both[1])):
        want, size = rotated(x.double().cpu().numpy(), pos.numpy(), freq, False, 1.0)
        check(y, want, size)


def test_no_rows_and_no_requests():
    q, k, _ = fused(4, 4, 2, 64, BF16, seed=2)
    freq = svp.rope_frequencies(64)
    out = torch.full_like(q.contiguous(), 3.0)
    svp.rope(q, None, i32([]), i32([0]), freq=freq, q_out=out)
    svp.rope(q, None, i32([5, 5]), i32([0, 0, 0]), freq=freq, q_out=out)
    assert (out == 3.0).all()
    a, b = svp.rope(q[:0], k[:0], i32([5]), i32([0, 0]), freq=freq)
    assert a.shape == (0, 4, 64) and b.shape == (0, 2, 64)


def test_values_that_are_not_finite_stay_in_their_pairs():
    x = torch.ones(1, 1, 64, device="cuda")
    x[0, 0, 3], x[0, 0, 40], x[0, 0, 63] = float("nan"), float("inf"), 3e38
    freq = svp.rope_frequencies(62)
    y, _ = svp.rope(x, None, i32([9]), i32([0, 1]), freq=freq)
    bad = {3, 34, 9, 40}
    for e in range(62):
        assert torch.isfinite(y[0, 0, e]).item() == (e not in bad)
    assert y[0, 0, 63] == x[0, 0, 63]


@pytest.mark.parametrize("rows,ctx,page", [([1], [0], 16), ([1, 1, 1], [15, 16, 170], 16), ([5, 0, 37, 1, 16], [0, 9, 100, 63, 1], 32),
                                           ([300, 2, 0, 129], [7, 127, 0, 500], 128), ([1] * 200, [3] * 200, 64)])
@pytest.mark.parametrize("new,kind", [(BF16, BF16), (F32, F32), (BF16, E4M3), (F32, E4M3), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("hq,hkv,d,rot,interleaved", [(8, 2, 128, 128, False), (4, 4, 64, 64, True), (3, 1, 256, 96, False),
                                                      (2, 2, 64, 18, False)])
def test_cache_write(rows, ctx, page, new, kind, hq, hkv, d, rot, interleaved):
    m = sum(rows)
    q, k, v = fused(m + 2, hq, hkv, d, new, seed=m + d)
    pool = Pool(len(rows), [c + r for c, r in zip(ctx, rows)], hkv, d, page, kind, stale="keep", layout="token" if d == 64 else "head")
    cache = pool.cuda()
    before = [bytes_of(x).clone() for x in pool.dev]
    same = Pool(len(rows), [c + r for c, r in zip(ctx, rows)], hkv, d, page, kind, stale="keep", layout="token" if d == 64 else "head")
    other = same.cuda()
    freq = svp.rope_frequencies(rot)
    ws = svp.Workspace(256)
    out = svp.rope_cache_write(q, k, v, i32(ctx), i32(packed(rows)), cache=cache, freq=freq, interleaved=interleaved, scale=0.75, ws=ws)
    assert ws.read_status() == 0
    alone, kr = svp.rope(q, k, i32(ctx), i32(packed(rows)), freq=freq, interleaved=interleaved, scale=0.75)
    assert torch.equal(out, alone)
    # v, and every place that belongs to another position, as cache_write leaves them
    svp.cache_write(kr, v.contiguous(), i32(ctx), i32(packed(rows)), cache=other)
    assert torch.equal(bytes_of(pool.dev[1]), bytes_of(same.dev[1]))
    if kind == E4M3:
        assert torch.equal(pool.dev_exps[1], same.dev_exps[1])
    pos = positions(ctx, rows)
    want, size = rotated(k[:m].double().cpu().numpy(), pos, freq, interleaved, 0.75)
    req = np.repeat(np.arange(len(rows)), rows)
    pg, tok = pool.table.numpy()[req, pos // page], pos % page
    if kind == E4M3:
        codes = bytes_of(pool.dev[0]).numpy()[pg, :, tok]
        b = pool.dev_exps[0].cpu().numpy()[pg, :, tok].astype(np.float64)
        two = 2.0 ** (b - 127)[..., None]
        got = e4m3_values(codes) * two
        top = np.abs(want).max(-1)
        # the smallest power of two that takes the row's largest to 448, but for rows within the rotation's error of it
        slack = (size.max(-1)) * FP32_PART
        assert (top - slack <= 448 * two[..., 0]).all() and ((top + slack > 224 * two[..., 0]) | (b == 15)).all()
        err = FP32_PART * size
        assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * two + 1.0625 * err).all()
    else:
        held = pool.dev[0].cpu()[torch.from_numpy(pg).long(), :, torch.from_numpy(tok).long()]
        check(held, want, size)
    written = np.zeros((pool.dev[0].shape[0], page), bool)
    written[pg, tok] = True
    now = bytes_of(pool.dev[0]).view(before[0].shape)
    keep = torch.from_numpy(~written)
    assert torch.equal(now.transpose(1, 2)[keep], before[0].transpose(1, 2)[keep])


def test_cache_write_takes_the_accepted_rows_only_and_turns_every_query():
    rows, ctx, take = [7, 16, 3, 5], [20, 0, 300, 16], [3, 16, 0, 99]
    m = sum(rows)
    q, k, v = fused(m, 4, 2, 128, BF16, seed=5)
    freq = svp.rope_frequencies(128)
    pools = [Pool(4, [c + r for c, r in zip(ctx, rows)], 2, 128, 16, BF16, stale="keep") for _ in range(2)]
    caches = [p.cuda() for p in pools]
    a = svp.rope_cache_write(q, k, v, i32(ctx), i32(packed(rows)), cache=caches[0], freq=freq, take=i32(take))
    b, kr = svp.rope(q, k, i32(ctx), i32(packed(rows)), freq=freq)
    svp.cache_write(kr, v.contiguous(), i32(ctx), i32(packed(rows)), cache=caches[1], take=i32(take))
    assert torch.equal(a, b)
    for x, y in zip(pools[0].dev, pools[1].dev):
        assert torch.equal(bytes_of(x), bytes_of(y))
    # without queries, and in place
    assert svp.rope_cache_write(None, k, v, i32(ctx), i32(packed(rows)), cache=caches[0], freq=freq) is None
    svp.rope_cache_write(q, k, v, i32(ctx), i32(packed(rows)), cache=caches[0], freq=freq, q_out=q)
    assert torch.equal(q, b)


def test_rows_with_infinities_are_nan_rows_of_an_8_bit_cache():
    q, k, v = fused(3, 1, 1, 64, F32, seed=1)
    k[1, 0, 5], v[2, 0, 7] = float("inf"), float("nan")
    pool = Pool(1, [3], 1, 64, 16, E4M3, stale="keep")
    cache = pool.cuda()
    svp.rope_cache_write(q, k, v, i32([0]), i32([0, 3]), cache=cache, freq=svp.rope_frequencies(64))
    kk, vv = svp.cache_read(None, i32([0, 3]), cache=cache, rows=3, dtype=F32)
    assert torch.isnan(kk[1]).all() and torch.isfinite(kk[[0, 2]]).all()
    assert torch.isnan(vv[2]).all() and torch.isfinite(vv[:2]).all()


def test_broken_requests_are_skipped_and_reported():
    m = 20
    q, k, v = fused(m, 2, 2, 64, BF16, seed=4)
    freq = svp.rope_frequencies(64)
    ws = svp.Workspace(256)
    out = torch.full_like(q.contiguous(), 9.0)
    # request 1 runs backwards
    svp.rope(q, None, i32([0, 0, 0]), i32([0, 8, 4, 12]), freq=freq, q_out=out, ws=ws)
    assert ws.read_status() == svp.DEV_BAD_SLOTS and (out[12:] == 9.0).all() and (out[:4] != 9.0).any()
    # request 1 is behind the rows
    out.fill_(9.0)
    svp.rope(q, None, i32([0, 0]), i32([0, 8, 21]), freq=freq, q_out=out, ws=ws)
    assert ws.read_status() == svp.DEV_BAD_SLOTS and (out[8:] == 9.0).all()
    # negative and too far positions
    out.fill_(9.0)
    svp.rope(q, None, i32([-1, 2 ** 31 - 4, 5]), i32([0, 4, 9, 12]), freq=freq, q_out=out, ws=ws)
    assert ws.read_status() == svp.DEV_BAD_CONTEXT and (out[:9] == 9.0).all() and (out[9:12] != 9.0).any()
    # a cache: positions past its table, a page outside the pool
    pool = Pool(3, [16, 16, 16], 2, 64, 16, BF16, stale="keep")
    pool.table[2, 0] = 1000
    cache = pool.cuda()
    before = [x.clone() for x in pool.dev]
    out.fill_(9.0)
    svp.rope_cache_write(q, k, v, i32([12, -3, 4]), i32([0, 5, 8, 12]), cache=cache, freq=freq, q_out=out, ws=ws)
    assert ws.read_status() == svp.DEV_BAD_CONTEXT
    assert (out[:8] == 9.0).all() and (out[8:12] != 9.0).any() and (out[12:] == 9.0).all()
    assert all(torch.equal(x, y) for x, y in zip(pool.dev, before))


def test_other_stream_and_captured():
    rows, ctx = [4, 9], [100, 7]
    m = sum(rows)
    q, k, v = fused(m, 4, 2, 128, BF16, seed=6)
    freq, cu, c = svp.rope_frequencies(128), i32(packed(rows)), i32(ctx)
    want = svp.rope(q, k, c, cu, freq=freq)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = svp.rope(q, k, c, cu, freq=freq, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    pool = Pool(2, [104, 16], 2, 128, 16, E4M3, stale="keep")
    cache = pool.cuda()
    q_out = torch.zeros_like(q.contiguous())
    svp.rope_cache_write(q, k, v, c, cu, cache=cache, freq=freq, q_out=q_out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        svp.rope_cache_write(q, k, v, c, cu, cache=cache, freq=freq, q_out=q_out)
    c.copy_(i32([90, 0]))
    g.replay()
    torch.cuda.synchronize()
    want, _ = svp.rope(q, k, i32([90, 0]), cu, freq=freq)
    assert torch.equal(q_out, want)


def test_binding_refusals():
    q, k, v = fused(4, 4, 2, 64, BF16, seed=6)
    freq, cu, c = svp.rope_frequencies(64), i32([0, 4]), i32([0])
    with pytest.raises(ValueError):
        svp.rope(None, None, c, cu, freq=freq)
    with pytest.raises(ValueError):
        svp.rope(q, k[:3], c, cu, freq=freq)
    with pytest.raises(ValueError):
        svp.rope(q, k.float(), c, cu, freq=freq)
    with pytest.raises(ValueError):
        svp.rope(q, k, c, cu, freq=freq.cpu())
    with pytest.raises(ValueError):
        svp.rope(q, k, c.long(), cu, freq=freq)
    with pytest.raises(ValueError):
        svp.rope(q, None, c, cu, freq=freq, k_out=k)
    with pytest.raises(ValueError):
        svp.rope(q, None, c, cu, freq=freq, q_out=k)
    with pytest.raises(ValueError):
        svp.rope(q, None, None, cu, freq=freq, pos=i32([0, 1]))
    with pytest.raises(ValueError):
        svp.rope(q.transpose(0, 1), None, c, cu, freq=freq)
    with pytest.raises(svp.SvpError):
        svp.rope(q, None, None, cu, freq=freq)
    with pytest.raises(svp.SvpError):
        svp.rope(q, None, c, cu, freq=svp.rope_frequencies(66))
