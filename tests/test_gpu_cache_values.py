"""chunk_attn over 8-bit pages at the ends of the value range: value rows of zeros, exponent bytes
0 and 255, in calls of few query rows a KV head and of many, against softmax attention in 64 bits.

A rounding to nearest is off by eps / 2 relative: bf16 2^-8, fp16 2^-11, fp32 2^-24."""
import math

import pytest
import torch

import speculative_decoding_verification_packed_gb300 as svp

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn

# (query heads, KV heads, d, rows of a request): 1, 4 and 16 query rows of a KV head, which 8-bit pages of
# d <= 128 take apart from more; then 20, 160 (two query tiles) and d 256; last, more heads than SMs, so that
# no context is split
CALLS = [(2, 2, 64, 1), (8, 2, 128, 1), (8, 2, 128, 4), (4, 2, 64, 8), (8, 2, 128, 5), (8, 2, 64, 40), (4, 2, 256, 1),
         (304, 304, 64, 1), (304, 304, 128, 2), (304, 304, 64, 17)]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Cache8:
    """One request's 8-bit cache of T positions, keys and values [T, hkv, d] written by cache_write."""

    def __init__(self, T, hkv, d, seed, page=16, k=None, v=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.hkv, self.d, self.page = T, hkv, d, page
        pages = -(-T // page)
        self.table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None].contiguous()
        self.codes = [torch.full((pages, hkv, page, d), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.exps = [torch.full((pages, hkv, page), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.cache = svp.make_cache(self.codes[0].view(E4M3), self.codes[1].view(E4M3), self.table,
                                    k_exp=self.exps[0], v_exp=self.exps[1])
        k = torch.randn(T, hkv, d, generator=g, device="cuda").to(BF16) if k is None else k
        v = torch.randn(T, hkv, d, generator=g, device="cuda").to(BF16) if v is None else v
        svp.cache_write(k, v, i32([0]), i32([0, T]), cache=self.cache)

    def at(self, pos):
        """(pages, tokens) of positions."""
        pos = torch.as_tensor(pos, device="cuda")
        return self.table[0][pos // self.page].long(), pos % self.page

    def set_bytes(self, which, pos, byte):
        pg, tok = self.at(pos)
        self.exps[which][pg, :, tok] = byte

    def rows(self, which):
        """(values [T, hkv, d], powers of two [T, hkv]) in 64 bits: byte 0 stands for 0, 255 for NaN."""
        pg, tok = self.at(torch.arange(self.T))
        b = self.exps[which][pg, :, tok].to(torch.int64)
        e = ((b - 127 + 1023) << 52).view(torch.float64)
        x = self.codes[which][pg, :, tok].view(E4M3).double() * e[..., None]
        x = torch.where((b == 0)[..., None], torch.zeros_like(x), x)
        return torch.where((b == 255)[..., None], torch.full_like(x, float("nan")), x), e


def exact(c, q, rows, scale):
    """(o, lse, bounds) of `rows` last rows q [rows, hq, d] in 64 bits.  A = sum p |v| / l.  A probability
    is rounded to fp16: off by 2^-11, or, far below the largest, by 2^-25 where the largest product of
    a probability and its row's power of two is held at 2^7 or more; and by the error of its score, an
    fp32 sum of d products.  fp32 sums over the keys, exponentials and the logarithm add a few steps."""
    hq = q.shape[1]
    K, _ = c.rows(0)
    V, e = c.rows(1)
    G, T, d = hq // c.hkv, c.T, c.d
    qh = q.double().view(rows, c.hkv, G, d).permute(1, 0, 2, 3).reshape(c.hkv, rows * G, d)
    last = T - rows + torch.arange(rows, device="cuda").repeat_interleave(G)
    hidden = torch.arange(T, device="cuda")[None] > last[:, None]
    s = (qh @ K.permute(1, 2, 0) * scale).masked_fill(hidden, -math.inf)
    ds = (d + 2) * 2.0 ** -23 * (qh.abs() @ K.abs().permute(1, 2, 0) * scale).masked_fill(hidden, 0).amax(-1)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top)
    l = p.sum(-1, keepdim=True)
    v, ex = V.permute(1, 0, 2), e.permute(1, 0)[:, None]
    y = p @ v / l
    A = p @ v.abs() / l
    codes = (v.abs() / ex.transpose(1, 2))
    floor = 2.0 ** -32 * (p * ex).amax(-1, keepdim=True) * codes.sum(1, keepdim=True) / l
    steps = (T / 32 + 64) * 2.0 ** -23
    tol = (2.0 ** -11 + 2 * ds[..., None] + steps) * A + floor + 2.0 ** -8 * y.abs() + 1e-30
    lse = (top + torch.log(l)).squeeze(-1)
    ltol = ds + steps + lse.abs() * 2.0 ** -22

    def back(x):
        return x.view(c.hkv, rows, G, -1).permute(1, 0, 2, 3).reshape(rows, hq, -1)
    return back(y), back(lse).squeeze(-1), back(tol), back(ltol).squeeze(-1)


def attend(c, q, rows, scale=0.0):
    ws = svp.Workspace(svp.chunk_attn_workspace_size(q.shape[1], c.hkv, c.d))
    out, lse = svp.chunk_attn(q, i32([c.T - rows]), i32([0, rows]), cache=c.cache, w=rows, scale=scale, ws=ws)
    assert ws.read_status() == 0
    return out.double(), lse.double()


def check(c, q, rows, scale=0.0, out_too=True):
    out, lse = attend(c, q, rows, scale)
    o, l, tol, ltol = exact(c, q, rows, scale or 1 / math.sqrt(c.d))
    assert torch.isfinite(lse).all()
    assert ((lse - l).abs() <= ltol).all(), float(((lse - l).abs() / ltol).max())
    if out_too:
        assert ((out - o).abs() <= tol).all(), float(((out - o).abs() / tol).max())
    return out, lse


def query(rows, hq, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(rows, hq, d, generator=g, device="cuda").to(BF16)


# ------------------------------------------------------------------ value rows of zeros
@pytest.mark.parametrize("T", [600, 16384])
@pytest.mark.parametrize("hq,hkv,d,rows", CALLS)
def test_every_value_row_is_zero(hq, hkv, d, rows, T):
    """As cache_write stores them (byte 15): the output is 0 and the normaliser that of the scores."""
    if hkv > 2 and T > 600:
        T = 2500                       # (the 64-bit form's memory)
    c = Cache8(T, hkv, d, 1, v=torch.zeros(T, hkv, d, dtype=BF16, device="cuda"))
    assert (c.rows(1)[1] == 2.0 ** -112).all()
    out, _ = check(c, query(rows, hq, d, 2), rows)
    assert (out == 0).all()


@pytest.mark.parametrize("where", ["first", "last", "every other", "one row is not"])
@pytest.mark.parametrize("hq,hkv,d,rows", CALLS)
def test_some_value_rows_are_zero(hq, hkv, d, rows, where):
    T = 2500
    g = torch.Generator(device="cuda").manual_seed(3)
    v = torch.randn(T, hkv, d, generator=g, device="cuda").to(BF16)
    zero = {"first": slice(0, 2300), "last": slice(900, T), "every other": slice(0, T, 2)}.get(where)
    if zero is None:
        v[:1203] = 0
        v[1204:] = 0
    else:
        v[zero] = 0
    check(Cache8(T, hkv, d, 4, v=v), query(rows, hq, d, 5), rows)


@pytest.mark.parametrize("hq,hkv,d,rows", CALLS)
def test_a_value_row_of_zeros_takes_nearly_all_weight(hq, hkv, d, rows):
    """The first key, as probable as 2^20 of the others, has a value of zeros."""
    T = 2500
    g = torch.Generator(device="cuda").manual_seed(6)
    k, v = torch.zeros(T, hkv, d, dtype=BF16, device="cuda"), torch.randn(T, hkv, d, generator=g, device="cuda").to(BF16)
    k[0, :, 0] = 20.0
    v[0] = 0
    q = torch.zeros(rows, hq, d, dtype=BF16, device="cuda")
    q[..., 0] = 1.0
    check(Cache8(T, hkv, d, 7, k=k, v=v), q, rows, scale=math.log(2.0))


@pytest.mark.parametrize("low,high", [(1, 10), (1, 67), (20, 100), (100, 180), (150, 246)])
@pytest.mark.parametrize("hq,hkv,d,rows", [x for x in CALLS if x[2] <= 128 and x[0] // x[1] * x[3] <= 16])
def test_value_rows_of_any_power_of_two(hq, hkv, d, rows, low, high):
    """Bytes low..high in one request, the rows past its last one among the smallest."""
    T = 2500
    c = Cache8(T, hkv, d, 8)
    g = torch.Generator(device="cuda").manual_seed(9)
    used = c.exps[1] != 255
    c.exps[1][:] = torch.where(used, torch.randint(low, high + 1, c.exps[1].shape, generator=g, device="cuda").to(torch.uint8),
                               torch.ones_like(c.exps[1]))
    check(c, query(rows, hq, d, 10), rows)


# ------------------------------------------------------------------ byte 255: NaN
@pytest.mark.parametrize("at", [0, 700, 1999])
@pytest.mark.parametrize("hq,hkv,d,rows", CALLS)
def test_nan_in_a_value_row_alone(hq, hkv, d, rows, at):
    """Every element of a row that sees it is NaN; the normaliser, which has no value row in it, and the
    other heads are those of the finite rows."""
    T, other = 2500, hkv - 1
    q = query(rows, hq, d, 13)
    c = Cache8(T, hkv, d, 12)
    o, l, tol, ltol = exact(c, q, rows, 1 / math.sqrt(d))
    pg, tok = c.at([at])
    c.exps[1][pg, other, tok] = 255
    out, lse = attend(c, q, rows)
    G = hq // hkv
    assert ((lse - l).abs() <= ltol).all()
    assert torch.isnan(out[:, other * G:]).all()
    assert ((out - o).abs() <= tol)[:, :other * G].all()


@pytest.mark.parametrize("hq,hkv,d,rows", [x for x in CALLS if x[3] > 1])
def test_nan_in_the_value_row_of_the_last_key(hq, hkv, d, rows):
    """It is not in the normaliser of any row, and in calls of few rows not in the output of rows that do
    not see it."""
    T = 2500
    q = query(rows, hq, d, 15)
    c = Cache8(T, hkv, d, 14)
    o, l, tol, ltol = exact(c, q, rows, 1 / math.sqrt(d))
    c.set_bytes(1, [T - 1], 255)
    out, lse = attend(c, q, rows)
    assert ((lse - l).abs() <= ltol).all()
    assert torch.isnan(out[-1]).all()
    if d <= 128 and hq // hkv * rows <= 16:
        assert ((out - o).abs() <= tol)[:-1].all()


# ------------------------------------------------------------------ byte 0: zeros
@pytest.mark.parametrize("where", ["all", "first", "every other", "keys too"])
@pytest.mark.parametrize("hq,hkv,d,rows", CALLS)
def test_exponent_byte_0_stands_for_zeros(hq, hkv, d, rows, where):
    """Whatever the row's codes, as in a cache whose bytes are zeros."""
    T = 2500
    c = Cache8(T, hkv, d, 16)
    pos = torch.arange(T)
    pos = {"all": pos, "first": pos[:2300], "every other": pos[::2], "keys too": pos[100:2300]}[where]
    c.set_bytes(1, pos, 0)
    if where == "keys too":
        c.set_bytes(0, pos[:1000], 0)
    out, _ = check(c, query(rows, hq, d, 17), rows)
    if where == "all":
        assert (out == 0).all()


# ------------------------------------------------------------------ queries and keys of any size
def sized(rows, hq, hkv, d, qe, ke, seed):
    """A cache and query of normal numbers times 2^ke and 2^qe, and the scale of unit scores."""
    T = 2500
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = (torch.randn(T, hkv, d, generator=g, device="cuda") * 2.0 ** ke).to(BF16)
    q = (query(rows, hq, d, seed + 1).float() * 2.0 ** (qe / 2) * 2.0 ** (qe / 2)).to(BF16)
    return Cache8(T, hkv, d, seed + 2, k=k), q, 2.0 ** -(qe + ke) / math.sqrt(d)


@pytest.mark.parametrize("qe", [0, -85])
@pytest.mark.parametrize("hq,hkv,d,rows", CALLS)
def test_every_score_is_zero(hq, hkv, d, rows, qe):
    """Keys of zeros (byte 15), which hide from no row what it may not see."""
    T = 2500
    c = Cache8(T, hkv, d, 18, k=torch.zeros(T, hkv, d, dtype=BF16, device="cuda"))
    check(c, (query(rows, hq, d, 19).float() * 2.0 ** qe).to(BF16), rows)


@pytest.mark.parametrize("qe,ke", [(118, -50), (124, 0), (-116, 60), (-108, 40), (-60, 0)])
@pytest.mark.parametrize("hq,hkv,d,rows", CALLS)
def test_queries_of_any_size(hq, hkv, d, rows, qe, ke):
    c, q, scale = sized(rows, hq, hkv, d, qe, ke, 18)
    check(c, q, rows, scale=scale)


@pytest.mark.parametrize("qe,ke", [(-104, 112), (-90, 100), (60, -50)])
@pytest.mark.parametrize("hq,hkv,d,rows", CALLS)
def test_keys_of_any_size(hq, hkv, d, rows, qe, ke):
    c, q, scale = sized(rows, hq, hkv, d, qe, ke, 20)
    check(c, q, rows, scale=scale)


# ------------------------------------------------------------------ scratch of calls that bring none
def test_scratch_of_many_streams_is_bounded():
    """More streams than scratch buffers are kept for, all at once and in turn."""
    c = Cache8(3000, 2, 64, 22)
    q = query(1, 8, 64, 23)
    ctx, cu = i32([2999]), i32([0, 1])
    want = svp.chunk_attn(q, ctx, cu, cache=c.cache)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(24)]
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(svp.chunk_attn(q, ctx, cu, cache=c.cache))
            assert len(svp._chunk_ws) <= 16
    torch.cuda.synchronize()
    assert all(torch.equal(a, want[0]) and torch.equal(b, want[1]) for a, b in got)


# ------------------------------------------------------------------ rows of zeros among large values
@pytest.mark.parametrize("ve", [0, 30, 45])
@pytest.mark.parametrize("hq,hkv,d,rows", CALLS)
def test_value_rows_of_zeros_among_large_ones_keep_their_weight(hq, hkv, d, rows, ve):
    """A few keys have values of normal numbers times 2^ve and score 12 powers of two above the others,
    whose values are zeros and which have a good part of the weight together."""
    T = 2500 if hkv > 2 else 40000
    g = torch.Generator(device="cuda").manual_seed(24)
    k = torch.zeros(T, hkv, d, dtype=BF16, device="cuda")
    v = (torch.randn(T, hkv, d, generator=g, device="cuda") * 2.0 ** ve).to(BF16)
    loud = torch.arange(0, T, 5000 if hkv <= 2 else 2501, device="cuda")
    k[loud, :, 0] = 12.0
    quiet = torch.ones(T, dtype=torch.bool, device="cuda")
    quiet[loud] = False
    v[quiet] = 0
    q = torch.zeros(rows, hq, d, dtype=BF16, device="cuda")
    q[..., 0] = 1.0
    check(Cache8(T, hkv, d, 25, k=k, v=v), q, rows, scale=math.log(2.0))


@pytest.mark.parametrize("low,high", [(67, 167), (120, 220), (140, 240)])
@pytest.mark.parametrize("down", [False, True])
@pytest.mark.parametrize("hq,hkv,d,rows", CALLS)
def test_tiles_of_any_power_of_two_within_2_to_the_100(hq, hkv, d, rows, low, high, down):
    """Value rows of one power of two per 128 positions, over a range of 2^100 up or down the context."""
    T = 2500
    c = Cache8(T, hkv, d, 26)
    tiles = -(-T // 128)
    for t in range(tiles):
        at = tiles - 1 - t if down else t
        c.set_bytes(1, list(range(128 * t, min(T, 128 * t + 128))), low + (high - low) * at // (tiles - 1))
    check(c, query(rows, hq, d, 27), rows)


@pytest.mark.parametrize("up", [8, 24, 60])
@pytest.mark.parametrize("hq,hkv,d,rows", [x for x in CALLS if x[2] <= 128 and x[0] // x[1] * x[3] <= 16])
def test_digits_beside_a_value_row_of_zeros(hq, hkv, d, rows, up):
    """The first key's value is zeros and it is 2^up times as probable as the few others, whose
    probabilities keep their digits: what comes out is theirs."""
    T = rows + 2
    g = torch.Generator(device="cuda").manual_seed(28)
    k = torch.randn(T, hkv, d, generator=g, device="cuda") * 0.5
    v = torch.randn(T, hkv, d, generator=g, device="cuda").to(BF16)
    k[:, :, 0] = 0
    k[0] = 0
    k[0, :, 0] = up
    v[0] = 0
    q = query(rows, hq, d, 29)
    q[..., 0] = 1.0
    check(Cache8(T, hkv, d, 30, k=k.to(BF16), v=v), q, rows, scale=math.log(2.0))


# ------------------------------------------------------------------ NaN under no weight
@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("at", [100, 200, 8000])
@pytest.mark.parametrize("hq,hkv,d,rows", CALLS)
def test_nan_value_under_a_vanishing_probability(hq, hkv, d, rows, at, kind):
    """A value row of NaN whose key scores 2^300 below the first: 0 times NaN, as in the plain form, in
    whichever part of the keys it lies."""
    T = 9000 if hkv <= 2 else 300
    at = min(at, T - rows - 1)
    k = torch.zeros(T, hkv, d, dtype=BF16, device="cuda")
    v = torch.ones(T, hkv, d, dtype=BF16, device="cuda")
    k[0, :, 0] = 304.0
    v[at, hkv - 1] = float("nan")
    q = torch.zeros(rows, hq, d, dtype=BF16, device="cuda")
    q[..., 0] = 1.0
    if kind == E4M3:
        cache = Cache8(T, hkv, d, 31, k=k, v=v).cache
    else:
        pages = -(-T // 16)
        pools = [torch.zeros(pages, hkv, 16, d, dtype=BF16, device="cuda") for _ in range(2)]
        cache = svp.make_cache(*pools, torch.arange(pages, device="cuda", dtype=torch.int32)[None].contiguous())
        svp.cache_write(k, v, i32([0]), i32([0, T]), cache=cache)
    out, lse = svp.chunk_attn(q, i32([T - rows]), i32([0, rows]), cache=cache, w=rows, scale=math.log(2.0))
    G = hq // hkv
    assert torch.isnan(out[:, -G:]).all()
    assert (out[:, :-G] == 1).all()
    top = 304.0 if kind == BF16 else 320.0          # (304 = 9.5 * 32 goes to 10 * 32 in e4m3)
    assert (lse - top * math.log(2.0)).abs().max() < 1e-3


# ------------------------------------------------------------------ page ids
@pytest.mark.parametrize("bad", [-(1 << 31), -(1 << 31) + 1, -1, (1 << 31) - 1])
@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("rows,d", [(1, 64), (40, 128), (1, 256)])
def test_every_page_id_outside_the_pool_sets_the_status(rows, d, kind, bad):
    T, hkv, hq = 1000, 2, 8
    pages = -(-T // 16)
    g = torch.Generator(device="cuda").manual_seed(32)
    x = [torch.randn(pages, hkv, 16, d, generator=g, device="cuda").to(BF16).to(kind) for _ in range(2)]
    e = [torch.full((pages, hkv, 16), 127, dtype=torch.uint8, device="cuda") for _ in range(2)] if kind == E4M3 else [None, None]
    table = torch.arange(pages, device="cuda", dtype=torch.int32)[None].contiguous()
    cache = svp.make_cache(*x, table, k_exp=e[0], v_exp=e[1])
    q = query(rows, hq, d, 33)
    got = []
    for page in (bad, None):
        if page is None:                  # the same page as zeros
            table[0, 7] = 7
            for z in x:
                z.view(torch.uint8)[7] = 0
        else:
            table[0, 7] = page
        ws = svp.Workspace(svp.chunk_attn_workspace_size(hq, hkv, d))
        got.append(svp.chunk_attn(q, i32([T - rows]), i32([0, rows]), cache=cache, w=rows, ws=ws))
        assert ws.read_status() == (svp.DEV_BAD_CONTEXT if page is not None else 0)
    # (a page of zeros may have another power of two than the rows of zeros written here: two more roundings)
    assert (got[0][0].float() - got[1][0].float()).abs().max() <= 2 * 2.0 ** -8 * got[1][0].float().abs().max()
    assert (got[0][1] - got[1][1]).abs().max() <= 1e-4
