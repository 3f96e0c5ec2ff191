"""The pages' calls on the GPU against a model in plain Python that follows their definitions one request and one
page at a time: tables, counts, status bits, and every byte of the pools."""
import random

import numpy as np
import pytest
import torch

import speculative_decoding_verification_packed_gb300 as svp
from test_gpu_cache import BF16, F32, E4M3, bytes_of, i32

pytestmark = pytest.mark.gpu


class Model:
    def __init__(self, n, cols, page, num, table=None, used=None, refs=None):
        self.n, self.cols, self.page, self.num = n, cols, page, num
        self.table = [[-1] * cols for _ in range(n)] if table is None else [list(r) for r in table]
        self.used = [0] * n if used is None else list(used)
        self.refs = [0] * num if refs is None else list(refs)
        self.status = 0
        self.copies = []              # (from, to, tokens) in order

    def pages(self, tokens):
        return -(-tokens // self.page)

    def inside(self, page):
        return 0 <= page < self.num

    def resize(self, length):
        before = list(self.refs)
        want = []
        for i in range(self.n):
            u, w = self.used[i], None
            if not 0 <= u <= self.cols:
                self.status |= svp.DEV_BAD_CONTEXT
            elif length[i] >= 0:
                w = self.pages(length[i])
                last = self.table[i][w - 1] if 0 < w <= self.cols else -1
                if w > self.cols or (w <= u and length[i] % self.page and self.inside(last) and before[last] > 1):
                    self.status |= svp.DEV_BAD_CONTEXT
                    w = None
            want.append(w)
        for i in range(self.n):
            if want[i] is not None and want[i] < self.used[i]:
                for j in range(want[i], self.used[i]):
                    page = self.table[i][j]
                    self.table[i][j] = -1
                    if self.inside(page) and self.refs[page] > 0:
                        self.refs[page] -= 1
                    else:
                        self.status |= svp.DEV_BAD_CONTEXT
                self.used[i] = want[i]
        free = [x for x in range(self.num) if self.refs[x] == 0]
        asked = 0
        for i in range(self.n):
            if want[i] is not None and want[i] > self.used[i]:
                k = want[i] - self.used[i]
                if asked + k <= len(free):
                    for j in range(k):
                        page = free[asked + j]
                        self.table[i][self.used[i] + j] = page
                        self.refs[page] = 1
                    self.used[i] = want[i]
                else:
                    self.status |= svp.DEV_NO_PAGES
                asked += k

    def fork(self, src, dst, length):
        used, table = list(self.used), [list(r) for r in self.table]
        free = [x for x in range(self.num) if self.refs[x] == 0]
        asked, taken, full = 0, set(), False
        for s, t, k in zip(src, dst, length):
            if not (0 <= s < self.n and 0 <= t < self.n) or used[t] != 0:
                self.status |= svp.DEV_BAD_SLOTS
            elif k < 0 or not 0 <= used[s] <= self.cols or k > used[s] * self.page:
                self.status |= svp.DEV_BAD_CONTEXT
            elif t in taken:
                self.status |= svp.DEV_BAD_SLOTS
            else:
                taken.add(t)
                whole, part = k // self.page, k % self.page
                asked += part > 0
                if asked > len(free):
                    self.status |= svp.DEV_NO_PAGES
                    continue
                row = [-1] * self.cols
                for j in range(whole):
                    page = table[s][j]
                    if self.inside(page):
                        row[j] = page
                        self.refs[page] += 1
                    else:
                        self.status |= svp.DEV_BAD_CONTEXT
                if part:
                    row[whole] = free[asked - 1]
                    self.refs[row[whole]] = 1
                    if self.inside(table[s][whole]):
                        self.copies.append((table[s][whole], row[whole], part))
                    else:
                        self.status |= svp.DEV_BAD_CONTEXT
                if s != t:
                    self.table[t] = row
                self.used[t] = whole + (part > 0)

    def compact(self):
        live = sum(r != 0 for r in self.refs)
        movers = [x for x in range(live, self.num) if self.refs[x] != 0]
        holes = [x for x in range(live) if self.refs[x] == 0]
        to = dict(zip(movers, holes))
        for i in range(self.n):
            for j in range(min(max(self.used[i], 0), self.cols)):
                page = self.table[i][j]
                if page in to:
                    self.table[i][j] = to[page]
                elif live <= page < self.num and movers:
                    self.status |= svp.DEV_BAD_CONTEXT
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
            self.copies.append((a, b, self.page))
        return live


class Device:
    """The same state on the GPU, with pools of `layers` caches."""

    def __init__(self, m, kind=BF16, hkv=2, d=64, layers=1, layout="head", seed=0):
        self.m, self.kind = m, kind
        self.table = torch.tensor(m.table, dtype=torch.int32, device="cuda").view(m.n, m.cols)
        self.used, self.refs = i32(m.used), i32(m.refs)
        self.pages = svp.make_pages(self.table, self.used, self.refs, page_size=m.page)
        g = torch.Generator().manual_seed(seed)
        size = {F32: 4, BF16: 2, E4M3: 1}[kind]
        self.pools, self.exps, self.caches, self.want, self.wexp = [], [], [], [], []
        for _ in range(layers):
            pair, epair = [], []
            for _ in range(2):
                raw = torch.randint(0, 256, (m.num, hkv, m.page, d * size), dtype=torch.uint8, generator=g)
                self.want.append(raw.clone())
                x = raw.cuda().view(kind)
                if layout == "token":
                    x = x.transpose(1, 2).contiguous().transpose(1, 2)
                if layout == "wide":          # pages apart, with other data between
                    big = torch.zeros(m.num, hkv, m.page, d + 16, dtype=kind, device="cuda")
                    big[..., :d].copy_(x) if kind != E4M3 else big.view(torch.uint8)[..., :d].copy_(x.view(torch.uint8))
                    x = big[..., :d]
                pair.append(x)
                if kind == E4M3:
                    e = torch.randint(0, 256, (m.num, hkv, m.page), dtype=torch.uint8, generator=g)
                    self.wexp.append(e.clone())
                    epair.append(e.cuda())
            self.pools += pair
            self.exps += epair
            self.caches.append(svp.make_cache(pair[0], pair[1], self.table, **(
                dict(k_exp=epair[0], v_exp=epair[1]) if kind == E4M3 else {})))

    def check(self):
        torch.cuda.synchronize()
        m = self.m
        assert self.pages.ws.read_status() == m.status
        m.status = 0
        assert self.used.tolist() == m.used
        assert self.refs.tolist() == m.refs
        assert self.table.tolist() == m.table
        for a, b, k in m.copies:
            for w in self.want:
                w[b, :, :k] = w[a, :, :k]
            for w in self.wexp:
                w[b, :, :k] = w[a, :, :k]
        m.copies = []
        for x, w in zip(self.pools, self.want):
            assert torch.equal(bytes_of(x).view(w.shape), w)
        for x, w in zip(self.exps, self.wexp):
            assert torch.equal(x.cpu(), w)


@pytest.mark.parametrize("kind,page,hkv,d,layers,layout", [
    (BF16, 16, 2, 64, 1, "head"), (E4M3, 32, 8, 128, 3, "head"), (F32, 16, 1, 256, 2, "token"), (E4M3, 128, 2, 64, 2, "token"),
    (BF16, 64, 3, 128, 1, "wide"), (E4M3, 16, 1, 64, 5, "wide")])
@pytest.mark.parametrize("seed", range(4))
def test_random_steps(kind, page, hkv, d, layers, layout, seed):
    """Requests come, grow, shrink, are forked and leave, with compactions between; the pool runs out at times."""
    r = random.Random(seed * 1000 + page + layers)
    n, cols = r.randint(3, 40), r.randint(4, 12)
    m = Model(n, cols, page, r.randint(n * 2, n * cols))
    dev = Device(m, kind, hkv, d, layers, layout, seed)
    length = [0] * n
    for step in range(25):
        op = r.choice(["resize", "resize", "fork", "fork", "compact"])
        if op == "resize":
            ask = []
            for i in range(n):
                x = r.random()
                ask.append(-1 if x < 0.3 else 0 if x < 0.4 else r.randint(0, cols * page) if x < 0.6
                           else min(cols * page + (x > 0.98), max(0, length[i] + r.randint(-page, page))))
            m.resize(ask)
            svp.pages_resize(dev.pages, i32(ask))
            length = [a if a >= 0 and m.pages(a) == u else min(x, u * page) for a, u, x in zip(ask, m.used, length)]
        elif op == "fork":
            k = r.randint(1, n)
            src = [r.randint(-1, n) if r.random() < 0.05 else r.randrange(n) for _ in range(k)]
            empty = [i for i in range(n) if m.used[i] == 0] or [0]
            dst = [r.choice(empty) if r.random() < 0.9 else r.randint(-1, n) for _ in range(k)]
            ask = [r.randint(0, max(1, length[s])) if 0 <= s < n else 5 for s in src]
            if r.random() < 0.2:
                ask[0] = r.choice([-1, cols * page + 1])
            m.fork(src, dst, ask)
            svp.pages_fork(dev.pages, i32(src), i32(dst), i32(ask), caches=dev.caches)
            length = [x if x else u * page for u, x in zip(m.used, length)]
        else:
            live = torch.zeros(1, dtype=torch.int32, device="cuda")
            want = m.compact()
            svp.pages_compact(dev.pages, caches=dev.caches, live=live)
            assert live.item() == want
        dev.check()


@pytest.mark.parametrize("num", [1, 31, 32, 33, 1023, 8192, 8193, 70000, 300000])
def test_lowest_free_pages_of_any_pool(num):
    """Free pages at the borders of warps, blocks and windows; a pool used up to its last page, and one short."""
    r = random.Random(num)
    refs = [1 if r.random() < 0.9 else 0 for _ in range(num)]
    refs[-1] = 0
    free = refs.count(0)
    cols = max(1, free)
    m = Model(2, cols + 1, 16, num, refs=refs)
    dev = Device(m, hkv=1, layers=0)
    ask = [(free // 2) * 16, (free - free // 2) * 16]
    m.resize(ask)
    svp.pages_resize(dev.pages, i32(ask))
    dev.check()
    assert m.refs.count(0) == 0
    back = [m.page, 0]
    m.resize(back)
    svp.pages_resize(dev.pages, i32(back))
    dev.check()
    ask = [16, (free + 1) * 16]                       # one page more than there is: left as it was
    m.resize(ask)
    svp.pages_resize(dev.pages, i32(ask))
    assert m.status == svp.DEV_NO_PAGES and m.used[1] == 0
    dev.check()


@pytest.mark.parametrize("num", [1, 2, 33, 8191, 8192, 8200, 70000, 300000])
@pytest.mark.parametrize("share", [0.0, 0.02, 0.5, 0.98, 1.0])
def test_compact_pools_of_any_size(num, share):
    r = np.random.default_rng(num + int(share * 100))
    refs = (r.random(num) < share).astype(np.int32)
    held = np.flatnonzero(refs)
    r.shuffle(held)
    n, cols = 7, max(1, len(held))
    cuts = np.sort(r.integers(0, len(held) + 1, n - 1))
    table, used = np.full((n, cols), -1, np.int32), []
    for i, part in enumerate(np.split(held, cuts)):
        table[i, :len(part)] = part
        used.append(len(part))
    m = Model(n, cols, 16, num, table.tolist(), used, refs.tolist())
    dev = Device(m, hkv=1, layers=1 if num <= 70000 else 0)
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    svp.pages_compact(dev.pages, caches=dev.caches, live=live)
    assert m.compact() == live.item() == len(held)
    dev.check()
    svp.pages_compact(dev.pages, caches=dev.caches, live=live)      # nothing is left to move
    m.compact()
    dev.check()


def test_pools_past_32_bits():
    """Pages whose elements lie more than 2^31 into their pools: copied by a fork, written by rope_cache_write, moved by a
    compaction, and read as a common beginning."""
    pages_n, hkv, page, d = 70000, 8, 16, 256
    pool = [torch.empty(pages_n, hkv, page, d, dtype=BF16, device="cuda") for _ in range(2)]
    assert pool[0].numel() > 2 ** 31
    refs = torch.ones(pages_n, dtype=torch.int32, device="cuda")        # others hold all but the pages at either end
    refs[:8] = refs[-20:] = 0
    table, used = torch.full((3, 8), -1, dtype=torch.int32, device="cuda"), i32([0, 0, 0])
    refs[:8] = 1
    p = svp.make_pages(table, used, refs, page_size=page)
    cache = svp.make_cache(pool[0], pool[1], table)
    svp.pages_resize(p, i32([40, 0, 0]))
    first = pages_n - 20
    assert table[0, :3].tolist() == [first, first + 1, first + 2]
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(40, h, d, generator=g, device="cuda").to(BF16) for h in (16, hkv, hkv))
    freq = svp.rope_frequencies(d)
    cu, ctx = i32([0, 40, 40, 40]), i32([0, 0, 0])
    qr, kr = svp.rope(q, k, ctx, cu, freq=freq)
    assert torch.equal(svp.rope_cache_write(q, k, v, ctx, cu, cache=cache, freq=freq), qr)
    svp.pages_fork(p, i32([0, 0]), i32([1, 2]), i32([40, 39]), caches=[cache])
    assert table[1, :3].tolist() == [first, first + 1, first + 3] and table[2, :3].tolist() == [first, first + 1, first + 4]
    for i, t in ((0, 40), (1, 40), (2, 39)):
        at = i32([0] * (i + 1) + [t] * (3 - i))
        a, b = svp.cache_read(None, at, cache=cache, rows=t)
        assert torch.equal(a, kr[:t]) and torch.equal(b, v[:t])
    # a token each, behind the two pages that they share
    rows, one = i32([0, 1, 2, 3]), i32([39, 39, 38])
    args = (qr[:3], one, rows)
    out, lse = svp.prefix_attn(*args, i32([0, 3]), i32([32]), cache=cache, w=1)
    want, wl = svp.chunk_attn(*args, cache=cache, w=1)
    assert ((out.float() - want.float()).abs() <= 4 * 2.0 ** -8 * v.float().abs().max()).all()
    assert ((lse - wl).abs() <= 2.0 ** -16 * (1 + wl.abs())).all()
    refs[1:4] = 0                                                       # three others leave
    live = i32([0])
    svp.pages_compact(p, caches=[cache], live=live)
    assert live.item() == 69980 + 5 - 3 and table[:, :3].max() < live.item() and p.ws.read_status() == 0
    moved = svp.prefix_attn(*args, i32([0, 3]), i32([32]), cache=cache, w=1)
    assert torch.equal(moved[0], out) and torch.equal(moved[1], lse)


def test_many_requests_and_forks():
    n, cols, page = 1024, 9, 16
    m = Model(n, cols, page, 9000)
    dev = Device(m, hkv=1)
    ask = [100 if i % 2 == 0 else 0 for i in range(n)]
    m.resize(ask)
    svp.pages_resize(dev.pages, i32(ask))
    dev.check()
    src = [2 * (f % 37) for f in range(512)]
    dst = [2 * f + 1 for f in range(512)]
    length = [f % 101 for f in range(512)]
    m.fork(src, dst, length)
    svp.pages_fork(dev.pages, i32(src), i32(dst), i32(length), caches=dev.caches)
    dev.check()
    ask = [0 if i % 3 else -1 for i in range(n)]
    m.resize(ask)
    svp.pages_resize(dev.pages, i32(ask))
    dev.check()
    m.compact()
    svp.pages_compact(dev.pages, caches=dev.caches)
    dev.check()


def test_shared_parts_of_pages_are_not_kept():
    """A request that would keep part of a page that another holds is left as it was, whatever the other does in the
    same call; with a whole page less it shrinks."""
    m = Model(3, 6, 16, 20)
    dev = Device(m)
    for ask in ([80, 0, 0],):
        m.resize(ask)
        svp.pages_resize(dev.pages, i32(ask))
    m.fork([0, 0], [1, 2], [64, 70])
    svp.pages_fork(dev.pages, i32([0, 0]), i32([1, 2]), i32([64, 70]), caches=dev.caches)
    dev.check()
    for ask, bits in (([40, 0, -1], svp.DEV_BAD_CONTEXT), ([-1, -1, 0], 0), ([33, -1, -1], 0), ([32, -1, -1], 0)):
        m.resize(ask)
        svp.pages_resize(dev.pages, i32(ask))
        assert m.status == bits
        dev.check()


def test_rewound_behind_a_fork_is_reported():
    """A request forked at a page's end and then taken back into that page, with as many pages as before: its next
    write would go where its forks read, which is reported as a shrinking into a shared page is."""
    m = Model(3, 6, 16, 20)
    dev = Device(m)
    m.resize([64, 32, 0])
    svp.pages_resize(dev.pages, i32([64, 32, 0]))
    m.fork([0], [2], [64])
    svp.pages_fork(dev.pages, i32([0]), i32([2]), i32([64]), caches=dev.caches)
    dev.check()
    for ask, bits in (([64, 20, 64], 0), ([60, -1, -1], svp.DEV_BAD_CONTEXT), ([-1, -1, 49], svp.DEV_BAD_CONTEXT),
                      ([65, -1, 64], 0), ([60, -1, 0], svp.DEV_BAD_CONTEXT), ([60, -1, -1], 0), ([52, -1, 0], 0)):
        m.resize(ask)
        svp.pages_resize(dev.pages, i32(ask))
        assert m.status == bits
        dev.check()


def test_broken_tables_are_reported_and_stay_inside_the_pool():
    m = Model(4, 4, 16, 10, table=[[0, 1, 99, -7], [2, 3, -1, -1], [4, -1, -1, -1], [-1] * 4], used=[4, 9, 1, 0],
              refs=[1, 1, 1, 1, 0, 0, 0, 0, 0, 0])
    dev = Device(m)
    m.fork([0, 1], [3, 2], [64, 10])                       # page ids outside, a request whose count is none
    svp.pages_fork(dev.pages, i32([0, 1]), i32([3, 2]), i32([64, 10]), caches=dev.caches)
    assert m.status == svp.DEV_BAD_CONTEXT | svp.DEV_BAD_SLOTS
    dev.check()
    ask = [0, 0, 0, 0]                                     # one page that nobody counted
    m.resize(ask)
    svp.pages_resize(dev.pages, i32(ask))
    assert m.status == svp.DEV_BAD_CONTEXT
    dev.check()
    m2 = Model(2, 3, 16, 10, table=[[0, 9, 8], [7, -1, -1]], used=[3, 5], refs=[1, 0, 0, 0, 0, 0, 0, 1, 1, 0])
    dev2 = Device(m2)                                      # page 9 is held but free by its count
    m2.compact()
    svp.pages_compact(dev2.pages, caches=dev2.caches)
    assert m2.status == svp.DEV_BAD_CONTEXT
    dev2.check()


def test_no_pages_no_requests():
    m = Model(2, 0, 16, 5)
    dev = Device(m, layers=0)
    svp.pages_resize(dev.pages, i32([0, 3]))
    m.resize([0, 3])
    dev.check()
    svp.pages_fork(dev.pages, i32([]), i32([]), i32([]))
    svp.pages_compact(dev.pages)
    dev.check()
    m = Model(1, 4, 16, 0)
    dev = Device(m, layers=0)
    svp.pages_resize(dev.pages, i32([5]))
    m.resize([5])
    dev.check()
    svp.pages_compact(dev.pages, caches=dev.caches)
    dev.check()


def test_captured_and_replayed():
    """One graph of a step's calls, replayed while the lengths and the forks change."""
    n, cols, page = 8, 8, 16
    m = Model(n, cols, page, 64)
    dev = Device(m, E4M3, layers=2)
    length, src, dst, flen = i32([0] * n), i32([0, 0]), i32([6, 7]), i32([0, 0])
    done = i32([-1] * n)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        svp.pages_resize(dev.pages, length)
        svp.pages_fork(dev.pages, src, dst, flen, caches=dev.caches)
        svp.pages_resize(dev.pages, done)
        svp.pages_compact(dev.pages, caches=dev.caches)
    r = random.Random(3)
    for _ in range(12):
        ask = [r.randint(0, 100) if i < 6 else -1 for i in range(n)]
        f = [r.randrange(6), r.randrange(6)]
        k = [r.randint(0, max(0, ask[x])) for x in f]
        end = [-1] * 6 + [0, 0]
        for t, x in ((length, ask), (src, f), (flen, k), (done, end)):
            t.copy_(i32(x))
        g.replay()
        m.resize(ask)
        m.fork(f, [6, 7], k)
        m.resize(end)
        m.compact()
        dev.check()


def test_other_stream():
    m = Model(3, 4, 16, 12)
    dev = Device(m)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ask = i32([40, 0, 20])
    torch.cuda.synchronize()
    svp.pages_resize(dev.pages, ask, stream=side)
    svp.pages_compact(dev.pages, caches=dev.caches, stream=side)
    side.synchronize()
    m.resize([40, 0, 20])
    m.compact()
    dev.check()


def test_binding_refusals():
    m = Model(2, 4, 16, 8)
    dev, other = Device(m), Device(Model(2, 4, 16, 8))
    with pytest.raises(ValueError):
        svp.pages_resize(dev.pages, i32([1]))
    with pytest.raises(ValueError):
        svp.pages_resize(dev.pages, i32([1, 2]).long())
    with pytest.raises(ValueError):
        svp.pages_fork(dev.pages, i32([0]), i32([1, 1]), i32([3]))
    with pytest.raises(ValueError):
        svp.pages_compact(dev.pages, caches=other.caches)          # another table's cache
    with pytest.raises(ValueError):
        svp.pages_compact(dev.pages, live=i32([0, 0]))
    with pytest.raises(ValueError):
        svp.make_pages(dev.table, dev.refs, dev.used, page_size=16)
    with pytest.raises(svp.SvpError):
        svp.make_pages(dev.table, dev.used, dev.refs, page_size=24)
