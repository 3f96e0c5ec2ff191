"""What the pages' calls report and leave alone when a table holds entries that name no page, or a page that nobody
counts, against the model of test_gpu_pages with those rules as svp.h states them."""
import pytest
import torch

import speculative_decoding_verification_packed_gb300 as svp
from test_gpu_cache import BF16, E4M3, F32, i32
from test_gpu_pages import Device, Model

pytestmark = pytest.mark.gpu


class Stated(Model):
    def fork(self, src, dst, length):
        """A part of a page whose entry names none is passed on as -1, and takes no page."""
        used, table = list(self.used), [list(r) for r in self.table]
        free = [x for x in range(self.num) if self.refs[x] == 0]
        asked = 0
        for s, t, k in zip(src, dst, length):
            assert 0 <= s < self.n and 0 <= t < self.n and used[t] == 0 and 0 <= k <= used[s] * self.page
            assert dst.count(t) == 1 and s != t
            whole, part = k // self.page, k % self.page
            lost = part > 0 and not self.inside(table[s][whole])
            asked += part > 0 and not lost
            if asked > len(free):
                self.status |= svp.DEV_NO_PAGES
                continue
            row = [-1] * self.cols
            for j in range(whole):
                if self.inside(table[s][j]):
                    row[j] = table[s][j]
                    self.refs[row[j]] += 1
                else:
                    self.status |= svp.DEV_BAD_CONTEXT
            if lost:
                self.status |= svp.DEV_BAD_CONTEXT
            elif part:
                row[whole] = free[asked - 1]
                self.refs[row[whole]] = 1
                self.copies.append((table[s][whole], row[whole], part))
            self.table[t] = row
            self.used[t] = whole + (part > 0)


@pytest.mark.parametrize("kind,layers", [(BF16, 0), (BF16, 1), (E4M3, 3), (F32, 2)])
@pytest.mark.parametrize("bad", [-1, 12, 1 << 30, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("spare", [0, 1, 2, 3])
def test_a_fork_of_a_part_whose_entry_names_no_page(bad, kind, layers, spare):
    """Forks with such a part first, between and last, beside sound ones whose pages they must not take; `spare` of the
    two pages that those need (and one more) are free."""
    table = [[0, 1, 2, 3], [4, 5, bad, -1], [bad, -1, -1, -1], [-1] * 4, [-1] * 4, [-1] * 4, [-1] * 4, [-1] * 4, [-1] * 4]
    refs = [1] * 6 + [0] * 6
    for x in range(11, 5 + spare, -1):
        refs[x] = 1                        # (held by others)
    m = Stated(9, 4, 16, 12, table=table, used=[4, 3, 1, 0, 0, 0, 0, 0, 0], refs=refs)
    dev = Device(m, kind, layers=layers)
    src, dst, length = [1, 0, 2, 0, 1, 1], [3, 4, 5, 6, 7, 8], [33, 50, 7, 20, 47, 32]
    m.fork(src, dst, length)
    assert m.status & svp.DEV_BAD_CONTEXT and bool(m.status & svp.DEV_NO_PAGES) == (spare < 2)
    assert m.table[3] == [4, 5, -1, -1] and m.used[3] == 3
    svp.pages_fork(dev.pages, i32(src), i32(dst), i32(length), caches=dev.caches)
    dev.check()
    # given back: the entries that name nothing are reported, the pages come back
    back = [-1, -1, -1] + [0] * 6
    m.resize(back)
    svp.pages_resize(dev.pages, i32(back))
    dev.check()
    assert m.refs == refs


def test_such_forks_alone_take_no_page():
    """No free page at all, and none is needed."""
    m = Stated(3, 3, 32, 2, table=[[0, 7, -1], [-1] * 3, [-1] * 3], used=[2, 0, 0], refs=[1, 1])
    dev = Device(m)
    m.fork([0, 0], [1, 2], [40, 63])
    assert m.status == svp.DEV_BAD_CONTEXT and m.table[1] == m.table[2] == [0, -1, -1]
    svp.pages_fork(dev.pages, i32([0, 0]), i32([1, 2]), i32([40, 63]), caches=dev.caches)
    dev.check()


@pytest.mark.parametrize("num", [12, 40, 8200])
@pytest.mark.parametrize("moved", [False, True])
@pytest.mark.parametrize("stale", [True, False])
def test_an_entry_of_a_page_that_nobody_counts_is_reported_by_a_compaction(num, moved, stale):
    """Whether other pages move or the pool is compact already; it stays as it is."""
    last = num - 1
    refs = [1, 1, 1, 0] + [0] * (num - 4)
    table = [[0, 1, -1, -1], [2, -1, -1, -1]]
    if moved:                              # page 1 free, page 5 in use: it moves
        refs[1], refs[5], table[0][1] = 0, 1, 5
    if stale:
        table[1][1] = last
    m = Model(2, 4, 16, num, table=table, used=[2, 2 if stale else 1], refs=refs)
    dev = Device(m, layers=1)
    live = i32([-5])
    svp.pages_compact(dev.pages, caches=dev.caches, live=live)
    assert m.compact() == live.item() == 3
    assert m.table == [[0, 1, -1, -1], [2, last if stale else -1, -1, -1]]
    m.status = svp.DEV_BAD_CONTEXT if stale else 0
    dev.check()


def test_a_pool_without_a_free_page_has_nothing_to_report():
    m = Model(2, 3, 16, 4, table=[[3, 0, -1], [1, 2, 99]], used=[2, 3], refs=[1, 1, 1, 1])
    dev = Device(m)
    m.compact()
    svp.pages_compact(dev.pages, caches=dev.caches)
    assert m.status == 0                   # (an id that is no page's is not the compaction's affair)
    dev.check()
