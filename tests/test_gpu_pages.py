"""Copying, forking, freeing and compacting pages, against plain loops on the host."""
import pytest
import torch

from fp8_mla_kv_gb300 import mlasparse as M

pytestmark = pytest.mark.gpu
D = "cuda:0"


class Host:
    """The pool as plain Python, page by page."""

    def __init__(self, cache, page, refs, table):
        self.cache, self.page, self.refs, self.table = cache.clone(), page, refs.tolist(), table.tolist()

    def rows(self, p):
        return self.cache[p * self.page:(p + 1) * self.page]

    def free(self, rows):
        for r in rows:
            if not 0 <= r < len(self.table):
                continue
            for k, p in enumerate(self.table[r]):
                if 0 < p < len(self.refs) and self.refs[p] > 0:
                    self.refs[p] -= 1
                self.table[r][k] = -1

    def fork(self, parent, child, lens):
        width = len(self.table[0])
        todo = []
        vacant = [p for p in range(1, len(self.refs)) if self.refs[p] == 0]
        for p, c, n in zip(parent, child, lens):
            if not (0 <= p < len(self.table) and 0 <= c < len(self.table)) or p == c or not 0 <= n <= width * self.page:
                continue
            whole, rest = divmod(n, self.page)
            row = [e if e < len(self.refs) else -1 for e in self.table[p][:whole]]
            for e in row:
                if e > 0:
                    self.refs[e] += 1
            part = self.table[p][whole] if rest else -1
            row += [-1] * (width - whole)
            if 0 < part < len(self.refs):
                todo.append((c, whole, rest, part))
            self.table[c] = row
        for c, whole, rest, part in todo:
            if not vacant:
                continue
            new = vacant.pop(0)
            self.rows(new)[:rest] = self.rows(part)[:rest].clone()
            self.table[c][whole] = new
            self.refs[new] = 1

    def compact(self):
        P = len(self.refs)
        live = [p for p in range(1, P) if self.refs[p] > 0]
        n = len(live)
        low = [p for p in range(1, n + 1) if self.refs[p] <= 0]
        to = {p: p for p in live}
        to.update(dict(zip([p for p in live if p > n], low)))
        refs = [self.refs[0]] + [self.refs[p] if self.refs[p] <= 0 else 0 for p in range(1, P)]
        for p in live:
            refs[to[p]] = self.refs[p]
            if to[p] != p:
                self.rows(to[p])[:] = self.rows(p).clone()
        # a page whose count is negative or zero keeps that count, unless a live page moved there
        self.refs = refs
        self.table = [[(0 if e == 0 else to.get(e, -1)) if e >= 0 else e for e in r] for r in self.table]
        return [0] + [to.get(p, -1) for p in range(1, P)]


def pool(P, page, rows, width, live, row_bytes, seed, spare=0):
    g = torch.Generator().manual_seed(seed)
    cache = torch.randint(0, 256, (P * page + spare, row_bytes), generator=g, dtype=torch.uint8)
    order = (torch.randperm(P - 1, generator=g) + 1)[:live]
    table = torch.full((rows * width,), -1, dtype=torch.int32)
    at = torch.randperm(rows * width, generator=g)[:live]
    table[at] = order[:at.numel()].to(torch.int32)
    refs = torch.zeros(P, dtype=torch.int32)
    refs[table[table >= 0].long()] = 1
    return cache, refs, table.view(rows, width)


def same(h, cache, refs, table):
    torch.cuda.synchronize()
    assert refs.cpu().tolist() == h.refs
    assert table.cpu().tolist() == h.table
    assert torch.equal(cache.cpu(), h.cache)


@pytest.mark.parametrize("page,row,n", [(1, 656, 1), (1, 528, 37), (16, 656, 5), (64, 528, 60), (64, 656, 300), (7, 656, 90)])
def test_copy(page, row, n):
    P = 400
    g = torch.Generator().manual_seed(n)
    a = torch.randint(0, 256, (P * page + 3, row), generator=g, dtype=torch.uint8)
    b = torch.randint(0, 256, (P * page, row), generator=g, dtype=torch.uint8)
    src = torch.randint(0, P, (n,), generator=g).to(torch.int32)
    dst = (torch.randperm(P - 1, generator=g)[:n] + 1).to(torch.int32)
    if n > 4:
        src[1], dst[2], dst[3] = -1, -1, 0
    want = b.clone()
    for s, d in zip(src.tolist(), dst.tolist()):
        if s >= 0 and d > 0:
            want[d * page:(d + 1) * page] = a[s * page:(s + 1) * page]
    da, db = a.to(D), b.to(D)
    M.mla_page_copy(db, da, page, dst.to(D), src.to(D))
    torch.cuda.synchronize()
    assert M.mla_get_error() == 0
    assert torch.equal(db.cpu(), want) and torch.equal(da.cpu(), a)


def test_copy_within_a_cache_and_out_of_range():
    page, P = 16, 20
    a = torch.randint(0, 256, (P * page + 15, 656), dtype=torch.uint8)
    d = a.to(D)
    # page 20 is not whole, page 99 is past the cache: both dropped and flagged
    M.mla_page_copy(d, d, page, torch.tensor([3, 20, 5], dtype=torch.int32, device=D),
                    torch.tensor([7, 1, 99], dtype=torch.int32, device=D))
    assert M.mla_get_error() == M.MLA_ERR_PAGE_RANGE
    want = a.clone()
    want[48:64] = a[112:128]
    assert torch.equal(d.cpu(), want)


@pytest.mark.parametrize("P,page,rows,width,live,row", [(9, 1, 3, 4, 6, 656), (300, 16, 20, 9, 120, 528),
                                                        (5000, 4, 40, 60, 1500, 656), (2049, 2, 5, 300, 1400, 656)])
def test_free_fork_compact_in_turn(P, page, rows, width, live, row):
    cache, refs, table = pool(P, page, rows, width, live, row, seed=P, spare=page - 1)
    h = Host(cache, page, refs, table)
    d_cache, d_refs, d_table = cache.to(D), refs.to(D), table.to(D)
    g = torch.Generator().manual_seed(P + 1)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=D)  # noqa: E731
    for step in range(4):
        drop = torch.randperm(rows, generator=g)[: max(1, rows // 2)].tolist() 
        drop = drop + [drop[0], -1]                                     # a row twice, and none
        M.mla_page_free(d_refs, d_table, ints(drop))
        h.free(drop)
        same(h, d_cache, d_refs, d_table)
        kept = [r for r in range(rows) if r not in drop]
        child = [r for r in drop[:-2]]
        parent = [kept[int(torch.randint(0, len(kept), (1,), generator=g))] for _ in child] if kept else []
        child = child[:len(parent)]
        lens = [int(torch.randint(0, width * page + 1, (1,), generator=g)) for _ in child]
        if len(child) > 2:
            lens[0], lens[1], parent[2] = 0, width * page, -1
        M.mla_page_fork(d_cache, page, d_refs, d_table, ints(parent), ints(child), ints(lens))
        h.fork(parent, child, lens)
        assert (M.mla_get_error() & ~M.MLA_ERR_POOL_EMPTY) == 0
        same(h, d_cache, d_refs, d_table)
        # out of place first: what goes in stays
        before_r, before_t = d_refs.clone(), d_table.clone()
        ro, to, pm = torch.empty_like(d_refs), torch.empty_like(d_table), torch.empty_like(d_refs)
        keep = d_cache.clone()
        M.mla_page_compact(d_cache, page, d_refs, d_table, refcount_out=ro, table_out=to, page_map=pm)
        assert torch.equal(before_r, d_refs) and torch.equal(before_t, d_table)
        d_cache.copy_(keep)
        M.mla_page_compact(d_cache, page, d_refs, d_table)
        want_map = h.compact()
        same(h, d_cache, d_refs, d_table)
        assert torch.equal(ro, d_refs) and torch.equal(to, d_table) and pm.cpu().tolist() == want_map
        n = sum(v > 0 for v in h.refs[1:])
        assert all(v > 0 for v in h.refs[1:n + 1])
    assert M.mla_get_error() == 0


def test_fork_when_the_pool_runs_out():
    page, P = 8, 6
    cache = torch.randint(0, 256, (P * page, 656), dtype=torch.uint8)
    table = torch.full((5, 3), -1, dtype=torch.int32)
    table[0, :2] = torch.tensor([2, 4])
    refs = torch.tensor([0, 0, 1, 1, 1, 0], dtype=torch.int32)      # free: 1 and 5
    h = Host(cache, page, refs, table)
    dc, dr, dt = cache.to(D), refs.to(D), table.to(D)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=D)  # noqa: E731
    M.mla_page_fork(dc, page, dr, dt, ints([0, 0, 0]), ints([1, 2, 3]), ints([13, 9, 12]))
    h.fork([0, 0, 0], [1, 2, 3], [13, 9, 12])
    assert M.mla_get_error() == M.MLA_ERR_POOL_EMPTY
    same(h, dc, dr, dt)
    assert dt[3].tolist() == [2, -1, -1]


def test_a_last_page_that_cannot_be_copied():
    page, P = 8, 6
    cache = torch.randint(0, 256, (P * page, 656), dtype=torch.uint8)
    table = torch.tensor([[0, 3], [2, 0], [4, 9], [-1, -1], [-1, -1], [-1, -1]], dtype=torch.int32)
    refs = torch.tensor([0, 0, 1, 1, 1, 0], dtype=torch.int32)
    h = Host(cache, page, refs, table)
    dc, dr, dt = cache.to(D), refs.to(D), table.to(D)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=D)  # noqa: E731
    M.mla_page_fork(dc, page, dr, dt, ints([0, 1]), ints([3, 4]), ints([15, 15]))       # page 0 whole, then as the last one
    h.fork([0, 1], [3, 4], [15, 15])
    assert M.mla_get_error() == 0
    same(h, dc, dr, dt)
    assert dt[3].tolist() == [0, 1] and dt[4].tolist() == [2, -1]
    M.mla_page_fork(dc, page, dr, dt, ints([2]), ints([5]), ints([9]))                  # page 9 does not exist
    h.fork([2], [5], [9])
    assert M.mla_get_error() == M.MLA_ERR_PAGE_RANGE
    same(h, dc, dr, dt)
    assert dt[5].tolist() == [4, -1]


def test_bad_rows_pages_and_counts_are_flagged():
    page, P = 8, 6
    cache = torch.randint(0, 256, (P * page, 656), dtype=torch.uint8).to(D)
    keep = cache.clone()
    table = torch.tensor([[1, 9], [3, -1], [-1, -1]], dtype=torch.int32, device=D)
    refs = torch.tensor([0, 1, 0, 0, 0, 0], dtype=torch.int32, device=D)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=D)  # noqa: E731
    M.mla_page_fork(cache, page, refs, table, ints([0, 7, 0, 0]), ints([0, 2, 9, 2]), ints([8, 8, 8, 17]))
    assert M.mla_get_error() == M.MLA_ERR_PAGE_RANGE
    assert table.tolist() == [[1, 9], [3, -1], [-1, -1]] and refs.tolist() == [0, 1, 0, 0, 0, 0]
    M.mla_page_free(refs, table, ints([5]))
    assert M.mla_get_error() == M.MLA_ERR_PAGE_RANGE
    M.mla_page_free(refs, table, ints([1]))                 # page 3 had no count
    assert M.mla_get_error() == M.MLA_ERR_PAGE_COUNT
    M.mla_page_free(refs, table, ints([0]))                 # page 9 does not exist
    assert M.mla_get_error() == M.MLA_ERR_PAGE_RANGE
    assert refs.tolist() == [0] * 6 and (table == -1).all()
    table = torch.tensor([[9, 2, 0]], dtype=torch.int32, device=D)
    refs = torch.tensor([0, 0, 1, 0, 0, 0], dtype=torch.int32, device=D)
    M.mla_page_compact(cache, page, refs, table)
    assert M.mla_get_error() == M.MLA_ERR_PAGE_RANGE
    assert table.tolist() == [[-1, 1, 0]] and refs.tolist() == [0, 1, 0, 0, 0, 0]
    keep[8:16] = keep[16:24]
    assert torch.equal(cache, keep)


@pytest.mark.parametrize("P,live", [(4096, 0), (4096, 1), (4096, 4095), (4096, 2048), (1, 0), (2, 1), (31, 12), (33, 32),
                                    (65536, 30000), (65537, 65536), (150001, 70000), (70000, 1)])
def test_compact_at_the_ends(P, live):
    """The live pages last in the pool; up to 65,536 pages are planned by one CTA."""
    page = 1
    cache = torch.randint(0, 256, (P, 528), dtype=torch.uint8)
    refs = torch.zeros(P, dtype=torch.int32)
    if live:
        refs[-live:] = torch.arange(1, live + 1, dtype=torch.int32)
    table = torch.arange(P, dtype=torch.int32).view(1, P)
    h = Host(cache, page, refs, table)
    dc, dr, dt = cache.to(D), refs.to(D), table.to(D)
    M.mla_page_compact(dc, page, dr, dt)
    h.compact()
    same(h, dc, dr, dt)


def test_pages_in_a_graph():
    P, page, rows, width = 600, 16, 12, 10
    cache, refs, table = pool(P, page, rows, width, 60, 656, seed=4)
    dc, dr, dt = cache.to(D), refs.to(D), table.to(D)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=D)  # noqa: E731
    rows_t, parent, child, lens = ints([6, 7, 8]), ints([0, 0, 1]), ints([6, 7, 8]), ints([100, 37, 159])
    ws = M.alloc_page_workspace(P, 3)
    ws.fill_(0xFF)
    gr = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(gr):
        M.mla_page_free(dr, dt, rows_t)
        M.mla_page_fork(dc, page, dr, dt, parent, child, lens, workspace=ws)
        M.mla_page_compact(dc, page, dr, dt, workspace=ws)
    h = Host(cache, page, refs, table)
    for _ in range(3):
        gr.replay()
        h.free([6, 7, 8])
        h.fork([0, 0, 1], [6, 7, 8], [100, 37, 159])
        h.compact()
        same(h, dc, dr, dt)
    assert M.mla_get_error() == 0


def test_nothing_to_do():
    cache = torch.zeros((64, 656), dtype=torch.uint8, device=D)
    refs, table = torch.zeros(4, dtype=torch.int32, device=D), torch.full((2, 2), -1, dtype=torch.int32, device=D)
    none = torch.empty(0, dtype=torch.int32, device=D)
    M.mla_page_copy(cache, cache, 16, none, none)
    M.mla_page_free(refs, table, none)
    M.mla_page_fork(cache, 16, refs, table, none, none, none)
    M.mla_page_compact(cache, 16, refs, table)
    M.mla_page_compact(cache, 16, refs, table[:0])
    assert M.mla_get_error() == 0 and (cache == 0).all() and (refs == 0).all() and (table == -1).all()
