"""Pages of the paged cache: random lives of sequences against a model of lists, and what reserve, fork, release, compact and
copy_pages promise one by one.  Everything is exact: page numbers, counts and copied bits."""
import random

import pytest
import torch

import long_context_sparse_dsa_gb300 as dsa
from test_gpu_decode import DEV, _built, _dt  # noqa: F401
from test_gpu_decode_contract import _reports

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class World:
    """A cache with its counts on the GPU, and the same as lists."""

    def __init__(self, pages, page, L, dtype="bf16", d=64, di=64, seed=0):
        self.page, self.pages, self.L = page, pages, L
        self.cols = -(-L // page)
        self.dims = dsa.make_dims(L, 4, d, 4, di, 8, dtype=dtype)
        g = torch.Generator(device=DEV).manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device=DEV).to(_dt(dtype))  # noqa: E731
        self.cache = dsa.PagedCache(k=r(pages, page, d), v=r(pages, page, d), kpool=r(pages, page // 4, di), ktail=r(pages, 3, di))
        self.refs = _i32([0] * pages)
        self.m_refs = [0] * pages
        self.copy = {x: getattr(self.cache, x).clone() for x in ("k", "v", "kpool", "ktail")}

    def held(self, n):
        return -(-n // self.page)

    def ws(self, rows):
        return torch.full((dsa.page_workspace_bytes(self.dims, self.cache, rows),), 0xFF, dtype=torch.uint8, device=DEV)

    def m_reserve(self, lens, new, table):
        """The model; returns what is missing."""
        ask = []
        for b, (n, m) in enumerate(zip(lens, new)):
            if m <= n:
                continue
            if n % self.page and self.m_refs[table[b][n // self.page]] > 1:
                ask.append((b, n // self.page, True))
            ask += [(b, c, False) for c in range(self.held(n), self.held(m))]
        free = [p for p, c in enumerate(self.m_refs) if c == 0]
        if len(ask) > len(free):
            return len(ask) - len(free)
        for (b, c, cow), p in zip(ask, free):
            if cow:
                old, part = table[b][c], lens[b] % self.page
                for x, rows in (("k", part), ("v", part), ("kpool", part // 4), ("ktail", 3)):
                    self.copy[x][p, :rows] = self.copy[x][old, :rows]
                self.m_refs[old] -= 1
            table[b][c] = p
            self.m_refs[p] = 1
        return 0

    def same(self, table, m_table):
        dsa.check_device_error()
        assert self.refs.tolist() == self.m_refs
        assert table.tolist() == m_table
        for x, y in self.copy.items():
            assert torch.equal(getattr(self.cache, x), y), x


@pytest.mark.parametrize("pages,page,L,rows,dtype", [(60, 4, 64, 5, "bf16"), (40, 20, 200, 7, "fp32"), (5000, 16, 4000, 40, "bf16"),
                                                      (300, 64, 1000, 12, "bf16"), (150000, 4, 3000, 200, "bf16")])
def test_lives_of_sequences(pages, page, L, rows, dtype):
    """Growing, forking, cutting back, ending and compacting in random order."""
    w = World(pages, page, L, dtype=dtype, seed=pages)
    r = random.Random(pages)
    lens, m_table = [0] * rows, [[-1] * w.cols for _ in range(rows)]
    table = _i32(m_table)
    missing, seen = _i32([0]), set()
    for step in range(24 if pages < 100000 else 8):
        what = r.choice(["grow", "grow", "fork", "cut", "compact"]) if step > 1 else "grow"
        if what == "grow":
            new = [min(L, n + r.choice([0, 1, 3, page, 5 * page + 2, L // 4])) for n in lens]
            missing.fill_(-1)
            dsa.cache_reserve(w.dims, w.cache, w.refs, _i32(lens), _i32(new), table, missing, w.ws(rows))
            short = w.m_reserve(lens, new, m_table)
            assert missing.item() == short
            seen.add("short" if short else "grown")
            if not short:
                lens = new
        elif what == "fork":
            par = [r.randint(-1, rows - 1) for _ in range(rows)]
            l2, t2 = _i32([9] * rows), torch.full((rows, w.cols), 9, dtype=torch.int32, device=DEV)
            dsa.cache_fork(w.dims, w.cache, w.refs, _i32(lens), table, _i32(par), l2, t2)
            dsa.cache_release(w.dims, w.cache, w.refs, _i32(lens), table)
            new_lens = [lens[p] if p >= 0 else 0 for p in par]
            new_table = [[m_table[p][c] if p >= 0 and c < w.held(lens[p]) else -1 for c in range(w.cols)] for p in par]
            for row in new_table:
                for p in row:
                    if p >= 0:
                        w.m_refs[p] += 1
            for n, row in zip(lens, m_table):
                for c in range(w.held(n)):
                    w.m_refs[row[c]] -= 1
            assert torch.all(table == -1) and l2.tolist() == new_lens
            lens, m_table, table = new_lens, new_table, t2
        elif what == "cut":
            keep = [r.randint(0, n + 5) // 4 * 4 for n in lens]
            dsa.cache_release(w.dims, w.cache, w.refs, _i32(lens), table, keep=_i32(keep))
            for b, (n, m) in enumerate(zip(lens, keep)):
                for c in range(w.held(m), w.held(n)):
                    w.m_refs[m_table[b][c]] -= 1
                    m_table[b][c] = -1
            lens = [min(n, m) for n, m in zip(lens, keep)]
        else:
            remap, used = torch.full((pages,), 9, dtype=torch.int32, device=DEV), _i32([-1])
            dsa.cache_compact(w.dims, w.cache, w.refs, _i32(lens), table, remap, used, w.ws(rows))
            n = sum(c > 0 for c in w.m_refs)
            src = [p for p in range(n, pages) if w.m_refs[p]]
            dst = [p for p in range(n) if not w.m_refs[p]]
            to = [p if c else -1 for p, c in enumerate(w.m_refs)]
            for a, b in zip(src, dst):
                to[a], w.m_refs[b], w.m_refs[a] = b, w.m_refs[a], 0
            for x in w.copy.values():
                x[dst] = x[src]
            m_table = [[to[p] if p >= 0 else -1 for p in row] for row in m_table]
            assert used.item() == n and remap.tolist() == to
        w.same(table, m_table)
    assert "grown" in seen


def test_all_or_nothing():
    w = World(10, 16, 256, seed=1)
    table = _i32([[-1] * 16] * 3)
    missing = _i32([5])
    ws = w.ws(3)
    dsa.cache_reserve(w.dims, w.cache, w.refs, _i32([0, 0, 0]), _i32([100, 60, 1]), table, missing, ws)   # 7 + 4 + 1 pages
    assert missing.item() == 2 and torch.all(table == -1) and torch.all(w.refs == 0)
    dsa.cache_reserve(w.dims, w.cache, w.refs, _i32([0, 0, 0]), _i32([80, 60, 1]), table, missing, ws)    # 5 + 4 + 1
    assert missing.item() == 0 and table[:, :5].tolist() == [[0, 1, 2, 3, 4], [5, 6, 7, 8, -1], [9, -1, -1, -1, -1]]
    # a copy counts as a request: the branch of row 2 finds no page
    l2, t2 = _i32([0]), _i32([[0] * 16])
    dsa.cache_fork(w.dims, w.cache, w.refs, _i32([80, 60, 1]), table, _i32([2]), l2, t2)
    dsa.cache_reserve(w.dims, w.cache, w.refs, l2, _i32([2]), t2, missing, w.ws(1))
    assert missing.item() == 1 and t2[0, 0] == 9 and w.refs[9] == 2
    dsa.check_device_error()


def test_bad_rows_are_skipped_and_reported():
    w = World(12, 16, 64, seed=2)
    missing = _i32([0])
    base = [[0, 1, -1, -1], [2, 12, -1, -1], [3, -1, -1, -1]]
    refs = [1, 2, 2, 2] + [0] * 8
    # row 0 of bad length; row 1's next token on a bad page; row 2 sound, its page shared
    table = _i32(base)
    w.refs.copy_(_i32(refs))
    dsa.cache_reserve(w.dims, w.cache, w.refs, _i32([65, 20, 5]), _i32([66, 40, 33]), table, missing, w.ws(3))
    _reports(dsa.DSA_ERR_BAD_PAGE)
    assert table.tolist() == [base[0], base[1], [4, 5, 6, -1]] and missing.item() == 0
    assert w.refs.tolist() == [1, 2, 2, 1, 1, 1, 1] + [0] * 5
    # a new length out of range
    table = _i32(base)
    w.refs.copy_(_i32(refs))
    dsa.cache_reserve(w.dims, w.cache, w.refs, _i32([20, 16, 5]), _i32([65, -1, 6]), table, missing, w.ws(3))
    _reports(dsa.DSA_ERR_BAD_PAGE)
    assert table.tolist() == [base[0], base[1], [4, -1, -1, -1]]
    # release: a page without a count, a page that is not there, a bad length, a negative keep
    table = _i32(base + [[4, 0, -1, -1]])
    w.refs.copy_(_i32(refs))
    dsa.cache_release(w.dims, w.cache, w.refs, _i32([-1, 32, 5, 32]), table, keep=_i32([0, 0, -4, 0]))
    _reports(dsa.DSA_ERR_BAD_PAGE)
    assert w.refs.tolist() == [0, 2, 1, 2] + [0] * 8
    assert table.tolist() == [base[0], [-1] * 4, base[2], [-1] * 4]
    # fork: a parent that is not there, a bad page, a bad length
    w.refs.copy_(_i32(refs))
    l2, t2 = _i32([9] * 4), _i32([[9] * 4] * 4)
    dsa.cache_fork(w.dims, w.cache, w.refs, _i32([100, 20, 5]), _i32(base), _i32([0, 1, 3, 2]), l2, t2)
    with pytest.raises(dsa.DSAError):
        dsa.check_device_error()
    assert l2.tolist() == [0, 20, 0, 5] and t2.tolist() == [[-1] * 4, [2, -1, -1, -1], [-1] * 4, [3, -1, -1, -1]]
    assert w.refs.tolist() == [1, 2, 3, 3] + [0] * 8
    # compact: a row that names a free page, and one that is not there
    w.refs.copy_(_i32([1, 0, 1, 1] + [0] * 7 + [1]))
    table = _i32([[11, 0, -1, -1], [2, 12, -1, -1], [3, 1, -1, -1]])
    remap, used = _i32([0] * 12), _i32([0])
    dsa.cache_compact(w.dims, w.cache, w.refs, _i32([30, 30, 30]), table, remap, used, w.ws(3))
    _reports(dsa.DSA_ERR_BAD_PAGE)
    assert table.tolist() == [[1, 0, -1, -1], [2, -1, -1, -1], [3, -1, -1, -1]] and used.item() == 4
    assert remap.tolist() == [0, -1, 2, 3] + [-1] * 7 + [1] and w.refs.tolist() == [1] * 4 + [0] * 8


@pytest.mark.parametrize("pages", [1, 1023, 1024, 1025, 4096 + 7])
@pytest.mark.parametrize("fill", ["none", "all", "last", "odd", "front"])
def test_compact_of_any_cache(pages, fill):
    w = World(pages, 4, 4 * pages, seed=pages)
    used_pages = {"none": [], "all": range(pages), "last": [pages - 1], "odd": range(1, pages, 2), "front": range((pages + 1) // 2)}[fill]
    order = list(used_pages)
    random.Random(1).shuffle(order)
    n = len(order)
    table = _i32([order + [-1] * (pages - n)])
    w.refs[torch.tensor(order, dtype=torch.int64, device=DEV)] = 1
    was = {x: getattr(w.cache, x).clone() for x in ("k", "v", "kpool", "ktail")}
    remap, used = _i32([9] * pages), _i32([-1])
    dsa.cache_compact(w.dims, w.cache, w.refs, _i32([4 * n]), table, remap, used, w.ws(1))
    dsa.check_device_error()
    assert used.item() == n and w.refs.tolist() == [1] * n + [0] * (pages - n)
    got = table[0, :n].long()
    assert sorted(got.tolist()) == list(range(n))
    old = torch.tensor(order, dtype=torch.int64, device=DEV)
    for x, y in was.items():
        assert torch.equal(getattr(w.cache, x)[got], y[old]), x
    stay = old < n
    assert torch.equal(got[stay], old[stay]) and torch.equal(remap[old].long(), got)


@pytest.mark.parametrize("pages,rows", [(1, 1), (3, 2), (257, 5), (1030, 40), (16383, 512), (16384, 513), (16385, 30), (40001, 512)])
@pytest.mark.parametrize("room", [True, False])
def test_reserve_in_any_cache(pages, rows, room):
    """Around the sizes at which the calls' kernels change; with too few free pages nothing changes."""
    w = World(pages, 4, 32, seed=pages + rows)
    r = random.Random(rows)
    full = [p for p in range(pages) if r.random() < (0.3 if room else 0.97)] or [0]
    for p in full:
        w.m_refs[p] = r.choice([1, 1, 2, 3])
    w.refs.copy_(_i32(w.m_refs))
    lens, table = [r.randrange(9) for _ in range(rows)], [[-1] * w.cols for _ in range(rows)]
    own = r.sample(full, len(full))
    for b, n in enumerate(lens):
        for c in range(w.held(n)):
            if not own:      # the pages are given away: this row has fewer
                lens[b] = 4 * c
                break
            table[b][c] = own.pop()
    new = [n + r.choice([0, 1, 2, 5, 23]) for n in lens]
    dev, missing = _i32(table), _i32([-1])
    dsa.cache_reserve(w.dims, w.cache, w.refs, _i32(lens), _i32(new), dev, missing, w.ws(rows))
    assert missing.item() == w.m_reserve(lens, new, table)
    w.same(dev, table)


@pytest.mark.parametrize("dtype,page,n", [("bf16", 64, 1), ("fp32", 20, 37), ("bf16", 4, 2000), ("bf16", 128, 300)])
def test_copy_pages_between_caches(dtype, page, n):
    a, b = World(n + 3, page, 64, dtype=dtype, seed=1), World(2 * n + 5, page, 64, dtype=dtype, seed=2)
    r = random.Random(n)
    src, dst = [r.randrange(n + 3) for _ in range(n)], r.sample(range(2 * n + 5), n)
    if n > 30:
        src[5], dst[7] = -1, -3
    dsa.cache_copy_pages(a.dims, a.cache, b.cache, _i32(src), _i32(dst))
    dsa.check_device_error()
    for x, y in b.copy.items():
        for s, t in zip(src, dst):
            if s >= 0 and t >= 0:
                y[t] = a.copy[x][s]
        assert torch.equal(getattr(b.cache, x), y), x
    dsa.cache_copy_pages(a.dims, a.cache, b.cache, _i32([0, n + 3, 1]), _i32([2 * n + 5, 0, 1]))
    _reports(dsa.DSA_ERR_BAD_PAGE)
    for x, y in b.copy.items():
        y[1] = a.copy[x][1]
        assert torch.equal(getattr(b.cache, x), y), x


def test_caches_with_some_of_the_arrays():
    """A layer without an indexer keeps k and v only: its pages are reserved, forked, copied and compacted too."""
    full = World(9, 16, 64, seed=3)
    only = dsa.PagedCache(k=full.cache.k.clone(), v=full.cache.v.clone())
    refs, table = _i32([0] * 7 + [2, 0]), _i32([[7, -1, -1, -1]])
    ws = torch.zeros(dsa.page_workspace_bytes(full.dims, only, 1), dtype=torch.uint8, device=DEV)
    missing, remap, used = _i32([0]), _i32([0] * 9), _i32([0])
    was = only.k.clone(), only.v.clone()
    dsa.cache_reserve(full.dims, only, refs, _i32([5]), _i32([17]), table, missing, ws)
    assert table.tolist() == [[0, 1, -1, -1]] and refs.tolist() == [1, 1] + [0] * 5 + [1, 0]
    for x, y in zip((only.k, only.v), was):
        y[0, :5] = y[7, :5]
        assert torch.equal(x, y)
    refs[7] = 0
    refs[8], refs[1], table[0, 1] = 1, 0, 8
    dsa.cache_compact(full.dims, only, refs, _i32([17]), table, remap, used, ws)
    assert table.tolist() == [[0, 1, -1, -1]]
    for x, y in zip((only.k, only.v), was):
        y[1] = y[8]
        assert torch.equal(x, y)
    dsa.check_device_error()


def test_a_captured_step_is_replayed_with_other_contents():
    """Release, fork and reserve of branches as one graph."""
    w = World(64, 16, 256, seed=4)
    lens, table = _i32([40, 100]), _i32([[-1] * 16] * 2)
    missing, ws = _i32([0]), w.ws(4)
    dsa.cache_reserve(w.dims, w.cache, w.refs, _i32([0, 0]), lens, table, missing, ws)
    par, bl, bg, bt = _i32([0, 0, 1, 1]), _i32([0] * 4), _i32([0] * 4), _i32([[-1] * 16] * 4)

    def step():
        dsa.cache_release(w.dims, w.cache, w.refs, bg, bt)
        dsa.cache_fork(w.dims, w.cache, w.refs, lens, table, par, bl, bt)
        torch.add(bl, 20, out=bg)
        dsa.cache_reserve(w.dims, w.cache, w.refs, bl, bg, bt, missing, ws)

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for parents in ([0, 0, 1, 1], [1, 1, 1, -1], [0, -1, -1, -1], [1, 0, 1, 0]):
        par.copy_(_i32(parents))
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        dsa.check_device_error()
        assert missing.item() == 0
        names = {}
        for t in (table, bt):
            for p in t.flatten().tolist():
                if p >= 0:
                    names[p] = names.get(p, 0) + 1
        assert {p: c for p, c in enumerate(w.refs.tolist()) if c} == names
        for i, p in enumerate(parents):
            n = [40, 100][p] if p >= 0 else 0
            assert bl[i] == n and int((bt[i] >= 0).sum()) == -(-(n + 20) // 16)
            if p >= 0:
                own = bt[i, n // 16].item()
                assert own != table[p, n // 16].item() and w.refs[own] == 1
                src = table[p, n // 16].long()
                assert torch.equal(w.cache.k[own, :n % 16], w.cache.k[src, :n % 16])
                assert torch.equal(w.cache.ktail[own], w.cache.ktail[src])
