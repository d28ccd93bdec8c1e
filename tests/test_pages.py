"""The pages of the paged cache: giving back, reserving, forking, compacting and copying them.

Every result is exact: numbers of pages and holds are integers, page contents are copied bit for bit.  The reference
is the definition in include/mla.h, one list entry and one table entry after the other."""
import ctypes

import numpy as np
import pytest

import mla_gb300 as m
from test_paged import BAD_CACHES, FAKE, fake_cache

gpu = pytest.mark.gpu
OK, INVALID, NO_PAGES = 0, -1, -7


# ---- refusals (CPU: nothing is enqueued) --------------------------------------------------------------------
def fake_pool(**kw):
    v = dict(table=FAKE + (5 << 20), refs=FAKE + (6 << 20), rows=8, max_pages=4, n_pages=8, page=64)
    v.update(kw)
    return m.MlaPagePool(*[v[n] for n in ("table", "refs", "rows", "max_pages", "n_pages", "page")])


def call(name, cache=None, pool=None, **kw):
    a = dict(a=FAKE, b=FAKE + 4096, c=FAKE + 8192, n=3, ws=FAKE + (9 << 20), wsb=1 << 20)
    a.update(kw)
    cache, pool = ctypes.byref(cache or fake_cache()), ctypes.byref(pool or fake_pool())
    tail = (a["ws"], a["wsb"], None)
    L = m.lib()
    if name in ("free", "reserve"):
        return getattr(L, "mla_pages_" + name)(pool, a["a"], a["b"], a["n"], *tail)
    if name == "fork":
        return L.mla_pages_fork(cache, pool, a["a"], a["b"], a["c"], a["n"], *tail)
    if name == "compact":
        return L.mla_pages_compact(cache, pool, a["a"], a["b"], *tail)
    other = ctypes.byref(kw.get("to") or fake_cache(**{n: FAKE + (40 << 20) + (i << 20) for i, n in enumerate(
        ("k_codes", "v_codes", "k_pe", "k_scales", "v_scales"))}))
    return L.mla_pages_copy(cache, other, a["a"], a["b"], a["n"], *tail)


CALLS = ["free", "reserve", "fork", "compact", "copy"]
BAD_POOLS = [(dict(table=None), -1), (dict(refs=None), -1), (dict(rows=0), -1), (dict(rows=(1 << 24) + 1), -1),
             (dict(max_pages=0), -1), (dict(n_pages=0), -1), (dict(table=FAKE + (5 << 20) + 2), -2),
             (dict(refs=FAKE + 1), -2), (dict(page=48), -4), (dict(page=8), -4), (dict(n_pages=1 << 25), -4),
             (dict(max_pages=(1 << 24) + 1), -4)]


@pytest.mark.parametrize("over,rc", BAD_POOLS)
def test_bad_pools_are_refused(over, rc):
    for name in CALLS[:4]:
        assert call(name, pool=fake_pool(**over)) == rc


@pytest.mark.parametrize("over,rc", BAD_CACHES)
def test_bad_caches_are_refused(over, rc):
    for name in CALLS[2:]:
        assert call(name, cache=fake_cache(**over)) == rc
    assert call("copy", to=fake_cache(**over)) == rc


def test_cache_and_pool_belong_together():
    for over in (dict(table=FAKE + (7 << 20)), dict(n_pages=7), dict(max_pages=5), dict(page=32)):
        for name in ("fork", "compact"):
            assert call(name, pool=fake_pool(**over)) == -1


@pytest.mark.parametrize("name", CALLS)
def test_lists_and_workspaces(name):
    assert call(name, a=None) == -1 and call(name, b=None) == -1
    assert call(name, a=FAKE + 2) == -2 and call(name, b=FAKE + 1) == -2
    assert call(name, ws=None) == -3 and call(name, wsb=256) == -3 and call(name, ws=FAKE + 8) == -2
    if name != "compact":
        assert call(name, n=0) == -1 and call(name, n=(1 << 20) + 1) == -1
    if name == "fork":
        assert call(name, c=None) == -1 and call(name, c=FAKE + 2) == -2


def test_copies_between_overlapping_caches():
    assert call("copy", to=fake_cache(page=32)) == -4 and call("copy", to=fake_cache(heads=32)) == -4
    here = fake_cache()
    moved = {n: getattr(here, n) + (64 << 20) for n in ("k_codes", "v_codes", "k_pe", "k_scales", "v_scales")}
    for n in moved:  # one shared array is enough
        assert call("copy", to=fake_cache(**dict(moved, **{n: getattr(here, n)}))) == -1, n
    # keys of one cache in the values of the other, its scales behind them
    assert call("copy", to=fake_cache(**dict(moved, v_codes=here.k_codes))) == -1
    assert call("copy", to=fake_cache(**dict(moved, k_scales=here.v_scales))) == -1
    assert call("copy", to=fake_cache(**dict(moved, k_pe=here.k_codes + 128))) == -1
    assert call("copy", to=fake_cache(n_pages=7)) == -1
    assert call("copy", to=fake_cache(), wsb=16) == -3  # one cache: the next check speaks


def test_workspace_sizes():
    L = m.lib()
    assert m.workspace_size(m.MODE_PAGES, 4, 1000, 8) < m.workspace_size(m.MODE_PAGES, 4, 100000, 8)
    assert m.workspace_size(m.MODE_PAGES, 4, 10, 9000) > m.workspace_size(m.MODE_PAGES, 4, 10, 8)
    for B, pages, rows in ((0, 8, 8), (1, 0, 8), (1, 8, -1), ((1 << 20) + 1, 8, 8), (1, 1 << 28, 8), (1, 8, 1 << 25)):
        assert L.mla_workspace_size(m.MODE_PAGES, B, pages, rows) == 0


def test_binding_refuses_wrong_tensors():
    import torch
    t = torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        m.make_page_pool(t, torch.zeros(4, dtype=torch.int32))
    assert m.mla_status_string(-7).startswith("MLA_ERR_NO_PAGES")


# ---- the definition -----------------------------------------------------------------------------------------
class Book:
    """A pool and the contents of its pages, changed one entry after the other."""

    def __init__(self, rows, max_pages, n_pages, page, seed=0, heads=4):
        rng = np.random.default_rng(seed)
        self.page, self.n_pages, self.max_pages, self.rows = page, n_pages, max_pages, rows
        self.table = np.full((rows, max_pages), -1, dtype=np.int32)
        self.refs = np.zeros(n_pages, dtype=np.int32)
        self.data = {"k_codes": rng.integers(0, 256, (n_pages, heads, page, 128), dtype=np.uint8),
                     "v_codes": rng.integers(0, 256, (n_pages, heads, page, 128), dtype=np.uint8),
                     "k_pe": rng.integers(-30000, 30000, (n_pages, page, 64), dtype=np.int16),
                     "k_scales": rng.random((n_pages, heads), dtype=np.float32),
                     "v_scales": rng.random((n_pages, heads), dtype=np.float32)}

    def want(self, P):
        return -(-P // self.page)

    def bad(self, r, P):
        return not (0 <= r < self.rows and 0 <= P <= self.max_pages * self.page)

    def take(self, needs):
        """Pages for each entry's needs, or None if there are too few."""
        free = np.flatnonzero(self.refs <= 0).tolist()
        if sum(needs) > len(free):
            return None
        out = []
        for n in needs:
            out.append(free[:n])
            free = free[n:]
        return out

    def free(self, rows, P):
        status = OK
        for r, p in zip(rows, P):
            if not 0 <= r < self.rows or p < 0:
                status = INVALID
                continue
            for e in range(self.want(p), self.max_pages):
                x = self.table[r, e]
                self.table[r, e] = -1
                if x == -1:
                    continue
                if not 0 <= x < self.n_pages or self.refs[x] <= 0:
                    status = INVALID
                else:
                    self.refs[x] -= 1
        return status

    def reserve(self, rows, P):
        status, todo, seen = OK, [], set()
        for r, p in zip(rows, P):
            if self.bad(r, p) or r in seen:
                status = INVALID
                todo.append([])
                continue
            seen.add(r)
            row = self.table[r, :self.want(p)]
            if (row >= self.n_pages).any():
                status = INVALID
            todo.append([(r, e) for e in np.flatnonzero(row < 0)])
        pages = self.take([len(x) for x in todo])
        if pages is None:
            return NO_PAGES
        for entries, got in zip(todo, pages):
            for (r, e), x in zip(entries, got):
                self.table[r, e] = x
                self.refs[x] = 1
        return status

    def fork(self, parents, children, P):
        status, todo, seen = OK, [], set()
        for a, c, p in zip(parents, children, P):
            ok = not self.bad(c, p) and 0 <= a < self.rows
            if ok:
                w = self.want(p)
                x = self.table[a, :w]
                ok = bool((self.table[c, :w] < 0).all() and (x >= 0).all() and (x < self.n_pages).all() and
                          (self.refs[x] > 0).all()) and c not in seen
                if ok:
                    seen.add(c)
            if not ok:
                status = INVALID
            todo.append((a, c, p) if ok else None)
        pages = self.take([1 if t and t[2] % self.page else 0 for t in todo])
        if pages is None:
            return NO_PAGES
        before = self.table.copy()
        for t, got in zip(todo, pages):
            if not t:
                continue
            a, c, p = t
            whole, rest = divmod(p, self.page)
            for e in range(whole):
                self.table[c, e] = before[a, e]
                self.refs[before[a, e]] += 1
            if rest:
                x, y = before[a, whole], got[0]
                self.table[c, whole] = y
                self.refs[y] = 1
                for n in ("k_codes", "v_codes"):
                    self.data[n][y, :, :rest] = self.data[n][x, :, :rest]
                self.data["k_pe"][y, :rest] = self.data["k_pe"][x, :rest]
                for n in ("k_scales", "v_scales"):
                    self.data[n][y] = self.data[n][x]
        return status

    def compact(self):
        status = OK
        held = self.refs > 0
        n_live = int(held.sum())
        moved = np.where(held, np.arange(self.n_pages), -1).astype(np.int32)
        src = [x for x in range(n_live, self.n_pages) if held[x]]
        dst = [x for x in range(n_live) if not held[x]]
        for x, y in zip(src, dst):
            moved[x] = y
            self.refs[y], self.refs[x] = self.refs[x], 0
            for n in self.data:
                self.data[n][y] = self.data[n][x]
        for r in range(self.rows):
            for e in range(self.max_pages):
                x = self.table[r, e]
                if x == -1:
                    continue
                y = moved[x] if 0 <= x < self.n_pages else -1
                self.table[r, e] = y
                if y < 0:
                    status = INVALID
        return status, moved, n_live

    def copy(self, other, src, dst):
        """Into other (or itself)."""
        status, last = OK, {}
        for i, d in enumerate(dst):
            if 0 <= d < other.n_pages:
                last[d] = i
        old = {n: x.copy() for n, x in self.data.items()}
        for i, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < self.n_pages and 0 <= d < other.n_pages) or last[d] != i or \
                    (other is self and s != d and s in last):
                status = INVALID
                continue
            for n in old:
                other.data[n][d] = old[n][s]
        return status


class Device:
    """The same on the GPU."""

    def __init__(self, book):
        import torch
        self.book = book
        self.t = {n: torch.from_numpy(x.copy()).cuda() for n, x in book.data.items()}
        self.t["k_pe"] = self.t["k_pe"].view(torch.bfloat16)
        self.t["table"] = torch.from_numpy(book.table.copy()).cuda()
        self.refs = torch.from_numpy(book.refs.copy()).cuda()
        self.cache = m.make_paged_cache(self.t)
        self.pool = m.make_page_pool(self.t["table"], self.refs, book.page)

    def ws(self, n):
        # what an earlier call left there does not matter
        return m.alloc_workspace(m.MODE_PAGES, n, self.book.n_pages, cap=self.book.rows).fill_(0xa5)

    def same(self):
        import torch
        assert np.array_equal(self.t["table"].cpu().numpy(), self.book.table)
        assert np.array_equal(self.refs.cpu().numpy(), self.book.refs)
        for n, x in self.book.data.items():
            got = self.t[n].view(torch.int16) if n == "k_pe" else self.t[n]
            assert np.array_equal(got.cpu().numpy(), x), n


def ints(x):
    import torch
    return torch.tensor(list(map(int, x)), dtype=torch.int32, device="cuda")


def both(book, dev, name, *lists):
    """The call on both sides; the same status and the same pool and pages afterwards."""
    want = getattr(book, name)(*lists)
    ws = dev.ws(len(lists[0]))
    args = [ints(x) for x in lists]
    f = getattr(m, "mla_pages_" + name)
    f(*([dev.cache] if name == "fork" else []), dev.pool, *args, ws)
    assert m.mla_device_status(ws) == want, name
    dev.same()
    return want


def both_compact(book, dev):
    import torch
    want, moved, n_live = book.compact()
    ws = dev.ws(1)
    got, n = torch.full((book.n_pages,), 77, dtype=torch.int32, device="cuda"), ints([-5])
    m.mla_pages_compact(dev.cache, dev.pool, got, n, ws)
    assert m.mla_device_status(ws) == want
    assert np.array_equal(got.cpu().numpy(), moved) and n.item() == n_live
    dev.same()


# ---- on the GPU ---------------------------------------------------------------------------------------------
@gpu
@pytest.mark.parametrize("rows,max_pages,n_pages,page,heads,seed", [
    (1, 1, 1, 16, 4, 0), (6, 5, 13, 16, 4, 1), (9, 7, 40, 32, 8, 2), (5, 33, 100, 64, 12, 3), (12, 3, 31, 128, 4, 4),
    (70, 40, 1025, 16, 4, 5), (40, 65, 2048, 16, 4, 6)])
def test_random_histories(gpu_available, rows, max_pages, n_pages, page, heads, seed):
    """Fifty calls in a row against the definition, wrong entries among them."""
    rng = np.random.default_rng(seed)
    book = Book(rows, max_pages, n_pages, page, seed, heads)
    dev = Device(book)
    seen = set()

    def some_rows(n):
        x = rng.integers(0, rows, n)
        return np.where(rng.random(n) < 0.03, rng.choice([-1, rows, 1 << 30]), x)

    for step in range(50):
        name = rng.choice(["free", "reserve", "reserve", "fork", "fork", "compact"])
        n = int(rng.integers(1, 2 * rows + 1))
        P = rng.integers(0, max_pages * page + 1, n) // rng.integers(1, 5)
        if rng.random() < 0.3:
            P = P // page * page
        if rng.random() < 0.1:
            P[0] = rng.choice([-1, max_pages * page + 1, (1 << 31) - 1])
        if name == "compact":
            both_compact(book, dev)
            continue
        lists = (some_rows(n), P) if name != "fork" else (some_rows(n), some_rows(n), P)
        if name == "reserve" and rng.random() < 0.8:  # few enough to succeed
            k = max(1, n // 4)
            lists = (lists[0][:k], lists[1][:k])
        if name == "fork":  # children that are empty, for the most part
            empty = np.flatnonzero((book.table < 0).all(1))
            if len(empty):
                lists = (lists[0], np.where(rng.random(n) < 0.8, rng.choice(empty, n), lists[1]), P)
        seen.add((name, both(book, dev, name, *lists)))
    if n_pages > 30:
        assert len(seen) >= 4


@gpu
@pytest.mark.parametrize("page,heads,P", [(16, 4, 0), (16, 4, 1), (16, 64, 15), (32, 12, 32), (64, 64, 1000), (64, 128, 63),
                                          (128, 8, 129), (128, 64, 255)])
def test_fork_of_one(gpu_available, page, heads, P):
    wide = -(-max(P, 1) // page) + 1
    book = Book(6, wide, 4 * wide + 6, page, P, heads)
    book.reserve([3], [wide * page])
    dev = Device(book)
    assert both(book, dev, "fork", [3, 3, 3], [0, 5, 2], [P, max(0, P - 1), P // 2]) == OK


@gpu
def test_one_row_twice(gpu_available):
    book = Book(5, 8, 30, 16, 1)
    dev = Device(book)
    assert both(book, dev, "reserve", [1, 4, 1, 1], [100, 128, 128, 16]) == INVALID   # the first entry counts
    assert both(book, dev, "fork", [1, 4, 1], [0, 0, 2], [50, 128, 97]) == INVALID    # so does it here
    assert both(book, dev, "free", [1, 1, 4, 1], [64, 20, 0, 128]) == OK              # the smallest P counts
    assert both(book, dev, "fork", [0, 0], [1, 4], [33, 50]) == INVALID               # row 1 still holds pages
    assert both(book, dev, "fork", [4, 4], [1, 4], [0, 0]) == OK                      # nothing to do


@gpu
def test_a_parent_may_not_be_made_in_the_same_call(gpu_available):
    book = Book(4, 4, 16, 16, 1)
    book.reserve([0], [40])
    dev = Device(book)
    assert both(book, dev, "fork", [0, 1, 2], [1, 2, 3], [40, 40, 0]) == INVALID


@gpu
def test_too_few_pages_change_nothing(gpu_available):
    book = Book(4, 10, 9, 16, 1)
    dev = Device(book)
    assert both(book, dev, "reserve", [0, 1], [80, 80]) == NO_PAGES
    assert both(book, dev, "reserve", [0, 1], [80, 64]) == OK             # the last page
    assert both(book, dev, "fork", [0], [2], [70]) == NO_PAGES
    assert both(book, dev, "fork", [0, 1], [2, 3], [64, 48]) == OK        # whole pages need none
    assert both(book, dev, "reserve", [9, 3], [16, 64]) == NO_PAGES       # (a wrong entry beside it)
    assert both(book, dev, "free", [0, 1, 2, 3], [0, 0, 0, 0]) == OK
    assert (book.refs == 0).all()


@gpu
def test_damaged_tables(gpu_available):
    """Entries that are no page, and pages that are held less often than they are listed."""
    for seed in range(4):
        book = Book(6, 6, 40, 16, seed)
        book.reserve([0, 1, 2, 3], [96, 50, 96, 16])
        book.table[0, 2], book.table[2, 0], book.table[1, 5], book.table[3, 3] = 40, 1 << 30, -7, -(1 << 31)
        book.refs[book.table[0, 1]] = 0
        dev = Device(book)
        if seed == 0:
            assert both(book, dev, "fork", [0, 0, 0, 2], [4, 5, 1, 5], [96, 16, 0, 16]) == INVALID
        elif seed == 1:
            assert both(book, dev, "free", [0, 2, 1, 3, 0], [0, 0, 0, 0, 0]) == INVALID
        elif seed == 2:
            assert both(book, dev, "reserve", [0, 1, 3], [96, 96, 96]) == INVALID
        else:
            both_compact(book, dev)
            book.free([0], [0])


@gpu
def test_holds_of_the_users_own(gpu_available):
    """A page with holds beyond the table's stays when its sequence goes, and moves with a compaction."""
    book = Book(3, 4, 12, 32, 1)
    book.reserve([0, 1], [128, 128])
    book.refs[5] += 2
    book.refs[11] = 1
    dev = Device(book)
    both(book, dev, "free", [1, 0], [0, 0])
    assert book.refs[5] == 2
    both_compact(book, dev)
    assert book.refs[:2].tolist() == [2, 1]


@gpu
@pytest.mark.parametrize("n_pages,share", [(1, 1.0), (1, 0.0), (31, 0.5), (1023, 0.3), (1024, 1.0), (1024, 0.5), (1025, 0.7),
                                           (4096, 0.01), (5000, 0.99), (9000, 0.5)])
def test_compact(gpu_available, n_pages, share):
    rng = np.random.default_rng(n_pages)
    book = Book(7, max(n_pages, 2), n_pages, 16, 1)
    held = np.flatnonzero(rng.random(n_pages) < share)
    if share == 1.0:
        held = np.arange(n_pages)
    rng.shuffle(held)
    for r, part in enumerate(np.array_split(held, 7)):
        book.table[r, :len(part)] = part
        book.refs[part] = 1
    dev = Device(book)
    both_compact(book, dev)
    both_compact(book, dev)   # nothing left to do


@gpu
@pytest.mark.parametrize("page,heads", [(16, 4), (32, 20), (128, 64), (64, 128)])
def test_copy(gpu_available, page, heads):
    rng = np.random.default_rng(page)
    a, b = Book(1, 1, 21, page, 1, heads), Book(1, 1, 17, page, 2, heads)
    da, db = Device(a), Device(b)

    def run(x, dx, y, dy, src, dst):
        want = x.copy(y, src, dst)
        ws = m.alloc_workspace(m.MODE_PAGES, len(src), y.n_pages).fill_(0xa5)
        m.mla_pages_copy(dx.cache, dy.cache, ints(src), ints(dst), ws)
        assert m.mla_device_status(ws) == want
        dy.same()
        return want

    assert run(a, da, b, db, [20], [16]) == OK
    assert run(a, da, b, db, rng.permutation(17), rng.permutation(17)) == OK
    assert run(a, da, b, db, [3, 3, 3], [0, 5, 9]) == OK                      # one source, several copies
    assert run(a, da, b, db, [1, 2, 4, 21, -1, 6], [7, 7, 7, 8, 9, 17]) == INVALID
    assert run(a, da, a, da, [0, 1, 2], [10, 11, 12]) == OK                   # in one cache
    assert run(a, da, a, da, [4, 5, 6, 7], [5, 14, 6, 14]) == INVALID         # 5 is written; 6 onto itself
    assert run(a, da, a, da, [0, 1], [1, 0]) == INVALID                       # an exchange is refused


@gpu
def test_large_lists(gpu_available):
    """More rows than the plan's shared memory holds claims for, more entries than it has threads; a row of more
    entries than a block takes at once."""
    rows, n_pages = 9000, 33000
    book = Book(rows, 3000, n_pages, 16, 1)
    dev = Device(book)
    order = np.random.default_rng(1).permutation(rows)
    P = (np.arange(rows) * 7) % 50
    assert both(book, dev, "reserve", order, P) == OK
    assert both(book, dev, "reserve", [order[0], order[5]], [16 * 2999 - 3, 16 * 3000]) == OK
    assert both(book, dev, "free", order[5:], P[5:] * 0) == OK
    assert both(book, dev, "fork", np.full(rows - 5, order[0]), order[5:], 3 + np.arange(rows - 5) % 40) == OK
    assert both(book, dev, "free", [order[0], order[0]], [16 * 1030, 16 * 1030 + 1]) == OK
    both_compact(book, dev)


@gpu
def test_captured_calls(gpu_available):
    """A step of free, reserve and fork, captured once and replayed with other lists, on a stream of its own."""
    import torch
    book = Book(12, 6, 64, 16, 1)
    dev = Device(book)
    ws = [dev.ws(4) for _ in range(3)]
    lists = [ints([0] * 4) for _ in range(7)]
    stream = torch.cuda.Stream()

    def step():
        m.mla_pages_free(dev.pool, lists[0], lists[1], ws[0])
        m.mla_pages_reserve(dev.pool, lists[2], lists[3], ws[1])
        m.mla_pages_fork(dev.cache, dev.pool, lists[4], lists[5], lists[6], ws[2])

    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    book.free([0] * 4, [0] * 4)
    book.reserve([0] * 4, [0] * 4)
    book.fork([0] * 4, [0] * 4, [0] * 4)
    dev.same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    rng = np.random.default_rng(5)
    for _ in range(12):
        new = [rng.integers(0, 12, 4), rng.integers(0, 60, 4), rng.permutation(12)[:4], rng.integers(0, 97, 4),
               rng.integers(0, 12, 4), rng.permutation(12)[:4], rng.integers(0, 97, 4)]
        for d, x in zip(lists, new):
            d.copy_(ints(x))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = [book.free(*new[:2]), book.reserve(*new[2:4]), book.fork(*new[4:])]
        assert [m.mla_device_status(w) for w in ws] == want
        dev.same()


@gpu
def test_calls_on_two_pools_at_once(gpu_available):
    import torch
    books = [Book(20, 40, 700, 16, s) for s in (1, 2)]
    devs = [Device(b) for b in books]
    streams = [torch.cuda.Stream() for _ in books]
    torch.cuda.synchronize()
    keep = []
    for _ in range(10):
        for b, d, s in zip(books, devs, streams):
            rng = np.random.default_rng(int(b.refs.sum()) + b.n_pages)
            lists = [rng.permutation(20)[:8], rng.integers(0, 600, 8)]
            with torch.cuda.stream(s):
                args, ws = [ints(x) for x in lists], d.ws(8)
                m.mla_pages_free(d.pool, *args, ws)
                m.mla_pages_reserve(d.pool, args[0], args[1] // 2 + 20, ws)
                keep += [args, ws]
            b.free(*lists)
            b.reserve(lists[0], lists[1] // 2 + 20)
    torch.cuda.synchronize()
    for d in devs:
        d.same()


@gpu
def test_forked_sequences_answer_alike(gpu_available):
    """Attention over the pages of a fork, of its parent and of both after a compaction; then each goes on by itself."""
    import torch
    page, heads, B = 32, 8, 3
    book = Book(2 * B, 8, 60, page, 1, heads)
    for n in ("k_codes", "v_codes"):
        book.data[n] &= 0xb7     # no NaN codes
    book.data["k_pe"][:] = 0x3f80
    dev = Device(book)
    g = torch.Generator(device="cuda").manual_seed(1)
    P = [100, 64, 37]
    both(book, dev, "reserve", range(B), P)
    both(book, dev, "fork", range(B), range(B, 2 * B), P)
    q = torch.empty((B, heads * 192), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    q2 = q.repeat(2, 1)

    def attend():
        out = torch.empty((2 * B, heads * 128), dtype=torch.bfloat16, device="cuda")
        ws = m.alloc_workspace(m.MODE_PAGED_ATTN, 2 * B, 1)
        m.mla_paged_attention(dev.cache, q2, ints([p - 1 for p in P] * 2), max(P), out, ws)
        assert m.mla_device_status(ws) == 0
        return out

    first = attend()
    assert torch.equal(first[:B], first[B:])
    both(book, dev, "free", [1], [0])
    both(book, dev, "reserve", [1], [P[1]])
    both(book, dev, "free", [1], [0])
    both(book, dev, "fork", [B + 1], [1], [P[1]])
    both_compact(book, dev)
    assert torch.equal(attend(), first)
    # each row appends a token of its own: the other one's answer stays
    both(book, dev, "reserve", range(2 * B), [p + 1 for p in P] * 2)
    kv = torch.empty((2 * B, heads, 256), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    pe = torch.empty((2 * B, 64), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    m.mla_paged_append(dev.cache, kv[..., :128], kv[..., 128:], pe, ints(P * 2), 1,
                       m.alloc_workspace(m.MODE_PAGED_APPEND, 2 * B, 1))
    k, first_page = dev.t["k_codes"].cpu().numpy(), book.table[:, 0]
    assert np.array_equal(first_page[:B], first_page[B:])
    assert np.array_equal(k[first_page], book.data["k_codes"][first_page])
    for r in range(B):
        last = book.table[[r, r + B], P[r] // page]
        assert last[0] != last[1] and not np.array_equal(k[last[0]], k[last[1]])


@gpu
def test_pages_past_32_bit_offsets(gpu_available):
    """A cache of more than 2^32 bytes of codes: its last pages forked, copied to each other and moved to the front."""
    import torch
    heads, page, n_pages = 64, 128, 4400  # 1 MiB of key codes a page
    t = m.alloc_paged_cache(n_pages, page, heads)
    t["table"] = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    t["table"][0, :3] = ints([n_pages - 1, n_pages - 5, n_pages - 2])
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[[n_pages - 1, n_pages - 5, n_pages - 2]] = 1
    refs[:4390] = 1  # (the user's own holds: the free pages lie behind them)
    names = [n for n in m.PAGED_TENSORS]
    g = torch.Generator(device="cuda").manual_seed(1)
    for n in names:
        x = torch.randint(1, 100, (10, *t[n].shape[1:]), device="cuda", generator=g)
        t[n][-10:] = x.to(t[n].dtype)
    was = {n: t[n][-10:].clone() for n in names}
    cache, pool = m.make_paged_cache(t), m.make_page_pool(t["table"], refs, page)
    ws = m.alloc_workspace(m.MODE_PAGES, 3, n_pages, cap=3)

    def ok():
        assert m.mla_device_status(ws) == 0

    m.mla_pages_fork(cache, pool, ints([0]), ints([2]), ints([300]), ws)
    ok()
    assert t["table"][2].tolist() == [n_pages - 1, n_pages - 5, 4390, -1]
    for n in ("k_codes", "v_codes"):
        assert torch.equal(t[n][4390, :, :44], was[n][8, :, :44]) and torch.equal(t[n][4390, :, 44:], was[n][0, :, 44:])
    assert torch.equal(t["k_pe"][4390, :44], was["k_pe"][8, :44])
    m.mla_pages_copy(cache, cache, ints([n_pages - 1, n_pages - 2, 4390]), ints([4391, 4392, 7]), ws)
    ok()
    for n in names:
        assert torch.equal(t[n][4391], was[n][9]) and torch.equal(t[n][4392], was[n][8])
        assert torch.equal(t[n][7], t[n][4390])
    tail = {n: t[n][4390].clone() for n in names}
    refs[5:4390] = 0
    moved, n_live = torch.empty(n_pages, dtype=torch.int32, device="cuda"), ints([0])
    m.mla_pages_compact(cache, pool, moved, n_live, ws)
    ok()
    # held: 0-4, 4390 (the tail), 4395 (two rows), 4398, 4399 (two rows); they go to 5, 6, 7, 8
    assert n_live.item() == 9 and t["table"].tolist() == [[8, 6, 7, -1], [-1] * 4, [8, 6, 5, -1]]
    assert refs.tolist() == [1] * 6 + [2, 1, 2] + [0] * (n_pages - 9)
    for n in names:
        for to, x in ((5, tail[n]), (6, was[n][5]), (7, was[n][8]), (8, was[n][9])):
            assert torch.equal(t[n][to], x), (n, to)


@gpu
def test_more_pages_than_one_block_sums_at_once(gpu_available):
    """1.1 million pages (only the pool is touched): the sums over the segments go round twice, through the workspace."""
    import torch
    n_pages, rows = 1100000, 5
    table = torch.full((rows, 4000), -1, dtype=torch.int32, device="cuda")
    refs = torch.ones(n_pages, dtype=torch.int32, device="cuda")
    free = np.sort(np.random.default_rng(1).permutation(n_pages)[:3000])
    refs[torch.from_numpy(free).cuda()] = 0
    pool = m.make_page_pool(table, refs, 16)
    lists = ints([4, 0, 2]), ints([16 * 900 - 3, 16 * 1300, 1])
    ws = m.alloc_workspace(m.MODE_PAGES, 3, n_pages, cap=rows).fill_(0xa5)
    m.mla_pages_reserve(pool, *lists, ws)
    assert m.mla_device_status(ws) == OK
    got = table.cpu().numpy()
    assert np.array_equal(got[4, :900], free[:900]) and np.array_equal(got[0, :1300], free[900:2200])
    assert got[2, 0] == free[2200] and (got >= 0).sum() == 2201 and int(refs.sum()) == n_pages - 3000 + 2201
    m.mla_pages_reserve(pool, ints([1, 3]), ints([16 * 800, 1]), m.alloc_workspace(m.MODE_PAGES, 2, n_pages, cap=rows))
    assert int((table >= 0).sum()) == 2201, "too few: nothing is changed"
    m.mla_pages_free(pool, *[x[:2] for x in (lists[0], ints([0, 16]))], ws)
    assert m.mla_device_status(ws) == OK and int(refs.sum()) == n_pages - 3000 + 2


@gpu
def test_binding_refuses_wrong_shapes_types_and_devices(gpu_available):
    import torch
    book = Book(4, 4, 20, 16, 1)
    dev = Device(book)
    table, refs = dev.t["table"], dev.refs
    for over in (dict(table=table.long()), dict(table=table[0]), dict(table=table[:, :2]), dict(refs=refs.float()),
                 dict(refs=refs.cpu()), dict(refs=refs[::2]), dict(refs=refs[:0])):
        with pytest.raises(ValueError):
            m.make_page_pool(**{**dict(table=table, refs=refs, page=16), **over})
    x, ws = ints([0, 1]), dev.ws(2)
    calls = [lambda a=x, b=x, w=ws: m.mla_pages_free(dev.pool, a, b, w),
             lambda a=x, b=x, w=ws: m.mla_pages_reserve(dev.pool, a, b, w),
             lambda a=x, b=x, w=ws: m.mla_pages_fork(dev.cache, dev.pool, a, b, ints([0, 0]), w),
             lambda a=x, b=x, w=ws: m.mla_pages_copy(dev.cache, dev.cache, a, b, w)]
    for f in calls:
        for over in (dict(a=x.long()), dict(a=x.cpu()), dict(b=x[:1]), dict(b=ints([0, 0, 1, 0])[::2]), dict(b=x.float()),
                     dict(w=ws.cpu())):
            with pytest.raises(ValueError):
                f(**over)
        with pytest.raises(m.MlaError) as e:
            f(w=ws[:256])
        assert e.value.status == -3
    for over in (dict(moved=ints([0] * 19)), dict(n_live=ints([0, 0])), dict(moved=torch.zeros(20, device="cuda"))):
        with pytest.raises(ValueError):
            m.mla_pages_compact(dev.cache, dev.pool, **{**dict(moved=ints([0] * 20), n_live=ints([0]), workspace=ws), **over})
    dev.same()


@gpu
@pytest.mark.parametrize("n", [1, 31, 32, 33, 500, 9000])
def test_copy_of_lists(gpu_available, n):
    """Random pairs in one cache and between two, with sources that are written, repeated destinations and numbers
    outside, in lists around the length of a warp and longer than a plan's threads."""
    rng = np.random.default_rng(n)
    a, b = Book(1, 1, 300, 16, 1), Book(1, 1, 200, 16, 2)
    da, db = Device(a), Device(b)

    def run(src, dst, x, dx, y, dy):
        want = x.copy(y, src, dst)
        ws = m.alloc_workspace(m.MODE_PAGES, len(src), y.n_pages).fill_(0xa5)
        m.mla_pages_copy(dx.cache, dy.cache, ints(src), ints(dst), ws)
        assert m.mla_device_status(ws) == want
        dx.same()
        dy.same()
        return want

    for _ in range(3):
        run(rng.integers(-2, 302, n), rng.integers(-2, 202, n), a, da, b, db)
        run(rng.integers(0, 300, n), rng.integers(0, 300, n), a, da, a, da)
        run(rng.integers(0, 200, n), rng.integers(0, 300, n), b, db, a, da)
    pages = rng.permutation(300)
    k = min(n, 150)
    assert run(pages[:k], pages[150:150 + k], a, da, a, da) == OK
    assert run(pages[:k], pages[:k], a, da, a, da) == OK  # each onto itself


@gpu
@pytest.mark.parametrize("page,cut", [(64, 150), (16, 47), (32, 1)])
def test_back_into_a_shared_page(gpu_available, page, cut):
    """A row that is cut inside a page it shares shows it in refs; its positions forked into an empty row go on by
    themselves, and the other row keeps its bits, whichever of the two was cut."""
    import torch
    heads, whole = 8, cut // page + 1
    for who in (0, 1):  # the parent is cut, the child is
        book = Book(4, whole + 3, 4 * whole + 8, page, cut, heads)
        for n in ("k_codes", "v_codes"):
            book.data[n] &= 0xb7     # no NaN codes
        dev = Device(book)
        both(book, dev, "reserve", [0], [whole * page + 5])
        both(book, dev, "fork", [0], [1], [whole * page])
        other, spare = 1 - who, 3
        assert both(book, dev, "free", [who], [cut]) == OK
        assert book.refs[book.table[who, cut // page]] == 2, "its last page is not its own"
        assert both(book, dev, "fork", [who], [spare], [cut]) == OK
        assert both(book, dev, "free", [who], [0]) == OK
        assert both(book, dev, "reserve", [spare], [cut + 4]) == OK
        last = book.table[spare, cut // page]
        assert book.refs[last] == 1 and last not in book.table[other]
        # four tokens far larger than what is there, so that the page's scale has to grow
        P = [-1] * 4
        P[spare] = cut
        kv = torch.full((16, heads, 256), 3e4, dtype=torch.bfloat16, device="cuda")
        pe = torch.ones((16, 64), dtype=torch.bfloat16, device="cuda")
        ws = m.alloc_workspace(m.MODE_PAGED_APPEND, 4, 4)
        m.mla_paged_append(dev.cache, kv[..., :128], kv[..., 128:], pe, ints(P), 4, ws)
        assert m.mla_device_status(ws) == 0
        written = {int(x) for x in book.table[spare, cut // page:] if x >= 0}
        same = [x for x in range(book.n_pages) if x not in written]
        for n, x in book.data.items():
            got = dev.t[n].view(torch.int16) if n == "k_pe" else dev.t[n]
            assert np.array_equal(got.cpu().numpy()[same], x[same]), n
        assert not np.array_equal(dev.t["k_codes"].cpu().numpy()[last], book.data["k_codes"][last])
