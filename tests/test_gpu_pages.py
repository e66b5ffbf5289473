"""Page bookkeeping against a plain sequential model in Python: every integer
is equal. Page copies byte for byte."""
import numpy as np
import pytest
import torch

import global_soft_capped_b200 as g2

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g2.load_library()
    yield
    assert g2.g2attn_get_device_error() == g2.G2ATTN_OK


class Model:
    """The calls' definition, one sequence after the other."""

    def __init__(self, n, cols, pages, bs):
        self.bs, self.cols = bs, cols
        self.table = -np.ones((n, cols), dtype=np.int32)
        self.lens = np.zeros(n, dtype=np.int32)
        self.refs = np.zeros(pages, dtype=np.int32)

    def free(self):
        return [int(p) for p in np.flatnonzero(self.refs == 0)]

    def grow(self, add, copies=False):
        free, asked, n = self.free(), 0, len(add)
        granted = np.zeros(n, dtype=np.int32)
        src, dst = -np.ones(n, dtype=np.int32), -np.ones(n, dtype=np.int32)
        counts = self.refs.copy()  # shared or not, before anything changes
        for s, a in enumerate(add):
            a = max(0, int(a))
            have, want = -(-int(self.lens[s]) // self.bs), -(-(int(self.lens[s]) + a) // self.bs)
            if want > self.cols:
                continue
            copy = a > 0 and self.lens[s] % self.bs != 0 and counts[self.table[s, have - 1]] > 1
            if copy and not copies:
                continue
            need = want - have + copy
            asked += need
            if need and asked > len(free):
                continue
            granted[s] = 1
            pages = free[asked - need:asked]
            if copy:
                src[s], dst[s] = self.table[s, have - 1], pages[0]
                self.refs[src[s]] -= 1
                self.table[s, have - 1], self.refs[dst[s]] = dst[s], 1
                pages = pages[1:]
            for page, c in zip(pages, range(have, want)):
                self.table[s, c], self.refs[page] = page, 1
            self.lens[s] += a
        return (granted, src, dst) if copies else granted

    def truncate(self, keep):
        for s, k in enumerate(keep):
            self.lens[s] = min(int(self.lens[s]), max(0, int(k)))
            for c in range(-(-int(self.lens[s]) // self.bs), self.cols):
                if self.table[s, c] >= 0:
                    self.refs[self.table[s, c]] -= 1
                    self.table[s, c] = -1

    def fork(self, parents):
        n, free, asked = len(parents), self.free(), 0
        old, was = self.table.copy(), self.lens.copy()
        src, dst = -np.ones(n, dtype=np.int32), -np.ones(n, dtype=np.int32)
        granted = np.ones(n, dtype=np.int32)
        for s, p in enumerate(parents):
            if not 0 <= p < n or p == s:
                continue
            full, part = int(was[p]) // self.bs, int(was[p]) % self.bs != 0
            asked += part
            if part and asked > len(free):
                granted[s] = 0
                continue
            for page in old[s]:
                if page >= 0:
                    self.refs[page] -= 1
            self.table[s] = -1
            self.table[s, :full] = old[p, :full]
            if part:
                src[s], dst[s] = old[p, full], free[asked - 1]
                self.table[s, full] = dst[s]
            for page in self.table[s]:
                if page >= 0:
                    self.refs[page] += 1
            self.lens[s] = was[p]
        return src, dst, granted

    def compact(self):
        live = int((self.refs != 0).sum())
        free = self.free()
        half = len(self.refs) // 2
        src, dst = -np.ones(half, dtype=np.int32), -np.ones(half, dtype=np.int32)
        for i, page in enumerate(p for p in np.flatnonzero(self.refs) if p >= live):
            src[i], dst[i] = page, free[i]
        new = np.arange(len(self.refs))
        for a, b in zip(src, dst):
            if a >= 0:
                new[a] = b
                self.refs[b], self.refs[a] = self.refs[a], 0
        used = self.table >= 0
        self.table[used] = new[self.table[used]]
        return src, dst, live

    def consistent(self):
        counts = np.bincount(self.table[self.table >= 0], minlength=len(self.refs))
        assert np.array_equal(counts, self.refs)


def dev(x):
    return torch.tensor(np.asarray(x, dtype=np.int32)).cuda()


class Pair:
    """The model and the device state, kept equal."""

    def __init__(self, n, cols, pages, bs):
        self.m, self.bs = Model(n, cols, pages, bs), bs
        self.table, self.lens, self.refs = dev(self.m.table), dev(self.m.lens), dev(self.m.refs)

    def same(self):
        self.m.consistent()
        for a, b in ((self.table, self.m.table), (self.lens, self.m.lens), (self.refs, self.m.refs)):
            assert np.array_equal(a.cpu().numpy(), b)

    def grow(self, add, copies=False):
        got = g2.pages_grow(self.table, self.lens, self.refs, dev(add), self.bs, copies=copies)
        want = self.m.grow(add, copies)
        for a, b in zip(got, want) if copies else [(got, want)]:
            assert np.array_equal(a.cpu().numpy(), b)
        self.same()
        return got

    def truncate(self, keep):
        g2.pages_truncate(self.table, self.lens, self.refs, dev(keep), self.bs)
        self.m.truncate(keep)
        self.same()

    def fork(self, parents):
        before = self.table.clone(), self.lens.clone()
        table, lens, src, dst, granted = g2.pages_fork(self.table, self.lens, self.refs,
                                                       dev(parents), self.bs)
        assert torch.equal(self.table, before[0]) and torch.equal(self.lens, before[1])
        self.table, self.lens = table, lens
        for a, b in zip((src, dst, granted), self.m.fork(list(parents))):
            assert np.array_equal(a.cpu().numpy(), b)
        self.same()
        return src, dst, granted

    def compact(self):
        src, dst, live = g2.pages_compact(self.table, self.refs)
        ms, md, ml = self.m.compact()
        assert np.array_equal(src.cpu().numpy(), ms) and np.array_equal(dst.cpu().numpy(), md)
        assert int(live) == ml
        self.same()
        return src, dst


@pytest.mark.parametrize("n,cols,pages,bs", [(1, 1, 1, 1), (3, 4, 10, 16), (33, 7, 150, 8),
                                             (64, 40, 1003, 1), (300, 9, 2000, 64),
                                             (1500, 6, 6000, 4)])
def test_random_life(n, cols, pages, bs):
    """Growing, truncating, forking and compacting in random order, pages
    running out now and then."""
    rng = np.random.default_rng(n + pages)
    p = Pair(n, cols, pages, bs)
    top = cols * bs
    for step in range(14):
        what = rng.integers(0, 5)
        if what <= 1 or step == 0:
            add = rng.integers(-2, max(2, top // 3), n) * (rng.random(n) < 0.7)
            p.grow(add, copies=bool(rng.random() < 0.6))
        elif what == 2:
            keep = np.where(rng.random(n) < 0.5, rng.integers(-1, top + 2, n), top)
            p.truncate(keep)
        elif what == 3:
            parents = np.where(rng.random(n) < 0.5, rng.integers(-1, n + 1, n), np.arange(n))
            p.fork(parents)
        else:
            p.compact()
    p.truncate(np.zeros(n))
    assert not p.refs.any() and (p.table == -1).all()


def test_more_pages_than_one_scan_step():
    """Free pages behind the first 16,384, a cache that is no multiple of 16."""
    pages = 3 * 16384 + 37
    p = Pair(40, 2000, pages, 4)
    p.m.refs[:] = 1                      # pages held by nobody here: in use
    free = np.sort(np.random.default_rng(1).permutation(pages)[:300])
    p.m.refs[free] = 0
    p.refs = dev(p.m.refs)
    add = np.full(40, 17)
    got = g2.pages_grow(p.table, p.lens, p.refs, dev(add), 4)
    assert np.array_equal(got.cpu().numpy(), p.m.grow(add)) and int(got.sum()) == 40
    assert np.array_equal(p.table.cpu().numpy(), p.m.table)
    got = g2.pages_grow(p.table, p.lens, p.refs, dev(add), 4)  # 60 of the needed ~170 are left
    want = p.m.grow(add)
    assert np.array_equal(got.cpu().numpy(), want) and 0 < int(got.sum()) < 40
    assert np.array_equal(p.refs.cpu().numpy(), p.m.refs)
    src, dst, live = g2.pages_compact(p.table, p.refs)
    ms, md, ml = p.m.compact()
    assert np.array_equal(src.cpu().numpy(), ms) and np.array_equal(dst.cpu().numpy(), md)
    assert int(live) == ml and np.array_equal(p.refs.cpu().numpy(), p.m.refs)
    assert np.array_equal(p.table.cpu().numpy(), p.m.table)


def test_refusals_are_in_order():
    p = Pair(4, 3, 5, 16)
    # 3 pages, a row that is too short (asks for nothing), 3 (does not fit), 1 (behind it)
    assert p.grow([48, 49, 33, 16]).tolist() == [1, 0, 0, 0]
    assert p.grow([0, 0, 32, -7]).tolist() == [1, 1, 1, 1]
    # requests whose sum passes 32 bits
    top = 2 ** 31 - 1
    assert p.grow([top, top, top, top]).tolist() == [0, 0, 0, 0]


def test_huge_requests_sum_past_32_bits():
    """Rows of 2^21 columns, 2,000 sequences: the ranks need 64 bits."""
    n, cols, pages = 2000, 1 << 21, 100
    table = torch.full((n, cols), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(n, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    add = torch.full((n,), cols, dtype=torch.int32, device="cuda")
    add[0] = 5
    granted = g2.pages_grow(table, lens, refs, add, 1)
    assert granted[0] == 1 and int(granted.sum()) == 1 and int(refs.sum()) == 5
    assert int((table >= 0).sum()) == 5


def test_lengths_past_32_bits_are_refused():
    """Pages of one row: the length asked for does not fit 32 bits."""
    p = Pair(2, 40, 100, 1)
    assert p.grow([30, 0]).tolist() == [1, 1]
    assert p.grow([2 ** 31 - 1, 2 ** 31 - 1]).tolist() == [0, 0]
    assert p.grow([10, 40]).tolist() == [1, 1]


def test_forks_of_one_parent_and_swaps():
    p = Pair(6, 4, 40, 8)
    p.grow([20, 16, 0, 5, 1, 0])
    src, dst, granted = p.fork([0, 0, 0, 4, 3, 1])      # one parent twice, a swap, a full one
    assert (granted == 1).all()
    assert src.tolist()[1] == src.tolist()[2] >= 0 and dst.tolist()[1] != dst.tolist()[2]
    assert src.tolist()[5] == -1 and src.tolist()[0] == -1


def test_growing_after_a_cut_inside_a_shared_page():
    """Two sequences share two full pages; both are cut inside the second one."""
    p = Pair(3, 4, 10, 8)
    p.grow([16, 0, 0])
    p.fork([0, 0, 0])                                    # three rows, two shared pages
    p.truncate([12, 11, 16])
    assert p.grow([3, 3, 1]).tolist() == [0, 0, 1]       # would write into the shared page
    granted, src, dst = p.grow([3, 6, 0], copies=True)
    assert granted.tolist() == [1, 1, 1] and src.tolist() == [1, 1, -1]
    assert dst.tolist() == [3, 4, -1] and p.refs.tolist()[:6] == [3, 1, 1, 1, 1, 1]
    granted, src, dst = p.grow([1, 1, 1], copies=True)   # nothing is shared now
    assert src.tolist() == dst.tolist() == [-1, -1, -1]


def test_fork_refused_without_pages():
    p = Pair(3, 2, 3, 8)
    p.grow([10, 8, 0])                                   # all three pages
    src, dst, granted = p.fork([0, 0, 1])                # 1 needs a page; 2 shares a full one
    assert granted.tolist() == [1, 0, 1]


def test_entries_outside_the_cache_are_ignored():
    table = torch.tensor([[5, 1 << 20, -7], [0, 9, 3]], dtype=torch.int32).cuda()
    refs = torch.tensor([1, 0, 0, 1, 0, 1, 0, 0], dtype=torch.int32).cuda()
    lens = torch.tensor([3, 3], dtype=torch.int32).cuda()
    g2.pages_truncate(table, lens, refs, dev([0, 1]), 1)
    assert refs.tolist() == [1, 0, 0, 0, 0, 0, 0, 0]
    assert table.tolist() == [[-1, -1, -7], [0, -1, -1]]
    guard = torch.tensor([[1 << 20, -1, 2], [0, 1, -9]], dtype=torch.int32).cuda()
    refs = torch.tensor([1, 1, 1, 0], dtype=torch.int32).cuda()
    out = g2.pages_fork(guard, dev([1 << 30, -4]), refs, dev([1, 0]), 4)
    g2.pages_compact(out[0], refs)
    torch.cuda.synchronize()


@pytest.mark.parametrize("caches,pages,row", [(1, 7, 8), (2, 50, 16384), (5, 12, 16384 + 8),
                                              (3, 9, 100008), (131, 6, 24)])
def test_copy(caches, pages, row):
    g = torch.Generator(device="cuda").manual_seed(row)
    data = [torch.randn(pages, row, generator=g, device="cuda").bfloat16() for _ in range(caches)]
    want = [c.clone() for c in data]
    perm = np.random.default_rng(row).permutation(pages)
    k = pages // 2
    src = np.concatenate([perm[:k], [-1, 3, pages, 0]])
    dst = np.concatenate([perm[k:2 * k], [0, -1, 1, pages + 5]])
    for a, b in zip(perm[:k], perm[k:2 * k]):
        for c in want:
            c[b] = c[a]
    g2.pages_copy(data, dev(src), dev(dst))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(data, want))


def test_copy_far_pages():
    """Offsets past 2^32 bytes."""
    data = torch.empty(3, (1 << 31) + 16, dtype=torch.uint8, device="cuda")
    data[0].fill_(1)
    data[2, 0], data[2, -1] = 200, 201
    g2.pages_copy([data], dev([2]), dev([1]))
    assert torch.equal(data[1], data[2]) and (data[0] == 1).all()


def test_graph_replay():
    """A captured step (grow, fork, truncate, compact) replayed on its state."""
    p = Pair(8, 6, 60, 4)
    add, parents, keep = dev([3] * 8), dev([0, 0, 2, 3, 4, 5, 6, 7]), dev([99] * 8)
    ws = g2.pages_workspace(8, 60)
    g2.pages_grow(p.table, p.lens, p.refs, dev([1] * 8), 4, workspace=ws)
    p.m.grow([1] * 8)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g2.pages_grow(p.table, p.lens, p.refs, add, 4, workspace=ws)
        table, lens, *_ = g2.pages_fork(p.table, p.lens, p.refs, parents, 4, workspace=ws)
        p.table.copy_(table)
        p.lens.copy_(lens)
        g2.pages_truncate(p.table, p.lens, p.refs, keep, 4)
        g2.pages_compact(p.table, p.refs, workspace=ws)
    for step in range(4):
        keep.copy_(dev([99, 99, 5, 99, 2, 99, 99, step]))
        graph.replay()
        torch.cuda.synchronize()
        p.m.grow([3] * 8)
        p.m.fork([0, 0, 2, 3, 4, 5, 6, 7])
        p.m.truncate([99, 99, 5, 99, 2, 99, 99, step])
        p.m.compact()
        p.same()


def test_helper_checks():
    t, l, r = dev(np.zeros((2, 3))), dev([0, 0]), dev(np.zeros(8))
    for bad in [lambda: g2.pages_grow(t[0], l, r, l, 4), lambda: g2.pages_grow(t, l[:1], r, l, 4),
                lambda: g2.pages_grow(t, l, r, l.long(), 4),
                lambda: g2.pages_truncate(t.t(), l, r, l, 4),
                lambda: g2.pages_copy([torch.zeros(4, 8).cuda(), torch.zeros(5, 8).cuda()], l, l),
                lambda: g2.pages_copy([], l, l),
                lambda: g2.pages_copy([torch.zeros(4, 8).cuda()], l, l[:1])]:
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(g2.G2AttnError):
        g2.pages_grow(t, l, r, l, 3)
    with pytest.raises(g2.G2AttnError):
        g2.pages_copy([torch.zeros(4, 3).cuda()], l, l)
