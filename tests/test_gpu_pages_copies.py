"""Copies that grow, fork and compact leave to the caller: what they count, and
that contents follow when each call's copies come before the next call."""
import numpy as np
import pytest
import torch

import global_soft_capped_b200 as g2
from test_gpu_pages import Pair

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g2.load_library()
    yield
    assert g2.g2attn_get_device_error() == g2.G2ATTN_OK


def cut_inside_a_shared_page(pages, n=2):
    """n sequences of 12 rows over two pages of 8 rows that all of them share."""
    p = Pair(n, 4, pages, 8)
    p.grow([16] + [0] * (n - 1))
    p.fork([0] * n)
    p.truncate([12] * n)
    assert p.refs.tolist()[:2] == [n, n] and not p.refs[2:].any()
    return p


@pytest.mark.parametrize("spare", [0, 1, 2, 3])
def test_all_holders_of_a_page_grow(spare):
    """Each asks for a copy, in order, the last one too; the page is free then."""
    p = cut_inside_a_shared_page(2 + spare, n=3)
    granted, src, dst = p.grow([2, 2, 2], copies=True)
    assert granted.tolist() == [int(s < spare) for s in range(3)]
    assert src.tolist() == [1 if s < spare else -1 for s in range(3)]
    assert dst.tolist() == [2 + s if s < spare else -1 for s in range(3)]
    assert p.refs.tolist() == [3, 3 - spare] + [1] * spare
    assert p.lens.tolist() == [14 if s < spare else 12 for s in range(3)]
    # a refused one is alone on the page in the end, and then needs no page
    if spare == 2:
        granted, src, dst = p.grow([0, 0, 2], copies=True)
        assert granted.tolist() == [1, 1, 1] and src.tolist() == [-1, -1, -1]


def test_contents_follow_the_copies():
    """Random steps on two caches and plain histories: each call's copies are
    issued before the next call, which may hand out the pages they read."""
    n, cols, pages, bs = 7, 6, 40, 4
    rng = np.random.default_rng(5)
    p = Pair(n, cols, pages, bs)
    caches = [torch.full((pages, bs, 8), -1, dtype=torch.int32, device="cuda") for _ in range(2)]
    hist = [[] for _ in range(n)]
    mark, reused = 0, 0

    def read(s):
        rows = [(int(p.m.table[s, j // bs]), j % bs) for j in range(int(p.m.lens[s]))]
        at = torch.tensor(rows, dtype=torch.long).reshape(-1, 2).cuda()
        return [c[at[:, 0], at[:, 1], 0].tolist() for c in caches]

    freed = set()
    for step in range(60):
        what = rng.integers(0, 4)
        if what <= 1:
            add = rng.integers(0, 4, n)
            before = p.m.lens.copy()
            granted, src, dst = p.grow(add, copies=True)
            new = {int(x) for x in p.m.table.ravel() if x >= 0}
            reused += len(freed & new)
            freed = {int(x) for x in src.tolist() if x >= 0 and p.m.refs[int(x)] == 0}
            g2.pages_copy(caches, src, dst)
            for s in range(n):
                for j in range(int(before[s]), int(p.m.lens[s])):
                    mark += 1
                    hist[s].append(mark)
                    for c in caches:
                        c[int(p.m.table[s, j // bs]), j % bs] = mark
        elif what == 2:
            parents = np.where(rng.random(n) < 0.4, rng.integers(0, n, n), np.arange(n))
            src, dst, granted = p.fork(parents)
            g2.pages_copy(caches, src, dst)
            hist = [list(hist[int(q)]) if g else h
                    for q, g, h in zip(parents, granted.tolist(), hist)]
        else:
            keep = np.maximum(p.m.lens - rng.integers(0, 6, n), 0)
            p.truncate(keep)
            hist = [h[:int(k)] for h, k in zip(hist, keep)]
            if rng.random() < 0.3:
                src, dst = p.compact()
                g2.pages_copy(caches, src, dst)
                freed = set()
        for s in range(n):
            assert read(s) == [hist[s], hist[s]], (step, s)
    assert mark > 100 and reused > 0
