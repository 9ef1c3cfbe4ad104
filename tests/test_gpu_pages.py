"""csa2_pages_resize and csa2_slot_map on the GPU against a plain walk over the
sequences (integers: everything equal)."""
import random

import pytest
import torch

import ragged_util as ru
from fp4_compressed_sparse_gb300 import csa2

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp4_compressed_sparse_gb300 import build_lib
    build_lib.build()
    csa2.load()


class _Bare:
    """A cache's block table and counts without planes of their own size (the calls here read none of them)."""

    def __new__(cls, batch, per, n_pages, page=128, ratio=1):
        u8 = torch.zeros(16, dtype=torch.uint8, device=DEV)
        c = csa2.Cache.__new__(csa2.Cache)
        c.batch, c.capacity, c.ratio, c.page_entries, c.max_pages, c.n_pages = batch, per * page, ratio, page, per, n_pages
        c.block_table = torch.full((batch, per), -1, dtype=torch.int32, device=DEV)
        c.n_tokens = torch.zeros(batch, dtype=torch.int64, device=DEV)
        c.cmp_buf = torch.zeros(16, device=DEV) if ratio == 2 else None
        c.keep = u8
        p = u8.data_ptr()
        c.struct = csa2.CacheStruct(batch, c.capacity, ratio, csa2.SWA_MXFP8, *([p] * 8), c.cmp_buf.data_ptr() if ratio == 2 else None,
                                    c.n_tokens.data_ptr(), c.block_table.data_ptr(), page, per, n_pages, csa2.ENTRY_FP4)
        return c


class Walk:
    """The definition, sequence by sequence."""

    def __init__(self, batch, per, n_pages, page, ratio):
        self.page, self.ratio, self.per, self.n_pages = page, ratio, per, n_pages
        self.table = [[-1] * per for _ in range(batch)]
        self.held = [0] * batch
        self.free, self.n = list(range(n_pages - 1, -1, -1)), n_pages

    def resize(self, lens):
        need, ok = [], []
        for h, n in zip(self.held, lens):
            k = -(-(n // self.ratio) // self.page) if n is not None else h
            fits = n is not None and k <= self.per
            need.append(k if fits else h)
            ok.append(fits)
        back = [(b, p) for b, (h, k) in enumerate(zip(self.held, need)) for p in range(k, h)]
        for j, (b, p) in enumerate(back):
            self.free[self.n + len(back) - 1 - j] = self.table[b][p]
            self.table[b][p] = -1
        self.n += len(back)
        asked, taken, top = 0, 0, self.n
        for b, (h, k) in enumerate(zip(self.held, need)):
            if k > h:
                asked += k - h
                if asked > top:
                    ok[b] = False
                    continue
                for p in range(h, k):
                    self.table[b][p] = self.free[top - 1 - taken]
                    taken += 1
            self.held[b] = k
        self.n -= taken
        return ok


def _same(c, pool, w):
    assert pool.held.tolist() == w.held
    assert int(pool.n_free) == w.n
    assert c.block_table.tolist() == w.table
    assert pool.free.tolist() == w.free


@pytest.mark.parametrize("batch,per,n_pages,page,ratio", [
    (1, 1, 1, 128, 1), (3, 8, 11, 128, 2), (32, 40, 700, 128, 1), (257, 9, 900, 256, 2), (1024, 20, 9000, 128, 1),
    (1500, 17, 14000, 128, 1), (2300, 4, 5000, 256, 2)])
def test_resize_walk(batch, per, n_pages, page, ratio):
    """Lengths that grow, shrink, end and come back, with a pool that runs out now and then; the
    sequence list, the counts, the table and the whole free list after each step."""
    c = _Bare(batch, per, n_pages, page, ratio)
    pool, w = csa2.PagePool(c), Walk(batch, per, n_pages, page, ratio)
    rng, granted, err = random.Random(batch), torch.zeros(batch, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    cap, long = per * page * ratio, False  # (of a single page, the fourth length is too long)
    for step in range(6):
        lens = [rng.choice([0, 1, page * ratio, page * ratio + 1, cap, rng.randint(0, cap)]) for _ in range(batch)]
        if step == 3:
            lens = [0] * batch
        long |= max(lens) // ratio > per * page
        ok = w.resize(lens)
        csa2.pages_resize(c, pool, target=torch.tensor(lens, device=DEV), granted=granted, err=err)
        assert granted.tolist() == [int(o) for o in ok]
        _same(c, pool, w)
    assert int(err) == (csa2.DEVERR_CAPACITY if long else 0)
    used = [p for row in c.block_table.tolist() for p in row if p >= 0]
    assert len(set(used)) == len(used) and sorted(used + pool.free[:w.n].tolist()) == list(range(n_pages))


def test_taking_and_giving_back_restores():
    c = _Bare(40, 12, 400)
    pool = csa2.PagePool(c)
    a = torch.randint(0, 800, (40,), device=DEV)
    csa2.pages_resize(c, pool, target=a)
    was = [t.clone() for t in (c.block_table, pool.free, pool.n_free, pool.held)]
    csa2.pages_resize(c, pool, target=a + 600)
    assert not torch.equal(was[0], c.block_table)
    csa2.pages_resize(c, pool, target=a)
    for x, y in zip(was, (c.block_table, pool.free, pool.n_free, pool.held)):
        assert torch.equal(x, y)


def test_resize_errors_leave_the_sequence():
    """Too long, negative, a broken list, a broken count: the bit, and that sequence as it was."""
    c = _Bare(4, 3, 12)
    pool, w, err = csa2.PagePool(c), Walk(4, 3, 12, 128, 1), torch.zeros(1, dtype=torch.int32, device=DEV)
    csa2.pages_resize(c, pool, target=torch.tensor([100, 200, 300, 0], device=DEV))
    w.resize([100, 200, 300, 0])
    got = torch.zeros(4, dtype=torch.int32, device=DEV)
    for lens, plain, bit in (([385, 200, 129, 5], [None, 200, 129, 5], csa2.DEVERR_CAPACITY), ([1, -1, 384, 5], [1, None, 384, 5], csa2.DEVERR_INDEX),
                             ([2 ** 62, 0, 0, 0], [None, 0, 0, 0], csa2.DEVERR_CAPACITY)):
        err.zero_()
        ok = w.resize(plain)
        csa2.pages_resize(c, pool, target=torch.tensor(lens, device=DEV), granted=got, err=err)
        assert int(err) == bit and got.tolist() == [int(o) for o in ok]
        _same(c, pool, w)
    # a bound that decreases: the sequences whose rows it touches stay; max_new
    c.n_tokens.copy_(torch.tensor([0, 10, 20, 30]))
    for cu, mx, plain in (([0, 200, 100, 140, 150], 300, [None, None, 60, 40]), ([0, 130, 131, 132, 133], 5, [None, 11, 21, 31])):
        err.zero_()
        ok = w.resize(plain)
        csa2.pages_resize(c, pool, cu_new=torch.tensor(cu, dtype=torch.int32, device=DEV), total=200, max_new=mx, granted=got, err=err)
        assert int(err) == csa2.DEVERR_INDEX and got.tolist() == [int(o) for o in ok]
        _same(c, pool, w)
    for t, v in ((pool.n_free, -1), (pool.n_free, 13), (pool.held, 4)):
        err.zero_()
        keep = t.clone()
        t[0] = v
        was = [x.clone() for x in (c.block_table, pool.free, pool.n_free, pool.held)]
        csa2.pages_resize(c, pool, target=torch.tensor([300, w.held[1] * 128, w.held[2] * 128, w.held[3] * 128], device=DEV), granted=got, err=err)
        assert int(err) == csa2.DEVERR_INDEX and got[0] == 0
        for x, y in zip(was, (c.block_table, pool.free, pool.n_free, pool.held)):
            assert torch.equal(x, y)
        t.copy_(keep)


@pytest.mark.parametrize("ratio,page", [(1, 128), (2, 256), (1, None)])
def test_slot_map_is_where_the_append_writes(ratio, page):
    """Slots against the address map of the append, positions against counts; rows of no sequence."""
    B, cap = 5, 1024
    c = csa2.Cache(B, cap, ratio=ratio, page_entries=page)
    if page:
        pool = csa2.PagePool(c, free=torch.randperm(c.n_pages, device=DEV).to(torch.int32),
                             n_free=torch.tensor([c.n_pages], dtype=torch.int32, device=DEV), held=torch.zeros(B, dtype=torch.int32, device=DEV))
        c.block_table.fill_(-1)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    c.n_tokens.copy_(torch.tensor([0, 7, 127, 500, 3]))
    counts = [1, 0, 300, 5, 2]
    total = sum(counts)
    cu = torch.tensor([0, 1, 1, 301, 306, 308], dtype=torch.int32, device=DEV)
    if page:
        csa2.pages_resize(c, pool, cu_new=cu, total=total, max_new=300, err=err)
    slots, pos = (torch.full((total + 4,), 77, dtype=torch.int64, device=DEV) for _ in range(2))
    csa2.slot_map(c, cu, slots, pos, max_new=300, err=err)
    at = 0
    for b, n in enumerate(counts):
        t = int(c.n_tokens[b]) + torch.arange(n, device=DEV)
        assert torch.equal(pos[at:at + n], t)
        there = t // ratio < (int(c.n_tokens[b]) + n) // ratio
        assert torch.equal(slots[at:at + n], torch.where(there, ru.phys(c, b, torch.where(there, t // ratio, 0)), -1))
        at += n
    assert (slots[total:] == -1).all() and (pos[total:] == -1).all() and int(err) == 0
    only = torch.zeros(total + 4, dtype=torch.int64, device=DEV)
    csa2.slot_map(c, cu, None, only, max_new=300)
    assert torch.equal(only, pos)
    if page:  # a page that no one gave: -1 and the bit, the position all the same
        c.block_table[3, :] = -1
        csa2.slot_map(c, cu, slots, pos, max_new=300, err=err)
        assert int(err) == csa2.DEVERR_INDEX and (slots[301:306] == -1).all() and torch.equal(only, pos)
        err.zero_()
    # a list that decreases, a bound that is broken, entries behind the capacity
    csa2.slot_map(c, torch.tensor([0, 5, 3, 10, 12, 14], dtype=torch.int32, device=DEV), slots, pos, max_new=300, err=err)
    assert int(err) == csa2.DEVERR_INDEX and (pos[:3] == -1).all() and (pos[10:12] >= 0).all()
    err.zero_()
    csa2.slot_map(c, cu, slots, pos, max_new=299, err=err)
    assert int(err) == csa2.DEVERR_INDEX and (pos[1:301] == -1).all() and pos[0] == 0
    err.zero_()
    c.n_tokens[2] = cap * ratio - 10
    csa2.slot_map(c, cu, slots, pos, max_new=300, err=err)
    assert int(err) & csa2.DEVERR_CAPACITY and (slots[20:301] == -1).all() and int(pos[300]) == cap * ratio + 289


def test_a_captured_step():
    """Pages and slots in a graph, replayed with other counts."""
    B, per = 6, 10
    c, d = _Bare(B, per, 40), _Bare(B, per, 40)
    pools = [csa2.PagePool(c), csa2.PagePool(d)]
    cu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    bufs = [[torch.zeros(600, dtype=torch.int64, device=DEV) for _ in range(2)] for _ in range(2)]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()

    def step(c, pool, b):
        csa2.pages_resize(c, pool, cu_new=cu, total=600, max_new=400)
        csa2.slot_map(c, cu, b[0], b[1], max_new=400)
    with torch.cuda.graph(graph, stream=side):
        step(d, pools[1], bufs[1])
    for counts in ([100, 0, 300, 1, 1, 1], [1, 1, 1, 1, 200, 0], [400, 0, 0, 0, 0, 1]):
        cu.copy_(torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist()))
        step(c, pools[0], bufs[0])
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((c.block_table, pools[0].free, pools[0].held, *bufs[0]), (d.block_table, pools[1].free, pools[1].held, *bufs[1])):
            assert torch.equal(x, y)
        for k in (c, d):
            k.n_tokens += torch.tensor(counts, device=DEV)
            k.n_tokens[counts.index(max(counts))] = 0


@pytest.mark.parametrize("batch,per,page", [(4, 5, 128), (300, 9, 128), (1500, 6, 256)])
def test_ids_outside_the_pool_do_not_go_back(batch, per, page):
    """A sequence that would give back an id that is no page stays as it was, and nobody gets the id; one that
    keeps such an id gives back what lies behind it."""
    n_pages = batch * per
    c = _Bare(batch, per, n_pages, page)
    pool, w = csa2.PagePool(c), Walk(batch, per, n_pages, page, 1)
    granted, err = (torch.zeros(n, dtype=torch.int32, device=DEV) for n in (batch, 1))
    lens = [page * (per - b % 2) for b in range(batch)]
    w.resize(lens)
    csa2.pages_resize(c, pool, target=torch.tensor(lens, device=DEV), granted=granted, err=err)
    assert int(err) == 0
    # (sequence, entry, id): behind the new length, the last entry of a chunk of sequences among them
    bad = {0: (per - 1, -1), batch // 2: (1, n_pages), batch - 1: (per - 2, 2 ** 30), 2: (0, -5)}
    for b, (p, v) in bad.items():
        c.block_table[b, p] = v
        w.table[b][p] = v
    lens = [1 if b % 3 != 1 else page * per for b in range(batch)]  # a third grows by what the others give back
    for b in bad:
        lens[b] = 1
    plain = [None if b in bad and b != 2 else n for b, n in enumerate(lens)]
    for last in (False, True):  # (the same call again: the same answer)
        ok = w.resize(plain)
        err.zero_()
        csa2.pages_resize(c, pool, target=torch.tensor(lens, device=DEV), granted=granted, err=err)
        assert int(err) == csa2.DEVERR_INDEX and granted.tolist() == [int(o) for o in ok]
        assert all(granted[b] == (b == 2) for b in bad)
        _same(c, pool, w)
    # mended, they go back
    for b, (p, v) in bad.items():
        if b != 2:
            page_id = next(i for i in range(n_pages) if i not in set(w.free[:w.n]) | {x for row in w.table for x in row})
            c.block_table[b, p] = page_id
            w.table[b][p] = page_id
    ok, _ = w.resize(lens), err.zero_()
    csa2.pages_resize(c, pool, target=torch.tensor(lens, device=DEV), granted=granted, err=err)
    assert int(err) == 0 and granted.tolist() == [int(o) for o in ok] == [1] * batch
    _same(c, pool, w)
