"""Page handling against the list implementation: tables, counts, contents."""
import random

import numpy as np
import pytest

import cache_ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gsk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_softmax_kv_gb300 as g
    g.build()
    return g


def i32(v):
    return torch.tensor(np.asarray(v, dtype=np.int64), device="cuda").to(torch.int32)


class World:
    """The device's pool beside the lists. A page's bytes and scales come from its number."""

    def __init__(self, gsk, pages=40, seqs=8, width=6, page=16, heads=2, D=64, block=8):
        self.g, self.p = gsk, cache_ref.Pages(pages, seqs, width, page)
        g = torch.Generator(device="cuda").manual_seed(pages)
        self.first = torch.randint(0, 256, (pages, heads, page, D), generator=g, device="cuda", dtype=torch.uint8)
        self.scale0 = torch.rand((pages, heads, page // block), generator=g, device="cuda")
        self.cache, self.scales = self.first.clone().view(torch.float8_e4m3fn), self.scale0.clone()
        self.table, self.lens, self.refs = i32(self.p.table), i32(self.p.lens), i32(self.p.refs)
        self.status = i32([0])

    def fork(self, a, b):
        self.g.csa_cache_fork(self.table, self.lens, self.refs, i32(a), i32(b), self.p.page, self.status)
        self.p.fork(a, b)

    def reserve(self, s, r):
        self.g.csa_cache_reserve(self.cache, self.scales, self.table, self.lens, self.refs, i32(s), i32(r), self.status)
        self.p.reserve(s, r)

    def grow(self, s, r):
        """reserve, and the rows are there (as an append would make them)"""
        self.reserve(s, r)
        for i, n in zip(s, r):
            self.p.lens[i] += n
        self.lens.copy_(i32(self.p.lens))

    def free(self, s):
        self.g.csa_cache_free(self.table, self.lens, self.refs, i32(s))
        self.p.free(s)

    def compact(self):
        live = i32([0])
        self.g.csa_cache_compact(self.cache, self.scales, self.table, self.refs, live)
        assert live.item() == self.p.compact()

    def check(self, status=0):
        assert self.table.tolist() == self.p.table
        assert self.lens.tolist() == self.p.lens
        assert self.refs.tolist() == self.p.refs
        assert self.status.item() == self.p.status == status
        held = [i for i, r in enumerate(self.p.refs) if r > 0]
        src = [self.p.data[i] for i in held]
        assert torch.equal(self.cache.view(torch.uint8)[held], self.first[src])
        assert torch.equal(self.scales[held], self.scale0[src])


def test_a_life_of_pages(gsk):
    w = World(gsk)
    w.grow([0, 3, 1], [20, 16, 1])
    w.check()
    w.fork([0, 0, 3], [4, 5, 6])
    w.check()
    w.grow([0, 4, 5], [3, 1, 30])                            # all holders of the shared page: the last keeps it
    w.check()
    w.reserve([3], [0])
    w.reserve([6, 3], [1, 1])                                # the shared page is full: only new ones
    w.check()
    w.free([0, 6, 6, 99, -1])
    w.check()
    w.compact()
    w.check()
    w.grow([2], [33])
    w.free([1])
    w.compact()
    w.check()


def test_empty_lists_and_an_empty_pool(gsk):
    w = World(gsk)
    w.fork([], [])
    w.reserve([], [])
    w.free([])
    w.compact()
    w.check()
    gsk.csa_cache_copy_pages(w.cache, w.scales, i32([]), i32([]))
    w.check()


@pytest.mark.parametrize("call,status", [
    (lambda w: w.fork([8], [1]), 1), (lambda w: w.fork([0], [-1]), 1), (lambda w: w.fork([0, 0], [1, 1]), 2),
    (lambda w: w.fork([0, 1], [1, 3]), 2), (lambda w: w.fork([0], [0]), 2 | 4), (lambda w: w.fork([0], [2]), 4),
    (lambda w: w.reserve([0, 9], [1, 1]), 1), (lambda w: w.reserve([0, 0], [1, 1]), 2),
    (lambda w: w.reserve([0, 1], [1, 97]), 16), (lambda w: w.reserve([0, 1], [2 ** 31 - 1, 5]), 16),
    (lambda w: w.reserve([3, 4, 5, 6, 7, 1], [96] * 6), 8)])
def test_a_refused_call_changes_nothing(gsk, call, status):
    w = World(gsk, pages=30)
    w.grow([0, 2], [20, 7])
    call(w)
    w.check(status)


def test_exactly_enough(gsk):
    w = World(gsk, pages=12, seqs=4, width=6)
    w.grow([0, 1], [96, 96])
    w.check()
    w.reserve([0], [0])
    w.reserve([2], [1])
    w.check(8)


def test_seeded_lives(gsk):
    """Random calls, valid and refused ones, over several pool shapes."""
    for seed, (pages, seqs, width, page, heads, D, block) in enumerate(
            [(60, 12, 5, 16, 1, 64, 16), (200, 40, 4, 32, 1, 512, 32), (5000, 30, 90, 16, 1, 64, 1), (90, 9, 12, 64, 3, 128, 16)]):
        w, r = World(gsk, pages, seqs, width, page, heads, D, block), random.Random(seed)
        for _ in range(40):
            kind = r.choice("rrrffxc")
            if kind == "r":
                s = r.sample(range(seqs), r.randint(1, seqs))
                rows = [r.choice([0, 1, 2, page, r.randint(1, width * page // 2)]) for _ in s]
                w.reserve(s, rows)
                if w.p.status == 0:
                    for i, n in zip(s, rows):
                        w.p.lens[i] += n
                    w.lens.copy_(i32(w.p.lens))
            elif kind == "f":
                empty = [i for i in range(seqs) if not w.p.lens[i] and w.p.table[i][0] < 0]
                full = [i for i in range(seqs) if i not in empty]
                if empty and full:
                    c = r.sample(empty, r.randint(1, len(empty)))
                    w.fork([r.choice(full) for _ in c], c)
            elif kind == "x":
                w.free(r.sample(range(seqs), r.randint(1, max(1, seqs // 3))))
            else:
                w.compact()
            assert w.status.item() == w.p.status
            w.status.zero_()
            w.p.status = 0
            w.check()


def test_shortened_sequences(gsk):
    """Rows taken back (lengths lowered by the caller): pages that are shared and
    will be written again are replaced, without a copy where no row is left."""
    w = World(gsk)
    w.grow([0], [50])
    w.fork([0], [1])
    for n in (40, 32, 16, 0):
        w.p.lens[1] = n
        w.lens.copy_(i32(w.p.lens))
        w.reserve([1], [5])
        # a replaced page without rows holds nothing to compare
        for e in range(-(-n // 16), 6):
            if w.p.table[1][e] >= 0:
                w.p.data[w.p.table[1][e]] = w.p.table[1][e]
        assert w.table.tolist() == w.p.table and w.refs.tolist() == w.p.refs
        for e in range(-(-n // 16)):
            p = w.p.table[1][e]
            assert torch.equal(w.cache.view(torch.uint8)[p], w.first[w.p.data[p]])


def test_copy_pages(gsk):
    w = World(gsk, pages=30, heads=3, page=64, D=128)
    src, dst = [3, 3, 5, 9, 40, -1, 7], [10, 11, 12, 9, 13, 14, 30]   # equal and outside ones are skipped
    gsk.csa_cache_copy_pages(w.cache, w.scales, i32(src), i32(dst))
    want, ws = w.first.clone(), w.scale0.clone()
    for s, d in ((3, 10), (3, 11), (5, 12)):
        want[d], ws[d] = w.first[s], w.scale0[s]
    assert torch.equal(w.cache.view(torch.uint8), want) and torch.equal(w.scales, ws)
    big = World(gsk, pages=5, heads=1024, page=16, D=64, block=1)
    gsk.csa_cache_copy_pages(big.cache, big.scales, i32([0]), i32([4]))
    assert torch.equal(big.cache.view(torch.uint8)[4], big.first[0]) and torch.equal(big.scales[4], big.scale0[0])
    assert torch.equal(big.cache.view(torch.uint8)[:4], big.first[:4])


def test_bad_pages_in_tables(gsk):
    w = World(gsk)
    w.grow([0, 1], [40, 20])
    w.table[0, 1] = 10 ** 6
    gsk.csa_cache_fork(w.table, w.lens, w.refs, i32([0]), i32([2]), 16, w.status)
    assert w.status.item() == 32 and w.table[2].tolist() == w.table[0].tolist()
    w.status.zero_()
    w.table[1, 1] = 99
    gsk.csa_cache_reserve(w.cache, w.scales, w.table, w.lens, w.refs, i32([1]), i32([20]), w.status)
    assert w.status.item() == 32 and w.table[1, 2].item() >= 0
    gsk.csa_cache_free(w.table, w.lens, w.refs, i32([0, 1, 2]))
    gsk.csa_cache_compact(w.cache, w.scales, w.table, w.refs)
    assert (w.table == -1).all()


def test_many_sequences_and_streams(gsk):
    n = 3000
    w = World(gsk, pages=9001, seqs=2 * n, width=2, page=16, heads=1, D=64, block=16)
    w.grow(list(range(n)), [1 + i % 20 for i in range(n)])
    w.check()
    side = torch.cuda.Stream()
    a, b = list(range(n)), list(range(n, 2 * n))
    ia, ib, one = i32(a), i32(b), i32([1] * n)
    torch.cuda.synchronize()
    gsk.csa_cache_fork(w.table, w.lens, w.refs, ia, ib, 16, w.status, stream=side)
    w.p.fork(a, b)
    gsk.csa_cache_reserve(w.cache, w.scales, w.table, w.lens, w.refs, ib, one, w.status, stream=side)
    w.p.reserve(b, [1] * n)
    torch.cuda.current_stream().wait_stream(side)
    w.check()
    w.free(list(range(0, 2 * n, 2)))
    w.compact()
    w.check()


def test_refusals(gsk):
    w = World(gsk)
    one = i32([0])
    with pytest.raises(ValueError):
        gsk.csa_cache_fork(w.table, w.lens, w.refs, i32([0, 1]), one, 16, w.status)
    with pytest.raises(gsk.CsaError):
        gsk.csa_cache_fork(w.table, w.lens, w.refs, one, one, 17, w.status)
    with pytest.raises(ValueError):
        gsk.csa_cache_fork(w.table, w.lens, w.refs, one, one, 16, i32([0, 0]))
    with pytest.raises(ValueError):
        gsk.csa_cache_reserve(w.cache, w.scales, w.table, w.lens, w.refs[:-1].contiguous(), one, one, w.status)
    with pytest.raises(TypeError):
        gsk.csa_cache_free(w.table, w.lens, w.refs, one.long())
    with pytest.raises(ValueError):
        gsk.csa_cache_compact(w.cache, w.scales, w.table[:, ::2], w.refs)
    w.check()


def test_a_request_of_more_than_a_million_pages(gsk):
    n = (1 << 20) + 50
    pages = n + 3
    cache = torch.zeros((pages, 1, 16, 64), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.zeros((pages, 1, 1), device="cuda")
    table, lens, refs, status = i32(np.full((2, n), -1)), i32([0, 0]), i32(np.zeros(pages)), i32([0])
    refs[5] = 1                                             # held by nobody in the table
    gsk.csa_cache_reserve(cache, scales, table, lens, refs, i32([1, 0]), i32([16 * n, 16 * 3]), status)
    assert status.item() == 8 and (table == -1).all() and refs.sum().item() == 1
    status.zero_()
    gsk.csa_cache_reserve(cache, scales, table, lens, refs, i32([1, 0]), i32([16 * n, 16 * 2]), status)
    free = torch.tensor([p for p in range(pages) if p != 5], dtype=torch.int32, device="cuda")
    assert status.item() == 0 and torch.equal(table[1], free[:n])
    assert torch.equal(table[0, :2], free[n:]) and (table[0, 2:] == -1).all() and (refs == 1).all()
    gsk.csa_cache_free(table, lens, refs, i32([1, 0]))
    assert (table == -1).all() and refs.sum().item() == 1
