"""GPU: forks, growth, compaction and copies of a paged cache's pages, against
plain Python lists.  Whole numbers, and values that are moved: all equal."""

import random

import pytest
import torch

import row_wise_top_topk_amd as mt
import serving_oracle as oracle

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def ints(x, device=DEV):
    return torch.tensor(x, dtype=torch.int32, device=device)


def filled(seed, rows, cols, pages, bs, fill=0.7):
    """A table whose rows hold pages of their own, in random order."""
    rng = random.Random(seed)
    free = list(range(pages))
    rng.shuffle(free)
    table, lengths, refs = [], [], [0] * pages
    for _ in range(rows):
        n = min(rng.randint(0, int(cols * bs * fill)), len(free) * bs)
        mine = [free.pop() for _ in range(-(-n // bs))]
        for p in mine:
            refs[p] = 1
        table.append(mine + [rng.choice([-1, 5, 1 << 29])] * (cols - len(mine)))
        lengths.append(n)
    return torch.tensor(table, dtype=torch.int32).view(rows, cols), ints(lengths, "cpu"), ints(refs, "cpu")


BIG = 1 << 13   # a cache of more pages than this is no longer the work of one workgroup


class Both:
    """The same rows on the GPU and with lists; ``big``: behind as many pages that are held."""

    def __init__(self, table, lengths, refs, bs, pad=0, big=False):
        rows, cols = table.shape
        if big:
            refs = torch.cat([torch.ones(BIG, dtype=torch.int32), refs])
            table = torch.where((table >= 0) & (table < 1 << 20), table + BIG, table)
        wide = torch.full((rows, cols + pad), 77, dtype=torch.int32, device=DEV)
        wide[:, :cols] = table
        self.wide, self.table, self.bs = wide, wide[:, :cols], bs
        self.lengths, self.refs = lengths.to(DEV), refs.to(DEV)
        self.plain = oracle.Pages(table, lengths, refs, bs)

    def same(self):
        assert self.table.tolist() == self.plain.table
        assert self.lengths.tolist() == self.plain.lengths
        assert self.refs.tolist() == self.plain.refs
        assert (self.wide[:, self.table.shape[1]:] == 77).all()

    def fork(self, parents):
        got, want = mt.pages_fork(self.table, self.lengths, self.refs, ints(parents), self.bs).tolist(), self.plain.fork(parents)
        assert got == want
        self.same()
        return got

    def grow(self, grow):
        got, want = mt.pages_grow(self.table, self.lengths, self.refs, ints(grow), self.bs).tolist(), self.plain.grow(grow)
        assert got == want
        self.same()
        return got

    def compact(self):
        got, want = mt.pages_compact(self.table, self.lengths, self.refs, self.bs).tolist(), self.plain.compact()
        assert got == want
        self.same()
        return got


def test_fork_by_hand():
    b = Both(ints([[4, 7, -1], [2, 0, 9], [6, -1, -1]], "cpu"), ints([20, 48, 5], "cpu"), ints([1, 0, 1, 0, 1, 0, 1, 1, 0, 1], "cpu"), 16)
    # row 1 becomes a fork of row 0, row 2 of what row 1 was (full pages only), row 0 goes on
    assert b.fork([0, 0, 1]) == [[-1, -1], [7, 1], [-1, -1]]
    assert b.table.tolist() == [[4, 7, -1], [4, 1, -1], [2, 0, 9]] and b.lengths.tolist() == [20, 20, 48]
    assert b.refs.tolist() == [1, 1, 1, 0, 2, 0, 0, 1, 0, 1]
    assert b.fork([-1, 3, 2]) == [[-1, -1]] * 3 and b.refs.tolist() == [1, 0, 1, 0, 0, 0, 0, 0, 0, 1]


@pytest.mark.parametrize("big", [False, True])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("rows,cols,pages", [(1, 1, 1), (2, 3, 5), (5, 7, 40), (33, 9, 400), (300, 20, 4500), (70, 300, 13000)])
def test_forks(rows, cols, pages, bs, big):
    rng = random.Random(rows * bs)
    b = Both(*filled(rows + bs, rows, cols, pages, bs), bs, pad=3, big=big)
    for kind in range(4):
        if kind == 0:
            parents = [rng.randrange(rows) for _ in range(rows)]
        elif kind == 1:
            parents = [rng.choice([i, i, rng.randrange(-2, rows + 2)]) for i in range(rows)]
        elif kind == 2:
            parents = [(i + 1) % rows for i in range(rows)]
        else:
            parents = [rng.randrange(rows)] * rows
        b.fork(parents)


@pytest.mark.parametrize("big", [False, True])
@pytest.mark.parametrize("bs", [16, 64])
@pytest.mark.parametrize("rows,cols,pages", [(1, 1, 0), (1, 4, 3), (6, 5, 12), (40, 30, 700), (257, 40, 6000), (3, 2000, 5000)])
def test_growth(rows, cols, pages, bs, big):
    rng = random.Random(rows + pages)
    b = Both(*filled(rows, rows, cols, pages, bs, 0.4), bs, pad=1, big=big)
    for most in (0, 1, bs, 5 * bs, cols * bs):
        b.grow([rng.randint(-1, most) for _ in range(rows)])
    b.fork([i if rng.random() < 0.5 else -1 for i in range(rows)])
    b.grow([rng.randint(0, cols * bs // 2) for _ in range(rows)])
    b.grow([(1 << 31) - 1] * rows)


@pytest.mark.parametrize("rows,cols,pages", [(1024, 4, 8192), (1025, 3, 4000), (1024, 5, 8192), (1, 4096, 8192), (1, 4097, 8192), (60, 40, 8193), (2000, 40, 65537)])
def test_calls_next_to_the_limits_of_one_workgroup(rows, cols, pages):
    rng = random.Random(rows)
    b = Both(*filled(rows, rows, cols, pages, 16, 0.9), 16)
    b.fork([rng.choice([i, i, -1, rng.randrange(rows)]) for i in range(rows)])
    b.grow([rng.randint(0, 8 * cols) for _ in range(rows)])
    b.compact()


def test_pages_run_out():
    b = Both(ints([[0, 1], [2, -1], [-1, -1]], "cpu"), ints([32, 7, 0], "cpu"), ints([1, 1, 1, 0, 0], "cpu"), 16)
    assert b.fork([1, 1, 1]) == [[2, 0], [-1, -1], [2, 1]]     # row 0's pages are free by then
    assert b.fork([0, 0, 2]) == [[-1, -1], [0, 2], [-1, -1]]
    assert b.grow([30, 20, 0]) == [0, 20, 0]                   # row 0 would pass its columns
    assert b.grow([0, 0, 10]) == [0, 0, 10]
    assert b.grow([0, 1, 10]) == [0, 1, 10]                    # both have the place: 28 and 27 tokens in two pages
    assert b.grow([10, 4, 0]) == [0, 4, 0]                     # no page is free for row 0
    assert b.grow([9, 0, 5]) == [9, 0, 5]                      # full pages, all of them
    assert b.grow([1, 1, 1]) == [0, 0, 0]
    b = Both(ints([[0, 1], [2, -1], [-1, -1]], "cpu"), ints([32, 7, 0], "cpu"), ints([1, 1, 1], "cpu"), 16)
    assert b.fork([0, 1, 1]) == [[-1, -1], [-1, -1], [2, -1]] and b.lengths.tolist() == [32, 7, 0]


@pytest.mark.parametrize("big", [False, True])
@pytest.mark.parametrize("bs", [16, 128])
@pytest.mark.parametrize("rows,cols,pages", [(1, 1, 1), (1, 2, 2), (4, 6, 64), (9, 20, 131), (20, 300, 4097), (60, 300, 20000)])
def test_compaction(rows, cols, pages, bs, big):
    rng = random.Random(pages)
    b = Both(*filled(rows, rows, cols, pages, bs), bs, pad=2, big=big)
    b.compact()
    b.fork([rng.choice([i, -1, rng.randrange(rows)]) for i in range(rows)])
    b.compact()
    assert all(x == [-1, -1] for x in b.compact())


def test_compaction_moves_pages_of_the_callers_own():
    b = Both(ints([[9, -1]], "cpu"), ints([3], "cpu"), ints([0, 0, 0, 0, 1, 0, 3, 0, 0, 1], "cpu"), 16)
    assert b.compact()[:4] == [[4, 0], [6, 1], [9, 2], [-1, -1]] and b.refs.tolist() == [1, 3, 1] + [0] * 7


def test_pages_that_are_not_there():
    # entries outside the pages are handed on and count nowhere
    table = ints([[3, -5, 1 << 30, 2], [7, 0, -1, -1]], "cpu")
    for big in (False, True):
        b = Both(table, ints([60, 20], "cpu"), ints([1, 0, 1, 1, 0, 0], "cpu"), 16, big=big)
        b.fork([0, 0])
        b.grow([4, 4])
        b.compact()
        b.fork([1, 0])
        b.fork([5, 5])
        # a last page that is not there
        b = Both(ints([[3, 1 << 30]], "cpu"), ints([20], "cpu"), ints([0, 0, 0, 1], "cpu"), 16, big=big)
        b2 = Both(ints([[3, 1 << 30], [-1, -1]], "cpu"), ints([20, 0], "cpu"), ints([0, 0, 0, 1], "cpu"), 16, big=big)
        b.grow([16])
        assert b2.fork([0, 0]) == [[-1, -1], [-1, -1]]


def test_lengths_outside_the_table():
    for big in (False, True):
        b = Both(ints([[0, 1], [2, 3]], "cpu"), ints([1000, -7], "cpu"), ints([1, 1, 0, 0], "cpu"), 16, big=big)
        assert b.grow([1, 20]) == [0, 20]
        b.fork([1, 0])
        b.compact()


def test_pages_of_many_chunks():
    # a cache of 300000 pages, nearly all in use
    pages, rows, cols = 300000, 8, 1000
    refs = torch.ones(pages, dtype=torch.int32)
    refs[torch.randperm(pages, generator=torch.Generator().manual_seed(1))[:5000]] = 0
    b = Both(torch.full((rows, cols), -1, dtype=torch.int32), torch.zeros(rows, dtype=torch.int32), refs, 16)
    b.grow([16 * 700 + i for i in range(rows)])
    b.grow([1, 5000, 1, 0, 1, 16, 17, 18])
    b.fork([0, 0, 0, 3, 4, -1, 4, 4])
    b.compact()


def test_empty():
    none = torch.zeros(0, 4, dtype=torch.int32, device=DEV)
    z = torch.zeros(0, dtype=torch.int32, device=DEV)
    refs = ints([1, 0, 0, 1])
    assert mt.pages_fork(none, z, refs, z, 16).shape == (0, 2) and mt.pages_grow(none, z, refs, z, 16).shape == (0,)
    assert mt.pages_compact(none, z, refs, 16).tolist() == [[3, 1], [-1, -1]] and refs.tolist() == [1, 1, 0, 0]
    narrow = torch.zeros(2, 0, dtype=torch.int32, device=DEV)
    lengths = ints([0, 5])
    assert mt.pages_grow(narrow, lengths, z, ints([0, 1]), 16).tolist() == [0, 0]
    assert mt.pages_fork(narrow, lengths, z, ints([1, 1]), 16).tolist() == [[-1, -1], [-1, -1]] and lengths.tolist() == [0, 5]
    assert mt.pages_compact(narrow, lengths, z, 16).shape == (0, 2)


def cache(pages, hk, bs, d, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    codes = [torch.randint(0, 256, (pages, hk, bs, d), generator=g, device=DEV, dtype=torch.uint8).view(torch.float8_e4m3fn)
             for _ in range(2)]
    return codes + [torch.rand(pages, hk, generator=g, device=DEV) for _ in range(2)] + [torch.rand(pages, hk, d, generator=g, device=DEV)]


def copied(tensors, pairs):
    out = [t.clone() for t in tensors]
    for src, dst in pairs:
        if 0 <= src < tensors[0].shape[0] and 0 <= dst < tensors[0].shape[0]:
            for t, o in zip(tensors, out):
                o[dst] = t[src]
    return out


def bits(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t.view(torch.int32)


@pytest.mark.parametrize("hk,bs,d", [(1, 16, 64), (3, 32, 64), (8, 64, 128), (2, 128, 128)])
@pytest.mark.parametrize("n", [0, 1, 5, 60])
@pytest.mark.parametrize("means", [True, False])
def test_copies(hk, bs, d, n, means):
    pages = 131
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(n)).tolist()
    pairs = list(zip(order[:n], order[n:2 * n]))
    for i in range(0, n, 7):
        pairs[i] = [(-1, -1), (pairs[i][0], -1), (-1, pairs[i][1]), (pages, pairs[i][1]), (pairs[i][0], 1 << 30)][i % 5]
    x = cache(pages, hk, bs, d)
    want = copied(x, pairs)
    mt.pages_copy(*x[:4], ints(pairs).view(-1, 2), k_mean=x[4] if means else None)
    for i in range(5 if means else 4):
        assert torch.equal(bits(x[i]), bits(want[i]))


def test_many_copies():
    # more pairs than workgroups, one page to many
    x = cache(9000, 1, 16, 64)
    pairs = [(i % 5, 20 + i) for i in range(8980)]
    want = [t.clone() for t in x]
    for o, t in zip(want, x):
        o[20:] = t[torch.arange(8980, device=DEV) % 5]
    mt.pages_copy(*x[:4], ints(pairs), k_mean=x[4])
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(x, want))


def test_compaction_keeps_what_the_rows_read():
    rng = random.Random(4)
    rows, cols, pages, bs = 12, 9, 260, 16
    b = Both(*filled(2, rows, cols, pages, bs), bs)
    x = cache(pages, 2, bs, 64)

    def held():
        return [[[bits(t)[p].clone() for t in x] for p in row[:-(-n // bs)]] for row, n in zip(b.table.tolist(), b.lengths.tolist())]

    def equal(a, c):
        return all(torch.equal(s, t) for r, q in zip(a, c) for u, v in zip(r, q) for s, t in zip(u, v))

    b.fork([i if rng.random() < 0.6 else -1 for i in range(rows)])
    before = held()
    mt.pages_copy(*x[:4], ints(b.compact()).view(-1, 2), k_mean=x[4])
    assert equal(before, held())
    parents = [rng.randrange(rows) for _ in range(rows)]
    before = held()
    mt.pages_copy(*x[:4], ints(b.fork(parents)), k_mean=x[4])
    assert equal([before[p] for p in parents], held())


def test_refusals():
    table, lengths, refs = torch.zeros(2, 4, dtype=torch.int32, device=DEV), ints([0, 0]), ints([0] * 9)
    bad = [(table.long(), lengths, refs, lengths), (table[0], lengths, refs, lengths), (table.t(), lengths, refs, lengths),
           (table, lengths.long(), refs, lengths), (table, ints([0]), refs, lengths), (table, lengths, refs.view(3, 3), lengths),
           (table, lengths, refs.cpu(), lengths), (table, lengths, refs, ints([0])), (table, lengths, refs, None),
           (table[:1].expand(2, 4), lengths, refs, lengths), (table, lengths, ints([0] * 18)[::2], lengths)]
    for args in bad:
        for call in (mt.pages_fork, mt.pages_grow):
            with pytest.raises(ValueError):
                call(*args, 16)
    for args in bad[:7]:
        with pytest.raises(ValueError):
            mt.pages_compact(*args[:3], 16)
    x = cache(4, 1, 16, 64)
    for copies in (ints([0, 1]), ints([[0, 1, 2]]), ints([[0, 1]]).long(), ints([[0, 1]], "cpu"), ints([[0, 1], [0, 1]]).t()[:, :1].t()[:, ::2]):
        with pytest.raises(ValueError):
            mt.pages_copy(*x[:4], copies)
    with pytest.raises(ValueError):
        mt.pages_copy(*x[:4], ints([[0, 1]]), k_mean=x[4][:3])
    with pytest.raises(ValueError):
        mt.pages_copy(x[0], x[1][:3], *x[2:4], ints([[0, 1]]))
