"""GPU: tables of many rows: whole groups of rows before a row that asks for pages,
first forks of all rows at once, and calls whose time grows with the rows and not
with their square.  Whole numbers: all equal."""

import random

import pytest
import torch

import row_wise_top_topk_amd as mt
import serving_oracle as oracle
from test_gpu_pages import DEV, Both, filled

pytestmark = pytest.mark.gpu


class Pages(oracle.Pages):
    """With the lowest free page found from the last one on: a call takes pages only after it gave up others."""

    def take(self):
        while self.at < len(self.refs) and self.refs[self.at] > 0:
            self.at += 1
        if self.at == len(self.refs):
            return -1
        self.refs[self.at] = 1
        return self.at

    def fork(self, parents):
        self.at = 0
        return super().fork(parents)

    def grow(self, grow):
        self.at = 0
        return super().grow(grow)


def both(seed, rows, cols, pages, fill=0.7):
    table, lengths, refs = filled(seed, rows, cols, pages, 16, fill)
    b = Both(table, lengths, refs, 16, pad=1)
    b.plain = Pages(table, lengths, refs, 16)
    return b


@pytest.mark.parametrize("rows", [1025, 2048, 2049, 4096, 4097, 9000, 30001])
def test_forks_and_growth(rows):
    rng = random.Random(rows)
    b = both(rows, rows, 5, 4 * rows + 8192)
    for kind in range(5):
        if kind == 0:        # a parent in eight rows, which goes on or not
            parents = [i // 8 * 8 + 3 if i // 8 % 2 else (i // 8 * 8 + 11) % rows for i in range(rows)]
        elif kind == 1:
            parents = [rng.randrange(-1, rows) for _ in range(rows)]
        elif kind == 2:
            parents = [(i + 1) % rows for i in range(rows)]
        elif kind == 3:      # one parent for all, in the last row
            parents = [rows - 1] * rows
        else:
            parents = [i if rng.random() < 0.6 else -1 for i in range(rows)]
        b.fork([p if p < rows else -1 for p in parents])
        if kind != 2:
            b.grow([rng.choice([0, 0, 1, 7, 40, 200]) for _ in range(rows)])
    b.compact()


def test_pages_run_out_in_a_later_group():
    rows = 5000
    b = both(1, rows, 4, 3 * rows, 0.3)
    free = b.plain.refs.count(0)
    assert free > 3000
    grown = b.grow([40] * rows)
    assert any(grown[:1024]) and not any(grown[4096:])
    b.fork([rows - 1 - i // 3 for i in range(rows)])


def seconds(call):
    best = []
    for _ in range(4):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        best.append(a.elapsed_time(b))
    return min(best[1:])


@pytest.mark.parametrize("op", ["fork", "grow"])
def test_the_time_grows_with_the_rows(op):
    # four times as many rows: four times the work, not sixteen times
    times = []
    for rows in (1 << 18, 1 << 20):
        table = torch.arange(3 * rows, dtype=torch.int32, device=DEV).view(rows, 3)
        refs = torch.cat([torch.ones(3 * rows, dtype=torch.int32, device=DEV), torch.zeros(rows, dtype=torch.int32, device=DEV)])
        refs[table[:, 2].long()] = 0
        lengths = torch.full((rows,), 21, dtype=torch.int32, device=DEV)
        i = torch.arange(rows, device=DEV)
        if op == "fork":     # no parent goes on; of its four forks three ask for a page
            parents = ((i // 4 * 4 + 4) % rows).to(torch.int32)
            call = lambda: mt.pages_fork(table, lengths, refs, parents, 16)  # noqa: E731
        else:                # all ask for a page
            def call():
                lengths.fill_(21)
                refs[2 * rows:].zero_()
                mt.pages_grow(table, lengths, refs, torch.full_like(lengths, 20), 16)
        times.append(seconds(call))
    assert times[1] < 9 * times[0], times
