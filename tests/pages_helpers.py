"""Page pools in states that lengths set back by hand leave behind, and what holds after a reservation."""

from __future__ import annotations

import numpy as np

from oracle import serving


def random_pool(rng, B: int, per: int, spare: int, bs: int, gaps: bool = False):
    """A pool whose sequences name each other's pages, at whatever entry, also behind their tokens: lengths lie anywhere
    within the pages that they name.  ``gaps``: entries are missing between others behind the tokens, too."""
    pages = max(1, int(rng.integers(1, B * per + 1)))
    nb = pages + spare
    names = rng.permutation(nb)
    table, lens = [], []
    for _ in range(B):
        n = int(rng.integers(0, min(per, pages) + 1))
        row = names[rng.permutation(pages)[:n]].tolist() + [-1] * (per - n)
        lens.append(int(rng.integers(0, n * bs + 1)))
        if gaps:
            for j in range(-(-lens[-1] // bs), n):
                if rng.random() < 0.4:
                    row[j] = -1
        table.append(row)
    holders = [0] * nb
    for row in table:
        for p in row:
            if p >= 0:
                holders[p] += 1
    return serving.Pool(table, lens, holders, bs)


def nobody_else_writes(pool, new, out, table, holders):
    """What a reservation promises, from its result alone; table and holders as they were before it."""
    granted, src, dst = ([int(x) for x in a] for a in out)
    counted = [0] * len(holders)
    for row in pool.table:
        for p in row:
            if p >= 0:
                counted[p] += 1
    assert counted == list(pool.holders)  # no page lost, none counted twice
    for b, (row, n) in enumerate(zip(pool.table, pool.lens)):
        first, end = n // pool.bs, -(-(n + new[b]) // pool.bs)
        if not granted[b] or new[b] == 0:
            assert list(row) == list(table[b]) and src[b] == dst[b] == -1
            continue
        for j in range(len(row)):
            if not first <= j < end:
                assert row[j] == table[b][j]
                continue
            assert row[j] >= 0 and pool.holders[row[j]] == 1
            if row[j] != table[b][j]:
                assert holders[row[j]] == 0  # a free one
                assert table[b][j] < 0 or holders[table[b][j]] > 1  # an own one stays
                if table[b][j] >= 0 and j * pool.bs < n:
                    assert (src[b], dst[b]) == (table[b][j], row[j])
        if n % pool.bs == 0 or row[first] == table[b][first]:
            assert src[b] == dst[b] == -1
