"""Reservations for sequences whose tables name pages behind their tokens, on the GPU: lengths that the caller has set back
after a fork, pages of each other at whatever entry, entries missing between others."""

import numpy as np
import pytest

from io_aware_exact_11_gb300 import fa
from oracle import serving
from tests.pages_helpers import nobody_else_writes, random_pool
from tests.serving_helpers import bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.lib()
    yield
    fa.device_status()


def _i32(a):
    import torch
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def _dev(pool):
    return _i32(pool.table), _i32(pool.lens), _i32(pool.holders)


def _reserve(pool, new):
    """Reserves on the device and in the oracle: equal results, which hold what a reservation promises."""
    table, lens, holders = _dev(pool)
    before, held = [list(r) for r in pool.table], list(pool.holders)
    want = pool.reserve(list(new))
    got = fa.pages_reserve(table, lens, holders, _i32(new), pool.bs)
    got = [x.tolist() for x in got]
    after = serving.Pool(table.tolist(), lens.tolist(), holders.tolist(), pool.bs)
    nobody_else_writes(after, new, got, before, held)
    assert got == [list(x) for x in want]
    assert after.table == pool.table and after.lens == pool.lens and after.holders == pool.holders
    return got


def test_a_length_set_back_to_a_page_boundary():
    pool = serving.Pool([[0, 1, -1], [-1] * 3], [32, 0], [1, 1, 0, 0], 16)
    pool.fork([0], [1])
    pool.lens[1] = 16
    assert _reserve(pool, [0, 5]) == [[1, 1], [-1, -1], [-1, -1]]
    assert pool.table == [[0, 1, -1], [0, 2, -1]] and pool.holders == [2, 1, 1, 0]
    fa.device_status()


def test_a_length_set_back_into_a_page():
    pool = serving.Pool([[0, 1, -1], [-1] * 3], [32, 0], [1, 1, 0, 0, 0], 16)
    pool.fork([0], [1])
    pool.lens[1] = 10
    assert _reserve(pool, [0, 20]) == [[1, 1], [-1, 0], [-1, 2]]
    assert pool.table == [[0, 1, -1], [2, 3, -1]]
    fa.device_status()


def test_the_last_to_hold_a_page_keeps_it():
    pool = serving.Pool([[0, 1], [0, 1], [0, 1]], [16, 0, 10], [3, 3, 0, 0, 0, 0, 0], 16)
    assert _reserve(pool, [1, 20, 20]) == [[1, 1, 1], [-1, -1, 0], [-1, -1, 5]]
    fa.device_status()


@pytest.mark.parametrize("B,per,spare,bs", [(1, 1, 2, 16), (2, 3, 1, 16), (5, 4, 9, 32), (9, 7, 40, 128), (40, 12, 60, 16),
                                            (40, 12, 400, 64), (300, 6, 900, 16), (3, 1500, 4000, 16), (1100, 3, 700, 32)])
def test_random_tables(B, per, spare, bs):
    for seed in range(6 if B * per < 2000 else 2):
        rng = np.random.default_rng(1000 * seed + B + per)
        pool = random_pool(rng, B, per, spare, bs)
        most = max(2, per * bs // int(rng.choice([1, 3, 8])))
        new = [int(rng.integers(0, max(1, min(most, per * bs - n)) + 1)) if rng.random() < 0.8 else 0 for n in pool.lens]
        over = any(n + m > per * bs for n, m in zip(pool.lens, new))
        _reserve(pool, new)
        if over:
            with pytest.raises(fa.FAError, match="length"):
                fa.device_status()
        fa.device_status()


def test_entries_missing_between_others_get_pages_and_the_others_stay():
    pool = serving.Pool([[0, -1, 4, -1], [1, -1, -1, -1]], [16, 5], [1, 1, 0, 0, 1, 0], 16)
    assert _reserve(pool, [48, 12]) == [[1, 1], [-1, -1], [-1, -1]]
    assert pool.table == [[0, 2, 4, 3], [1, 5, -1, -1]] and pool.holders == [1] * 6
    fa.device_status()


@pytest.mark.parametrize("B,per,spare,bs", [(1, 4, 3, 16), (6, 9, 12, 32), (50, 40, 900, 16), (7, 70, 400, 64), (4, 1500, 6000, 16),
                                            (1100, 5, 3000, 16)])
def test_random_tables_with_gaps(B, per, spare, bs):
    for seed in range(5):
        rng = np.random.default_rng(1000 * seed + B + per)
        pool = random_pool(rng, B, per, spare, bs, gaps=True)
        if seed % 2:  # every page held by one: the gaps alone
            used = iter(rng.permutation(sum(p >= 0 for row in pool.table for p in row) + spare).tolist())
            pool.table = [[next(used) if p >= 0 else -1 for p in row] for row in pool.table]
            pool.holders = [0] * (max(list(used) + [p for row in pool.table for p in row]) + 1)
            for p in (p for row in pool.table for p in row if p >= 0):
                pool.holders[p] = 1
        _reserve(pool, [int(rng.integers(0, per * bs - n + 1)) if rng.random() < 0.8 else 0 for n in pool.lens])
        fa.device_status()


@pytest.mark.parametrize("seed", range(4))
def test_random_loops_with_lengths_set_back(seed):
    """Forks, reservations, appends and lengths that are set back with and without giving the pages behind them up."""
    rng = np.random.default_rng(seed)
    bs, B, per = int(rng.choice([16, 64])), int(rng.choice([6, 50])), 8
    nb = B * per + (0 if seed % 2 else 20)
    pool = serving.Pool([[-1] * per for _ in range(B)], [0] * B, [0] * nb, bs)
    for step in range(30):
        what = rng.integers(0, 5)
        if what == 0:
            empty = [b for b in range(B) if pool.lens[b] == 0 and max(pool.table[b]) < 0]
            full = [b for b in range(B) if pool.lens[b]]
            if empty and full:
                dst = rng.permutation(empty)[: int(rng.integers(1, len(empty) + 1))].tolist()
                src = rng.choice(full, len(dst)).tolist()
                dev = _dev(pool)
                pool.fork(src, dst)
                fa.pages_fork(*dev, _i32(src), _i32(dst), bs)
                assert [x.tolist() for x in dev] == [pool.table, pool.lens, pool.holders]
        elif what == 1:  # as after an eviction or a rollback
            for b in range(B):
                if rng.random() < 0.4:
                    whole = int(rng.choice([1, bs]))
                    pool.lens[b] = int(rng.integers(0, pool.lens[b] + 1)) // whole * whole
        elif what == 2:
            seqs = rng.permutation(B)[: int(rng.integers(1, B + 1))].tolist()
            dev = _dev(pool)
            keep = [int(rng.integers(0, per * bs)) for _ in seqs]
            pool.free(seqs, keep)
            fa.pages_free(*dev, _i32(seqs), bs, keep_lens=_i32(keep))
            assert [x.tolist() for x in dev] == [pool.table, pool.lens, pool.holders]
        else:
            new = [int(rng.integers(0, min(3 * bs, per * bs - n) + 1)) for n in pool.lens]
            granted = _reserve(pool, new)[0]
            for b in range(B):
                pool.lens[b] += new[b] if granted[b] and rng.random() < 0.8 else 0
    fa.device_status()


def test_what_others_hold_is_not_written():
    """A prompt of three pages, forked and set back to one and a half of them: what the fork writes then leaves the prompt's
    rows as they are, and it reads its own."""
    import torch
    rng = np.random.default_rng(3)
    hkv, d, bs, nb = 2, 64, 16, 12
    table, lens, holders = torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), _i32([0, 0]), _i32([0] * nb)
    kc, vc = (torch.zeros((nb, hkv, bs, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")

    def write(count):
        n = max(count)
        granted, old, new = fa.pages_reserve(table, lens, holders, _i32(count), bs)
        assert granted.tolist() == [1, 1]
        fa.cache_copy_pages(kc, vc, old, new)
        k, v = (bf16(rng.standard_normal((2, hkv, n, d))).cuda() for _ in "kv")
        fa.cache_append(k, v, kc, vc, table, lens, new_lens=_i32(count))
        lens.add_(_i32(count))
        return k, v
    k, v = write([48, 0])
    fa.pages_fork(table, lens, holders, _i32([0]), _i32([1]), bs)
    for back in (24, 16, 0):
        lens.copy_(_i32([48, back]))
        was = [x[:1, :, :back].clone() for x in fa.cache_gather(kc, vc, table[1:].contiguous(), _i32([back]), 48)]
        k2, v2 = write([0, 48 - back])
        rows = fa.cache_gather(kc, vc, table, lens, 48)
        for got, prompt, mine, kept in zip(rows, (k, v), (k2, v2), was):
            assert torch.equal(got[0], prompt[0])
            assert torch.equal(got[1, :, :back], kept[0]) and torch.equal(got[1, :, back:], mine[1])
    fa.device_status()


@pytest.mark.parametrize("table,lens,held,match", [
    ([[0, 9, -1], [1, -1, -1]], [16, 16], [1, 1, 0, 0, 0], "block-table"),   # an id that is none behind the tokens
    ([[0, 3, -1], [1, -1, -1]], [10, 16], [1, 1, 0, 0, 0], "nobody"),        # a page that is free, by its holders
    ([[3, -1, -1], [1, -1, -1]], [10, 16], [0, 1, 0, 0, 0], "nobody"),
    ([[-1, 0, -1], [1, -1, -1]], [10, 16], [1, 1, 0, 0, 0], "block-table"),  # no page under tokens that are there
    ([[0, -1, -1], [1, -1, -1]], [-1, 16], [1, 1, 0, 0, 0], "length")])
def test_tables_that_cannot_be_are_refused_and_reported(table, lens, held, match):
    dev = _i32(table), _i32(lens), _i32(held)
    pool = serving.Pool(table, lens, held, 16)
    want = pool.reserve([20, 17])
    got = fa.pages_reserve(*dev, _i32([20, 17]), 16)
    with pytest.raises(fa.FAError, match=match):
        fa.device_status()
    assert [x.tolist() for x in got] == [list(x) for x in want] == [[0, 1], [-1, -1], [-1, -1]]
    assert [x.tolist() for x in dev] == [pool.table, lens, pool.holders] and pool.table[0] == table[0]


def test_captured_and_replayed():
    """A graph of a reservation takes the sequences in turn where the state at the replay asks for it, and not otherwise."""
    import torch
    start = random_pool(np.random.default_rng(7), 30, 6, 200, 16)
    plain = serving.Pool([[-1] * 6 for _ in range(30)], [0] * 30, [0] * len(start.holders), 16)
    new = [min(20, 96 - n) for n in start.lens]
    dev, news, ws = _dev(plain), _i32(new), torch.empty(4096, dtype=torch.uint8, device="cuda")
    fa.pages_reserve(*_dev(plain), news, 16)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fa.pages_reserve(*dev, news, 16, workspace=ws)
    for pool in (plain, start, serving.Pool(*(list(x) for x in (plain.table, plain.lens, plain.holders)), 16)):
        for t, x in zip(dev, _dev(pool)):
            t.copy_(x)
        want = pool.reserve(new)
        graph.replay()
        assert [x.tolist() for x in out] == [list(x) for x in want]
        assert [x.tolist() for x in dev] == [pool.table, pool.lens, pool.holders]
    fa.device_status()


def test_a_length_that_cannot_be_is_not_served_without_tokens_either():
    pool = serving.Pool([[0, -1], [1, -1], [2, -1]], [-1, 5, 33], [1, 1, 1], 16)
    dev = _dev(pool)
    got = fa.pages_reserve(*dev, _i32([0, 0, 0]), 16)
    with pytest.raises(fa.FAError, match="length"):
        fa.device_status()
    assert [x.tolist() for x in got] == [list(x) for x in pool.reserve([0, 0, 0])] == [[0, 1, 0], [-1] * 3, [-1] * 3]
    assert [x.tolist() for x in dev] == [pool.table, pool.lens, pool.holders]
