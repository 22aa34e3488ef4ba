"""The oracle's page pool where a table names pages behind its sequence's tokens: what a reservation promises (no GPU)."""

import numpy as np
import pytest

from oracle import serving
from tests.pages_helpers import nobody_else_writes, random_pool


def test_a_length_set_back_to_a_page_boundary():
    p = serving.Pool([[0, 1, -1], [-1] * 3], [32, 0], [1, 1, 0, 0], 16)
    p.fork([0], [1])
    p.lens[1] = 16
    assert p.reserve([0, 5]) == ([1, 1], [-1, -1], [-1, -1])  # nothing of the sequence lies there to be copied
    assert p.table == [[0, 1, -1], [0, 2, -1]] and p.holders == [2, 1, 1, 0]


def test_a_length_set_back_into_a_page():
    p = serving.Pool([[0, 1, -1], [-1] * 3], [32, 0], [1, 1, 0, 0, 0], 16)
    p.fork([0], [1])
    p.lens[1] = 10
    assert p.reserve([0, 20]) == ([1, 1], [-1, 0], [-1, 2])
    assert p.table == [[0, 1, -1], [2, 3, -1]] and p.holders == [1, 1, 1, 1, 0]


def test_the_last_to_hold_a_page_keeps_it():
    p = serving.Pool([[0, 1], [0, 1], [0, 1]], [16, 0, 10], [3, 3, 0, 0, 0, 0, 0], 16)
    assert p.reserve([1, 20, 20]) == ([1, 1, 1], [-1, -1, 0], [-1, -1, 5])
    assert p.table == [[0, 2], [3, 4], [5, 1]] and p.holders == [1, 1, 1, 1, 1, 1, 0]


@pytest.mark.parametrize("gaps", [False, True])
@pytest.mark.parametrize("seed", range(200))
def test_no_page_that_is_written_has_another_holder(seed, gaps):
    rng = np.random.default_rng(seed)
    pool = random_pool(rng, int(rng.integers(1, 9)), int(rng.integers(1, 7)), int(rng.integers(0, 25)), 16, gaps)
    new = rng.integers(0, 40, len(pool.lens)).tolist()
    before, held = [list(r) for r in pool.table], list(pool.holders)
    out = pool.reserve(new)
    nobody_else_writes(pool, new, out, before, held)


def test_a_length_that_cannot_be_is_not_served_without_tokens_either():
    p = serving.Pool([[0, -1], [1, -1], [2, -1]], [-1, 5, 33], [1, 1, 1], 16)
    assert p.reserve([0, 0, 0]) == ([0, 1, 0], [-1] * 3, [-1] * 3)
