"""Rows moved together, pages copied, shared, freed and reserved, on the GPU against plain lists; and a serving loop that
uses them with the cache in four bits and the attention over it."""

import math

import numpy as np
import pytest

from io_aware_exact_11_gb300 import fa
from oracle import serving
from tests.four_bit_helpers import check_tree4
from tests.gpu_helpers import Guarded
from tests.serving_helpers import bf16, check_tree, np64

pytestmark = pytest.mark.gpu

CACHES = ["bf16", "e4m3", "e2m1"]


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


def _random_pool(rng, nb, hkv, bs, d, cache):
    """Pools of random bytes; returns (caches, scales, all of them as byte arrays [nb, hkv, bs, bytes])."""
    import torch
    width = {"bf16": 2 * d, "e4m3": d, "e2m1": d // 2}[cache]
    raw = [rng.integers(0, 256, (nb, hkv, bs, width)).astype(np.uint8) for _ in "kv"]
    sb = {"bf16": 0, "e4m3": 1, "e2m1": d // 32}[cache]
    scale = [rng.integers(0, 256, (nb, hkv, bs, sb)).astype(np.uint8) for _ in "kv"]
    dt = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e2m1": torch.uint8}[cache]
    dev = [torch.from_numpy(r).cuda().view(dt) for r in raw]
    sdev = [None, None]
    if sb:
        sdev = [torch.from_numpy(s if sb > 1 else s[..., 0].copy()).cuda() for s in scale]
    return dev, dict(k_scale=sdev[0], v_scale=sdev[1]), raw + (scale if sb else [])


def _same(dev, kw, host):
    import torch
    got = [t.view(torch.uint8).cpu().numpy() for t in dev] + [s.cpu().numpy() for s in kw.values() if s is not None]
    return all(np.array_equal(a.reshape(b.shape), b) for a, b in zip(got, host))


# ------------------------------------------------------------------------------------------------ rows


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,hkv,N,bs,first,kind", [
    (1, 1, 1, 16, [0], "some"), (3, 2, 8, 16, [0, 5, 40], "some"), (2, 4, 64, 32, [130, 3], "some"), (1, 2, 700, 64, [17], "rising"),
    (2, 1, 1300, 16, [0, 9], "rising"), (1, 3, 1100, 128, [2], "any"), (2, 2, 600, 16, [1, 0], "same"),
    (1, 1, 9000, 16, [100], "any"), (20, 4, 1100, 16, [3 * b for b in range(20)], "rising")])
def test_rows_are_moved_as_if_all_were_read_first(cache, d, B, hkv, N, bs, first, kind):
    rng = np.random.default_rng(N + d)
    reach = max(first) + 2 * N + 40
    per = -(-reach // bs)
    nb = B * per + 2
    dev, kw, host = _random_pool(rng, nb, hkv, bs, d, cache)
    table = rng.permutation(nb)[: B * per].reshape(B, per)
    keep, lens = np.zeros((B, N), dtype=np.int32), [int(rng.integers(0, N + 1)) if kind == "some" else N for _ in range(B)]
    for b in range(B):
        if kind in ("some", "rising"):  # rising positions, each at or behind its place
            keep[b] = first[b] + np.sort(rng.permutation(N + N // 2 + 20)[:N])
        elif kind == "any":             # in no order
            keep[b] = [rng.integers(first[b] + i, reach) for i in range(N)]
        else:                           # nothing moves but the last one
            keep[b] = first[b] + np.arange(N)
            keep[b, -1] += 3
        keep[b, lens[b]:] = -7  # not read
    want = [h.copy() for h in host]
    for b in range(B):
        of, to = keep[b, : lens[b]], first[b] + np.arange(lens[b])
        for old, new in zip(host, want):
            new[table[b][to // bs], :, to % bs] = old[table[b][of // bs], :, of % bs]
    fa.cache_compact(*dev, _i32(table), _i32(first), _i32(keep), keep_lens=_i32(lens), **kw)
    fa.device_status()
    assert _same(dev, kw, want)


def test_rows_that_cannot_be_moved_are_left_and_reported():
    rng = np.random.default_rng(3)
    dev, kw, host = _random_pool(rng, 9, 2, 16, 64, "e2m1")
    table = np.array([[0, 1, 2], [3, 4, 99], [5, 6, 7]])
    keep = _i32([[3, 2, 48, -1], [40, 10, 20, 30], [9, 9, 9, 9]])
    # row 1 before its place, rows 2 and 3 outside; a page that is none; a length that cannot be
    fa.cache_compact(*dev, _i32(table), _i32([2, 0, 0]), keep, keep_lens=_i32([4, 4, 5]), **kw)
    with pytest.raises(fa.FAError, match="pages"):
        fa.device_status()
    want = [h.copy() for h in host]
    for old, new in zip(host, want):
        new[0, :, 2] = old[0, :, 3]
        for i, t in ((1, 10), (2, 20), (3, 30)):
            new[3, :, i] = old[3 + t // 16, :, t % 16]
    assert _same(dev, kw, want)


def test_one_row_of_positions_for_all():
    import torch
    rng = np.random.default_rng(4)
    dev, kw, host = _random_pool(rng, 6, 1, 16, 128, "bf16")
    table = np.arange(6).reshape(2, 3)
    fa.cache_compact(*dev, _i32(table), _i32([4, 4]), _i32([9, 20, 33]))
    want = [h.copy() for h in host]
    for old, new in zip(host, want):
        for b in range(2):
            for i, t in enumerate((9, 20, 33)):
                new[3 * b, :, 4 + i] = old[3 * b + t // 16, :, t % 16]
    assert _same(dev, kw, want)
    with pytest.raises(ValueError):
        fa.cache_compact(*dev, _i32(table), _i32([4, 4]), _i32([[1], [2], [3]]))
    with pytest.raises(TypeError):
        fa.cache_compact(*dev, _i32(table), _i32([4, 4]), torch.zeros((2, 3), device="cuda"))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d,hkv,bs", [(64, 1, 16), (128, 4, 16), (128, 8, 128), (64, 3, 64)])
def test_pages_are_copied(cache, d, hkv, bs):
    rng = np.random.default_rng(d + bs)
    dev, kw, host = _random_pool(rng, 40, hkv, bs, d, cache)
    order = rng.permutation(40)
    src, dst = order[:15].copy(), order[15:30].copy()
    src[4] = dst[4] = -1
    src[5] = dst[5]
    src[6] = src[7]  # one page to two
    want = [h.copy() for h in host]
    for old, new in zip(host, want):
        for s, t in zip(src, dst):
            if s >= 0:
                new[t] = old[s]
    fa.cache_copy_pages(*dev, _i32(src), _i32(dst), **kw)
    fa.device_status()
    assert _same(dev, kw, want)
    fa.cache_copy_pages(*dev, _i32([-1, 40, 3, -2]), _i32([2, 1, 40, -2]), **kw)  # no pages: nothing is copied
    with pytest.raises(fa.FAError, match="block-table"):
        fa.device_status()
    assert _same(dev, kw, want)


# ------------------------------------------------------------------------------------------------ pages


def _dev(pool):
    return _i32(pool.table), _i32(pool.lens), _i32(pool.holders)


def _agree(dev, pool):
    return all(np.array_equal(a.cpu().numpy(), np.array(b)) for a, b in zip(dev, (pool.table, pool.lens, pool.holders)))


@pytest.mark.parametrize("seed", range(12))
def test_random_loops_agree_with_lists(seed):
    """Forks, reservations, appends, rollbacks and frees in a random order, some of them for want of pages in part."""
    rng = np.random.default_rng(seed)
    bs, B = int(rng.choice([16, 32, 64, 128])), int(rng.choice([1, 5, 33, 300]))
    per = int(rng.integers(1, 40))
    nb = int(rng.choice([max(2, B * per // 3), B * per + 5, 9000]))
    pool = serving.Pool([[-1] * per for _ in range(B)], [0] * B, [0] * nb, bs)
    table, lens, holders = _dev(pool)
    for step in range(25):
        what = rng.integers(0, 4)
        if what == 0:
            n = int(rng.integers(1, B + 1))
            src, dst = (rng.integers(0, B, n).tolist() for _ in range(2))
            pool.fork(src, dst)
            fa.pages_fork(table, lens, holders, _i32(src), _i32(dst), bs)
        elif what == 1:
            n = int(rng.integers(1, B + 1))
            seqs = rng.permutation(B)[:n].tolist()
            keep = None if rng.random() < 0.3 else rng.integers(0, per * bs + 1, n).tolist()
            pool.free(seqs, keep)
            fa.pages_free(table, lens, holders, _i32(seqs), bs, keep_lens=None if keep is None else _i32(keep))
        else:
            new = (rng.integers(0, int(rng.choice([2, 40, 400])), B) * (rng.random(B) < 0.7)).tolist()
            want = pool.reserve(new)
            got = fa.pages_reserve(table, lens, holders, _i32(new), bs)
            assert all(np.array_equal(a.cpu().numpy(), np.array(b)) for a, b in zip(got, want)), step
            if rng.random() < 0.8:  # the tokens are written; else the pages stay reserved
                for b in range(B):
                    pool.lens[b] += new[b] if want[0][b] else 0
                lens += _i32(new) * got[0]
        assert _agree((table, lens, holders), pool), step
    try:
        fa.device_status()  # pairs of a fork that were left out, lengths beyond the table
    except fa.FAError as e:
        assert e.status == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("nb,used", [(5000, 4990), (4097, 4096), (100000, 70000), (3, 1)])
def test_free_pages_are_found_wherever_they_are(nb, used):
    """Holders at an odd address, free pages few, far apart or at the very end."""
    import torch
    rng = np.random.default_rng(nb)
    held = np.zeros(nb, dtype=np.int64)
    held[rng.permutation(nb)[:used]] = 1
    B, per, bs = 40, 70, 16
    pool = serving.Pool([[-1] * per for _ in range(B)], [0] * B, held.tolist(), bs)
    table, lens, _ = _dev(pool)
    holders = torch.zeros(nb + 1, dtype=torch.int32, device="cuda")[1:]
    holders.copy_(_i32(held))
    for most in (20, 1100):
        new = rng.integers(0, most, B).tolist()
        want = pool.reserve(new)
        got = fa.pages_reserve(table, lens, holders, _i32(new), bs)
        assert all(np.array_equal(a.cpu().numpy(), np.array(b)) for a, b in zip(got, want))
        assert _agree((table, lens, holders), pool)
    fa.device_status()


def test_many_sequences_write_into_shared_pages():
    """4096 sequences in groups that share a last page, interleaved, with a holder that does not write and one too short
    of pages."""
    rng = np.random.default_rng(8)
    B, bs, G = 4096, 16, 512
    pool = serving.Pool([[-1] * 4 for _ in range(B)], [0] * B, [0] * 5000, bs)
    pool.reserve([20 if b % G == 0 else 0 for b in range(B)])
    for b in range(0, B, G):
        pool.lens[b] = 20
    dst = [b for b in rng.permutation(B).tolist() if b % G]
    src = [int(rng.integers(0, B // G)) * G for _ in dst]
    pool.fork(src, dst)
    table, lens, holders = _dev(pool)
    new = np.ones(B, dtype=int)
    new[rng.permutation(B)[:3]] = 0
    new[100:110] = 30
    want = pool.reserve(new.tolist())
    got = fa.pages_reserve(table, lens, holders, _i32(new), bs)
    assert all(np.array_equal(a.cpu().numpy(), np.array(b)) for a, b in zip(got, want))
    assert _agree((table, lens, holders), pool)
    fa.device_status()


def test_reserved_pages_are_given_back_up_to_the_lengths_themselves():
    import torch
    B, bs, nb, per = 300, 16, 4000, 12
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 5 * bs, B)
    table, held = np.full((B, per), -1), np.zeros(nb, dtype=int)
    order = iter(rng.permutation(nb))
    for b in range(B):
        for j in range(-(-lens[b] // bs)):
            table[b, j] = next(order)
            held[table[b, j]] = 1
    t, n, h = _i32(table), _i32(lens), _i32(held)
    granted, _, _ = fa.pages_reserve(t, n, h, _i32(rng.integers(1, 6 * bs, B)), bs)
    assert granted.all() and int(h.sum()) > held.sum()
    fa.pages_free(t, n, h, _i32(np.arange(B)), bs, keep_lens=n)
    fa.device_status()
    assert torch.equal(t, _i32(table)) and torch.equal(n, _i32(lens)) and torch.equal(h, _i32(held))


def test_bad_sequences_lengths_and_pages_are_left_out_and_reported():
    start = ([[0, 1, -1], [2, -1, -1], [-1] * 3, [-1] * 3], [20, 7, 0, 0], [1, 1, 1, 0, 0, 0, 0])

    def fresh():
        pool = serving.Pool(*start, 16)
        return pool, _dev(pool)

    def reported(match):
        with pytest.raises(fa.FAError, match=match) as e:
            fa.device_status()
        assert e.value.status == fa.FA_ERR_INVALID_ARG
    # no row of the table; dst not empty; named twice; read and filled
    for src, dst in (([0, 4], [2, 3]), ([0, 0], [2, -1]), ([0, 0], [2, 1]), ([0, 1], [3, 3]), ([0, 2], [2, 3])):
        pool, dev = fresh()
        pool.fork(src, dst)
        fa.pages_fork(*dev, _i32(src), _i32(dst), 16)
        reported("sequence")
        assert _agree(dev, pool)
    for seqs, keep, match in (([0, 7], None, "sequence"), ([1, 1], [3, 0], "sequence"), ([0, 1], [5, -1], "length")):
        pool, dev = fresh()
        pool.free(seqs, keep)
        fa.pages_free(*dev, _i32(seqs), 16, keep_lens=None if keep is None else _i32(keep))
        reported(match)
        assert _agree(dev, pool)
    pool, dev = fresh()
    want = pool.reserve([30, -1, 17, 49])
    got = fa.pages_reserve(*dev, _i32([30, -1, 17, 49]), 16)
    reported("length")
    assert all(np.array_equal(a.cpu().numpy(), np.array(b)) for a, b in zip(got, want)) and _agree(dev, pool)
    assert want[0] == [0, 0, 1, 0]
    # a page that is none under the next token; the others are served
    table, lens, held = _i32([[0, 77, -1], [2, -1, -1]]), _i32([20, 7]), _i32([1, 1, 1, 0])
    granted, src, dst = fa.pages_reserve(table, lens, held, _i32([1, 12]), 16)
    reported("block-table")
    assert granted.tolist() == [0, 1] and table.tolist() == [[0, 77, -1], [2, 3, -1]] and held.tolist() == [1, 1, 1, 1]
    # a page that nobody was said to hold, and one that is none
    table, lens, held = _i32([[0, 5], [1, -1]]), _i32([20, 9]), _i32([0, 1])
    fa.pages_free(table, lens, held, _i32([0, 1]), 16)
    reported("pages")
    assert held.tolist() == [0, 0] and table.tolist() == [[-1, -1]] * 2 and lens.tolist() == [0, 0]


def test_guards_and_workspace():
    import torch
    B, nb = 70, 9000
    pool = serving.Pool([[-1] * 5 for _ in range(B)], [0] * B, [0] * nb, 16)
    g = [Guarded((B, 5), torch.int32), Guarded((B,), torch.int32), Guarded((nb,), torch.int32)]
    for t, x in zip(g, _dev(pool)):
        t.t.copy_(x)
    size = fa.pages_reserve_workspace_size(B, nb)
    ws = Guarded((size,), torch.uint8)
    want = pool.reserve([33] * B)
    got = fa.pages_reserve(*(t.t for t in g), _i32([33] * B), 16, workspace=ws.t)
    assert got[0].tolist() == want[0] and _agree([t.t for t in g], pool)
    pool.lens = [33] * B
    g[1].t.fill_(33)
    pool.free(list(range(B)), [17] * B)
    fa.pages_free(*(t.t for t in g), _i32(range(B)), 16, keep_lens=_i32([17] * B))
    assert _agree([t.t for t in g], pool) and all(t.intact() for t in g) and ws.intact()
    with pytest.raises(fa.FAError):
        fa.pages_reserve(*(t.t for t in g), _i32([1] * B), 16, workspace=ws.t[: size - 256])
    with pytest.raises(TypeError):
        fa.pages_reserve(*(t.t for t in g), _i32([1] * B).long(), 16)
    with pytest.raises(TypeError):
        fa.pages_fork(*(t.t for t in g), _i32([1, 2]), _i32([3]), 16)
    with pytest.raises(TypeError):
        fa.pages_free(g[0].t, g[1].t, g[2].t.view(B * 0 + 90, 100), _i32([1]), 16)
    fa.device_status()


# ------------------------------------------------------------------------------------------------ together


class _Cached:
    """What the oracle sees of a cache: the rows of each sequence as read back."""

    def __init__(self, k, v, lens, cache):
        self.hkv, self.cache = k.shape[1], cache
        self.k, self.v = ([np64(t[b, :, :n]) for b, n in enumerate(lens)] for t in (k, v))


@pytest.mark.parametrize("cache", CACHES)
def test_a_loop_of_forked_sequences(cache):
    """A prompt is written once, continued in three ways (its last page shared), drafts are attended, the accepted ones
    moved together and the rest given back: every sequence's rows are those that it would have alone."""
    import torch
    rng = np.random.default_rng(21)
    B, hkv, Hq, d, bs, per, nb, T = 4, 2, 8, 64, 16, 8, 40, 4
    width = {"bf16": d, "e4m3": d, "e2m1": d // 2}[cache]
    dt = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e2m1": torch.uint8}[cache]
    kc, vc = (torch.zeros((nb, hkv, bs, width), dtype=torch.uint8, device="cuda").to(torch.float32).to(dt) for _ in "kv")
    kw = {}
    if cache != "bf16":
        shape = (nb, hkv, bs) if cache == "e4m3" else (nb, hkv, bs, d // 32)
        kw = {n: torch.full(shape, 127, dtype=torch.uint8, device="cuda") for n in ("k_scale", "v_scale")}
    table = torch.full((B, per), -1, dtype=torch.int32, device="cuda")
    lens, holders = _i32([0] * B), _i32([0] * nb)
    rows = [[np.zeros((hkv, 0, d)) for _ in "kv"] for _ in range(B)]  # what each sequence was given
    w, axes = fa.rope_frequencies(d)[0], np.arange(d // 2) % 3

    def write(count, n):
        """n new tokens (count[b] of them real), rotated on three axes, for every sequence."""
        granted, old, new = fa.pages_reserve(table, lens, holders, _i32(count), bs)
        assert granted.tolist() == [1] * B
        fa.cache_copy_pages(kc, vc, old, new, **kw)
        k, v = (bf16(rng.standard_normal((B, hkv, n, d))).cuda() for _ in "kv")
        at = (lens[:, None] + torch.arange(n, device="cuda").int()).int()
        q, k = fa.rope_axes(bf16(rng.standard_normal((B, Hq, n, d))).cuda(), k, w, axes, at[None].expand(3, B, n))
        fa.cache_append(k, v, kc, vc, table, lens, new_lens=_i32(count), **kw)
        return q, k, v

    def held(x):
        x = np64(x)
        if cache == "e4m3":
            y, e = serving.quantise_rows(x)
            return y * 2.0 ** e[..., None]
        return serving.quantise_groups(x)[2] if cache == "e2m1" else x

    _, k, v = write([37, 0, 0, 0], 37)
    rows[0] = [held(k[0]), held(v[0])]
    lens += _i32([37, 0, 0, 0])
    fa.pages_fork(table, lens, holders, _i32([0, 0, 0]), _i32([1, 2, 3]), bs)
    rows[1:] = [list(rows[0]) for _ in range(3)]
    assert int(holders.max()) == 4 and int((holders > 0).sum()) == 3
    for step in range(3):
        q, k, v = write([T] * B, T)
        total = lens + T
        o, lse = fa.decode_tree(q, kc, vc, table, total, **kw)
        n = [r[0].shape[1] + T for r in rows]
        full = _Cached(*fa.cache_gather(kc, vc, table, total, max(n), **kw), n, cache)
        for b in range(B):
            assert np.array_equal(full.k[b], np.concatenate([rows[b][0], held(k[b])], 1))
            assert np.array_equal(full.v[b], np.concatenate([rows[b][1], held(v[b])], 1))
        (check_tree4 if cache == "e2m1" else check_tree)(o, lse, q, full, [T] * B, None, 1 / math.sqrt(d), [0, Hq - 1])
        # Some drafts of each are accepted.
        taken = [sorted(rng.permutation(T)[: int(rng.integers(0, T + 1))].tolist()) for _ in range(B)]
        keep = np.zeros((B, T), dtype=np.int32)
        for b in range(B):
            keep[b, : len(taken[b])] = n[b] - T + np.array(taken[b], dtype=np.int64)
            for i, x in enumerate((k, v)):
                rows[b][i] = np.concatenate([rows[b][i], held(x[b])[:, taken[b]]], 1)
        fa.cache_compact(kc, vc, table, lens, _i32(keep), keep_lens=_i32([len(t) for t in taken]), **kw)
        lens += _i32([len(t) for t in taken])
        fa.pages_free(table, lens, holders, _i32(range(B)), bs, keep_lens=lens.clone())
        n = lens.tolist()
        back = fa.cache_gather(kc, vc, table, lens, max(n), **kw)
        for b in range(B):
            assert np.array_equal(np64(back[0][b, :, : n[b]]), rows[b][0]) and np.array_equal(np64(back[1][b, :, : n[b]]), rows[b][1])
    fa.pages_free(table, lens, holders, _i32([3, 1, 0, 2]), bs)
    assert int(holders.abs().max()) == 0 and int(table.max()) == -1
    fa.device_status()


def test_captured_replayed_and_on_other_streams():
    """Reservation, copies, writing, attention, compaction and freeing as one graph: replays give what eager calls do, on
    the state that they find; and the same on a stream of its own."""
    import torch
    rng = np.random.default_rng(22)
    B, hkv, Hq, d, bs, per, nb, T = 3, 1, 4, 128, 16, 12, 64, 2

    def state():
        z = [torch.zeros((nb, hkv, bs, d // 2), dtype=torch.uint8, device="cuda") for _ in "kv"]
        s = {n: torch.full((nb, hkv, bs, d // 32), 127, dtype=torch.uint8, device="cuda") for n in ("k_scale", "v_scale")}
        return z, s, torch.full((B, per), -1, dtype=torch.int32, device="cuda"), _i32([0] * B), _i32([0] * nb)

    k, v = (bf16(rng.standard_normal((B, hkv, T, d))).cuda() for _ in "kv")
    q = bf16(rng.standard_normal((B, Hq, T, d))).cuda()
    fork, keep_n, every = (_i32([0]), _i32([2])), _i32([1, 2, 0]), _i32(range(B))

    def step(st, stream=None):
        z, s, table, lens, held = st
        granted, old, new = fa.pages_reserve(table, lens, held, _new, bs, stream=stream)
        fa.cache_copy_pages(*z, old, new, stream=stream, **s)
        fa.cache_append(k, v, *z, table, lens, new_lens=_new, stream=stream, **s)
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            total = lens + _new
        out = fa.decode_tree(q, *z, table, total, draft_lens=_new, stream=stream, **s)
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            keep = torch.stack([lens + 1, lens + 1], 1).contiguous()
            got = torch.minimum(keep_n, _new // 2)
        fa.cache_compact(*z, table, lens, keep, keep_lens=got, stream=stream, **s)
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            lens += got
            left = lens.clone()
        fa.pages_free(table, lens, held, every, bs, keep_lens=left, stream=stream)
        return out

    _new = _i32([T, T, 0])
    eager, captured, other = state(), state(), state()
    step(state())  # first launches outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(captured)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(40):
        if i == 20:
            for st in (eager, captured, other):
                torch.cuda.synchronize()
                fa.pages_fork(*st[2:], *fork, bs)
            torch.cuda.synchronize()
            _new.copy_(_i32([T, 0, T]))
            torch.cuda.synchronize()
        want = step(eager)
        graph.replay()
        there = step(other, stream=side)
        torch.cuda.synchronize()
        for a, b, c in zip(want, out, there):
            assert torch.equal(a, b) and torch.equal(a, c), i
        for a, b, c in zip(eager[2:], captured[2:], other[2:]):
            assert torch.equal(a, b) and torch.equal(a, c), i
    assert eager[3].tolist() == [40, 20, 20 + 0]
    fa.device_status()
