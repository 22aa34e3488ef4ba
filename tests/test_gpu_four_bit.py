"""The paged cache in four bits on the GPU against the float64 oracle: rows written and read back, and attention over it."""

import math

import numpy as np
import pytest

from io_aware_exact_11_gb300 import fa
from oracle import serving
from tests.four_bit_helpers import Paged4, check_tree4, pack, values
from tests.gpu_helpers import Guarded
from tests.serving_helpers import bf16, np64, random_tree

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


def _mask(m):
    import torch
    return None if m is None else torch.from_numpy(m).cuda()


def _pools(nb, hkv, bs, d):
    import torch
    code = [torch.full((nb, hkv, bs, d // 2), 0x7F, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scale = [torch.full((nb, hkv, bs, d // 32), 255, dtype=torch.uint8, device="cuda") for _ in "kv"]
    return code, dict(k_scale=scale[0], v_scale=scale[1])


# ------------------------------------------------------------------------------------------------ rows


def _edges(rng, shape):
    """Rows with halfway values, powers of two far apart, zeros, subnormal and largest numbers, infinities and NaN."""
    x = np64(bf16(rng.standard_normal(shape) * np.exp2(rng.integers(-3, 4, (*shape[:-1], 1)))))
    flat = x.reshape(-1, shape[-1])
    kinds = [lambda r: np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], len(r) // 8) * rng.choice([-1, 1], len(r)),
             lambda r: r * 0.0, lambda r: r * 2.0 ** -128, lambda r: np.full(len(r), 2.0 ** -133), lambda r: r * 2.0 ** 120,
             lambda r: np.where(np.arange(len(r)) == 3, -3.3895e38, r), lambda r: np.where(np.arange(len(r)) == 40, np.inf, r),
             lambda r: np.where(np.arange(len(r)) == 1, np.nan, r), lambda r: -0.0 * np.abs(r),
             lambda r: r * np.exp2(np.arange(len(r)) % 60 - 30.0)]
    for i in range(len(flat)):
        if i % 3 == 0:
            flat[i] = kinds[i // 3 % len(kinds)](flat[i])
    return np64(bf16(flat.reshape(shape)))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,hkv,N,bs,bnhd,lens", [
    (1, 1, 1, 16, False, None), (3, 2, 7, 32, True, [7, 0, 3]), (2, 4, 65, 64, False, [65, 64]), (64, 4, 1, 16, True, None),
    (1, 8, 130, 128, False, None), (2, 8, 5000, 16, True, [5000, 4321])])
def test_rows_are_quantised_and_read_back(d, B, hkv, N, bs, bnhd, lens):
    import torch
    rng = np.random.default_rng(N + d)
    start = [int(s) for s in rng.integers(0, 50, B)]
    real = lens if lens is not None else [N] * B
    per = -(-(max(start) + N) // bs)
    nb = B * per + 2
    (kc, vc), sc = _pools(nb, hkv, bs, d)
    before = [t.clone() for t in (kc, vc, sc["k_scale"], sc["v_scale"])]
    table = rng.permutation(nb)[: B * per].reshape(B, per)
    x = {n: _edges(rng, (B, hkv, N, d)) if N < 1000 else np64(bf16(rng.standard_normal((B, hkv, N, d)))) for n in "kv"}
    dev = {n: bf16(x[n]).cuda() for n in "kv"}
    if bnhd:
        dev = {n: t.transpose(1, 2).contiguous().transpose(1, 2) for n, t in dev.items()}
    fa.cache_append(dev["k"], dev["v"], kc, vc, _i32(table), _i32(start), new_lens=None if lens is None else _i32(lens), **sc)
    L = max(start) + N
    gk, gv = fa.cache_gather(kc, vc, _i32(table), _i32([s + n for s, n in zip(start, real)]), L, **sc)
    fa.device_status()
    written = np.zeros((nb, bs), dtype=bool)
    for name, cache, scale, back, old, old_s in (("k", kc, sc["k_scale"], gk, before[0], before[2]),
                                                 ("v", vc, sc["v_scale"], gv, before[1], before[3])):
        cache, scale, back = cache.cpu().numpy(), scale.cpu().numpy(), np64(back)
        for b in range(B):
            at = start[b] + np.arange(real[b])
            page, slot = table[b][at // bs], at % bs
            written[page, slot] = True
            c, s, y = serving.quantise_groups(x[name][b, :, : real[b]])
            assert np.array_equal(scale[page, :, slot].transpose(1, 0, 2), s)
            assert np.array_equal(cache[page, :, slot].transpose(1, 0, 2), pack(c))
            assert np.array_equal(back[b, :, start[b] : start[b] + real[b]], y, equal_nan=True)
            assert (back[b, :, start[b] + real[b] :] == 0).all()
        assert np.array_equal(cache.transpose(0, 2, 1, 3)[~written], old.cpu().numpy().transpose(0, 2, 1, 3)[~written])
        assert np.array_equal(scale.transpose(0, 2, 1, 3)[~written], old_s.cpu().numpy().transpose(0, 2, 1, 3)[~written])


def test_every_code_and_scale_reads_back_exactly():
    import torch
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 256, (16, 1, 16, 64)).astype(np.uint8)
    scales = np.arange(16 * 16 * 4).reshape(16, 1, 16, 4).astype(np.uint8)  # every byte, four times
    table, n = _i32(np.arange(16)[None]), 256
    k, v = fa.cache_gather(*(torch.from_numpy(codes).cuda() for _ in "kv"), table, _i32([n]), n,
                           **{s: torch.from_numpy(scales).cuda() for s in ("k_scale", "v_scale")})
    want = values(codes, scales).reshape(1, 1, n, 128)
    # The two largest powers of two take the largest codes beyond bf16, whose values are infinite there.
    want = np.where(np.abs(want) > 3.4e38, np.copysign(np.inf, want), want)
    assert np.array_equal(np64(k), want, equal_nan=True) and np.array_equal(np64(v), want, equal_nan=True)


def test_bad_pages_and_lengths_are_reported():
    import torch
    rng = np.random.default_rng(2)
    (kc, vc), sc = _pools(4, 2, 16, 128)
    x = bf16(rng.standard_normal((2, 2, 20, 128))).cuda()
    table = _i32([[0, 99], [1, 2]])
    fa.cache_append(x, x, kc, vc, table, _i32([0, 0]), **sc)
    with pytest.raises(fa.FAError, match="block-table"):
        fa.device_status()
    k, _ = fa.cache_gather(kc, vc, table, _i32([20, 99]), 20, **sc)
    with pytest.raises(fa.FAError, match="paged cache"):
        fa.device_status()
    y = serving.quantise_groups(np64(x))[2]
    k = np64(k)
    assert np.array_equal(k[0, :, :16], y[0, :, :16]) and (k[0, :, 16:] == 0).all() and (k[1] == 0).all()
    assert (kc[3] == 0x7F).all()
    q = bf16(rng.standard_normal((2, 2, 1, 128))).cuda()
    fa.decode_tree(q, kc, vc, table, _i32([20, 20]), **sc)
    with pytest.raises(fa.FAError, match="decode tree"):
        fa.device_status()


# ------------------------------------------------------------------------------------------------ attention


def _run(seed, lens, Hq, hkv, T, d, bs, mask=None, drafts=None, parts=0, heads=None, q_scale=1.0, edit=None, **kw):
    rng = np.random.default_rng(seed)
    p = Paged4(rng, lens, hkv, d, bs, edit=edit)
    q = bf16(rng.standard_normal((len(lens), Hq, T, d)) * q_scale).cuda()
    if isinstance(mask, str):
        mask = random_tree(rng, len(lens), T, empty={"tree": 0.0, "holes": 0.4}[mask])
    scale = kw.pop("scale", 1 / math.sqrt(d))
    o, lse = fa.decode_tree(q, *p.args(), tree_mask=_mask(mask), draft_lens=None if drafts is None else _i32(drafts),
                            max_parts=parts, scale=scale, **p.kw(), **kw)
    fa.device_status()
    real = drafts if drafts is not None else [T if n else 0 for n in lens]
    check_tree4(o, lse, q, p, real, mask, scale, heads)
    return o, lse, q, p


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,Hq,hkv,T,bs,mask,drafts", [
    ([1], 1, 1, 1, 16, None, None),
    ([5, 128, 129, 127], 7, 1, 1, 16, None, None),
    ([130, 64, 300], 28, 4, 5, 16, "tree", None),
    ([8, 9, 260], 4, 2, 8, 64, "holes", None),
    ([33, 0, 700], 8, 2, 3, 32, "tree", None),
    ([40, 500, 3, 0], 8, 1, 12, 128, "tree", [12, 3, 3, 0]),
    ([257, 1000], 16, 1, 1, 32, None, None),
    ([90, 140], 17, 1, 1, 16, None, None),
    ([100, 257], 16, 2, 64, 64, "tree", [64, 50]),
    ([300], 2, 1, 130, 16, "holes", None),
    ([256], 1, 1, 256, 128, None, None)])
def test_tree(d, lens, Hq, hkv, T, bs, mask, drafts):
    for parts in (0, 1, 3):
        _run(T * d, lens, Hq, hkv, T, d, bs, mask, drafts, parts, heads=sorted({0, Hq // 2, Hq - 1}))


@pytest.mark.parametrize("parts", [1, 2, 7, 64, 256])
def test_parts_of_a_long_sequence(parts):
    _run(5, [4000, 1, 2047], 8, 2, 2, 128, 16, None, [2, 1, 2], parts, heads=[0, 7])


@pytest.mark.parametrize("T,G", [(1, 1), (3, 11), (3, 43), (5, 40)])
def test_many_pieces_and_pairs(T, G):
    """Short sequences, so that every part holds several, and some that are empty, one tile or cut in the middle."""
    _run(11, [128, 0, 129, 700, 1 + T, 256, 384, 0, 127], 2 * G, 2, T, 128, 32, "tree" if T > 1 else None, None, 5,
         heads=[0, G, 2 * G - 1])


def test_large_scores_and_rising_maxima():
    def rising(name, b, x):
        if name == "k":
            x *= np.linspace(0.1, 3, x.shape[1])[None, :, None]
    for Hq in (4, 24, 80):
        _run(7, [1500, 1000], Hq, 2, 4, 128, 32, "tree", parts=2, q_scale=8.0, edit=rising, heads=[0, Hq - 1])


@pytest.mark.parametrize("Hq", [4, 24, 80])
def test_rows_and_groups_of_very_different_size(Hq):
    """Powers of two up to 2^±20 apart from row to row, and of a row from group to group, in keys and values."""
    def spread(name, b, x):
        rows = np.exp2((np.arange(x.shape[1]) * 37 % 41) - 20.0)[None, :, None]
        groups = np.exp2((np.arange(x.shape[2]) // 32 * 13 % 17) - 12.0)[None, None]
        x *= groups * (rows if name == "v" else 1.0)
        x[:, 3] = 0.0
    _run(8, [700, 513], Hq, 2, 3, 128, 16, "tree", parts=3, edit=spread, heads=[0, Hq - 1])


@pytest.mark.parametrize("Hq", [2, 24, 60])
def test_what_unseen_drafted_keys_hold_does_not_matter(Hq):
    """Drafted token 2's key and value are NaN; only rows that see it may show it."""
    T = 6
    mask = np.tril(np.ones((1, T, T), dtype=bool))
    mask[:, :, 2] = False
    mask[0, 4, 2] = True
    mask[0, 5] = False

    def poison(name, b, x):
        x[:, x.shape[1] - T + 2] = np.nan
    for n in (T, 131, 128 + T):
        rng = np.random.default_rng(9)
        p = Paged4(rng, [n], 1, 128, 16, edit=poison)
        q = bf16(rng.standard_normal((1, Hq, T, 128))).cuda()
        o, lse = (np64(x) for x in fa.decode_tree(q, *p.args(), tree_mask=_mask(mask), max_parts=2, **p.kw()))
        assert np.isnan(o[:, :, 4]).all() and not np.isfinite(lse[:, :, 4]).any()
        mask2 = mask.copy()
        mask2[0, 4, 2] = False
        clean = Paged4(np.random.default_rng(9), [n], 1, 128, 16,
                       edit=lambda name, b, x: x.__setitem__((slice(None), x.shape[1] - T + 2), 0.0))
        ro, rl = (np64(x) for x in fa.decode_tree(q, *clean.args(), tree_mask=_mask(mask2), max_parts=2, **clean.kw()))
        rows = [0, 1, 2, 3, 5]
        assert np.array_equal(o[:, :, rows], ro[:, :, rows]) and np.array_equal(lse[:, :, rows], rl[:, :, rows])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq", [2, 24, 60, 128])
def test_huge_drafted_keys_reach_those_who_see_them_alone(Hq, d):
    """Drafted token 2's key is 2^50 to 2^100 times the others'.  (Those are multiplied by whole powers of two less, which is
    exact: rows that do not see it have the bits that they have without it.)"""
    T = 6
    mask = np.tril(np.ones((1, T, T), dtype=bool))
    mask[:, :, 2] = False
    for n in (T, 131, 128 + T):
        for power in (50, 100):
            def grow(name, b, x):
                if name == "k":
                    x[:, x.shape[1] - T + 2] = 2.0 ** power * np.where(np.arange(d) // 32 == 1, 2.0 ** -30, 1.0)
            p = Paged4(np.random.default_rng(11), [n], 1, d, 16, edit=grow)
            q = bf16(np.abs(np.random.default_rng(3).standard_normal((1, Hq, T, d)))).cuda()
            clean = Paged4(np.random.default_rng(11), [n], 1, d, 16,
                           edit=lambda name, b, x: x.__setitem__((slice(None), x.shape[1] - T + 2), 0.0) if name == "k" else None)
            seen = mask.copy()
            seen[0, 4, 2] = True
            o, lse = (np64(x) for x in fa.decode_tree(q, *p.args(), tree_mask=_mask(seen), max_parts=2, **p.kw()))
            ro, rl = (np64(x) for x in fa.decode_tree(q, *clean.args(), tree_mask=_mask(mask), max_parts=2, **clean.kw()))
            rows = [0, 1, 2, 3, 5]
            assert np.array_equal(o[:, :, rows], ro[:, :, rows]) and np.array_equal(lse[:, :, rows], rl[:, :, rows])
            fa.device_status()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq", [3, 30, 90, 128])
def test_a_huge_key_of_the_context_leaves_the_others_alone(Hq, d):
    """Far below the others' scores it has no weight, however large it is: the same bits."""
    def run(size):
        def grow(name, b, x):
            if name == "k":
                x[:, 70] = size
                x[:, 200, 32:] *= 2.0 ** -28
        p = Paged4(np.random.default_rng(21), [400, 300], 1, d, 16, edit=grow)
        q = bf16(np.abs(np.random.default_rng(4).standard_normal((2, Hq, 2, d)))).cuda()
        o, lse = (np64(x) for x in fa.decode_tree(q, *p.args(), max_parts=3, **p.kw()))
        fa.device_status()
        return o, lse
    o, lse = run(-2.0 ** 12)
    for power in (40, 80, 110):
        far, far_lse = run(-2.0 ** power)
        assert np.array_equal(o, far) and np.array_equal(lse, far_lse)


@pytest.mark.parametrize("Hq", [1, 20, 70])
def test_a_nan_value_of_the_context_reaches_its_group_alone(Hq):
    def poison(name, b, x):
        if name == "v":
            x[:, 50, 70] = np.nan
    rng = np.random.default_rng(12)
    p = Paged4(rng, [200], 1, 128, 16, edit=poison)
    q = bf16(rng.standard_normal((1, Hq, 2, 128))).cuda()
    o = np64(fa.decode_tree(q, *p.args(), **p.kw())[0])
    assert np.isnan(o[..., 64:96]).all() and np.isfinite(o[..., :64]).all() and np.isfinite(o[..., 96:]).all()


@pytest.mark.parametrize("Hq,T", [(4, 1), (16, 2), (28, 8), (64, 4)])
def test_strided_in_place_guarded_and_repeated(Hq, T):
    """Strided queries, results over the queries, a workspace of the smallest size, neighbours untouched, equal bits."""
    import torch
    rng = np.random.default_rng(13)
    p = Paged4(rng, [300, 77], 2 if Hq % 2 == 0 else 1, 64, 16)
    q = bf16(rng.standard_normal((2, T, Hq, 64))).cuda().transpose(1, 2)
    o, lse = fa.decode_tree(q, *p.args(), **p.kw())
    again, lse2 = fa.decode_tree(q, *p.args(), **p.kw())
    assert torch.equal(o, again) and torch.equal(lse, lse2)
    check_tree4(o, lse, q, p, [T, T], None, 0.125, [0, Hq - 1])
    got, ws = Guarded((2, Hq, T, 64), torch.bfloat16), Guarded((256,), torch.uint8)
    ls = Guarded((2, Hq, T), torch.float32)
    fa.decode_tree(q, *p.args(), out=got.t, lse=ls.t, workspace=ws.t, **p.kw())
    check_tree4(got.t, ls.t, q, p, [T, T], None, 0.125, [0, Hq - 1])
    assert got.intact() and ws.intact() and ls.intact()
    same = q.clone()
    fa.decode_tree(same, *p.args(), out=same, **p.kw())
    check_tree4(same, lse, q, p, [T, T], None, 0.125, [0, Hq - 1])


def test_keys_beyond_32_bit_offsets():
    """Pages whose codes lie beyond 2^31 bytes and 2^32 elements."""
    import torch
    hkv, bs, d = 8, 128, 128
    nb = (1 << 32) // (hkv * bs * d) + 40
    (kc, vc), sc = _pools(nb, hkv, bs, d)
    rng = np.random.default_rng(14)
    x = {n: bf16(rng.standard_normal((2, hkv, 300, d))).cuda() for n in "kv"}
    table = _i32([[nb - 1, 3, nb - 7], [nb - 2, nb - 9, 0]])
    fa.cache_append(x["k"], x["v"], kc, vc, table, _i32([0, 0]), **sc)
    gk, gv = fa.cache_gather(kc, vc, table, _i32([300, 300]), 300, **sc)
    y = {n: serving.quantise_groups(np64(x[n]))[2] for n in "kv"}
    assert np.array_equal(np64(gk), y["k"]) and np.array_equal(np64(gv), y["v"])

    class Seen:
        pass
    p = Seen()
    p.hkv, p.k, p.v = hkv, y["k"], y["v"]
    for G in (1, 5):
        q = bf16(rng.standard_normal((2, hkv * G, 4, d))).cuda()
        o, lse = fa.decode_tree(q, kc, vc, table, _i32([300, 300]), **sc)
        check_tree4(o, lse, q, p, [4, 4], None, 1 / math.sqrt(d), [0, hkv * G - 1])
    fa.device_status()


@pytest.mark.parametrize("T", [1, 4, 8, 20, 64])
def test_calls_behind_an_unread_timeout_end(T):
    """As with the other caches: their waits give up early, they end, and calls after the report are right.  (4 query heads a
    key/value head: 4, 16, 32, 80 and 256 rows.)"""
    import torch
    p = Paged4(np.random.default_rng(T), [3000, 500, T], 2, 128, 16)
    q = bf16(np.random.default_rng(1).standard_normal((3, 8, T, 128))).cuda()
    want, lse = fa.decode_tree(q, *p.args(), **p.kw())
    fa.device_status()
    fa.watchdog_selftest()
    for parts in (0, 1, 7):
        fa.decode_tree(q, *p.args(), max_parts=parts, **p.kw())
    with pytest.raises(fa.FAError) as ei:
        fa.device_status()
    assert ei.value.status == fa.FA_ERR_DEVICE_TIMEOUT
    got, lse2 = fa.decode_tree(q, *p.args(), **p.kw())
    assert torch.equal(got, want) and torch.equal(lse, lse2)
    fa.device_status()


def test_two_calls_at_once():
    """On two streams, each with its workspace: both have the bits that they have alone."""
    import torch
    calls = []
    for T, seed in ((2, 1), (16, 2)):
        p = Paged4(np.random.default_rng(seed), [2000, 900, 130], 2, 64, 32)
        q = bf16(np.random.default_rng(seed).standard_normal((3, 8, T, 64))).cuda()
        calls.append((p, q, fa.decode_tree(q, *p.args(), max_parts=8, **p.kw()), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        got = [[fa.decode_tree(q, *p.args(), max_parts=8, stream=s, **p.kw()) for _ in range(4)] for p, q, _, s in calls]
        torch.cuda.synchronize()
        for (_, _, want, _), outs in zip(calls, got):
            assert all(torch.equal(a, b) for out in outs for a, b in zip(out, want))
    fa.device_status()
