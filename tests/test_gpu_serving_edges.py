"""The operators around attention at the edges of their ranges."""

import math
from fractions import Fraction

import numpy as np
import pytest

from io_aware_exact_11_gb300 import fa
from tests.serving_helpers import Paged, bf16, check_tree, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.lib()
    fa.device_status()
    yield
    fa.device_status()


def _i32(a):
    import torch
    return torch.tensor(a, dtype=torch.int32, device="cuda")


# Drafted tokens with 4 query heads a key/value head: 4, 12, 32, 80 and 256 rows, on every kernel's side.
TOKENS = [1, 3, 8, 20, 64]


@pytest.mark.parametrize("cache,T", [("bf16", 2), ("bf16", 20), ("bf16", 64), ("e4m3", 2), ("e4m3", 20), ("e4m3", 64)])
def test_calls_behind_an_unread_timeout_end(cache, T):
    """A timeout that nobody has read makes the waits of later calls give up early, each for itself.  Such calls end, and
    the ones after the report are right.  (4 query heads a key/value head: 8, 80 and 256 rows.)"""
    import torch
    p = Paged(np.random.default_rng(T), [3000, 500, T], 2, 128, 16, cache)
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


def test_output_over_the_queries_needs_their_strides():
    import torch
    p = Paged(np.random.default_rng(7), [40, 50], 2, 64, 16, "bf16")
    q = torch.zeros((2, 4, 4, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fa.FAError, match="in place"):
        fa.decode_tree(q, *p.args(), out=q.transpose(1, 2))
    with pytest.raises(fa.FAError, match="in place"):
        fa.decode_tree(q.transpose(1, 2), *p.args(), out=q)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", TOKENS)
def test_an_infinite_value_in_the_context_is_infinite_in_every_row(T, d):
    """Every weight is positive, so a column with one infinity is that infinity, and one with both is NaN."""
    def edit(name, b, x):
        if name == "v":
            x[:, 70, 9], x[:, 200, 11], x[:, x.shape[1] - T - 1, 13] = np.inf, -np.inf, np.inf
            x[:, 70, 20], x[:, 71, 20] = np.inf, -np.inf
    p = Paged(np.random.default_rng(T), [300, 230 + T], 2, d, 32, "bf16", edit=edit)
    q = bf16(np.random.default_rng(1).standard_normal((2, 8, T, d))).cuda()
    for parts in (1, 3):
        o, lse = fa.decode_tree(q, *p.args(), max_parts=parts)
        with np.errstate(invalid="ignore"):  # inf - inf, as wanted
            check_tree(o, lse, q, p, [T, T], None, d ** -0.5)
        o = np64(o)
        assert np.isposinf(o[..., [9, 13]]).all() and np.isneginf(o[..., 11]).all() and np.isnan(o[..., 20]).all()
        assert np.isfinite(np.delete(o, [9, 11, 13, 20], 3)).all()


@pytest.mark.parametrize("T", TOKENS)
def test_an_infinite_value_under_a_weight_of_one(T):
    import torch
    def edit(name, b, x):
        if name == "v":
            x[:, 0, 9] = -np.inf
    p = Paged(np.random.default_rng(T), [1 + T], 2, 128, 16, "bf16", edit=edit)
    q = bf16(np.random.default_rng(2).standard_normal((1, 8, T, 128))).cuda()
    o, _ = fa.decode_tree(q, *p.args(), tree_mask=torch.zeros((T, T), dtype=torch.bool, device="cuda"))
    want = np.repeat(p.v[0][:, :1], 4, 0)  # one key: its weight is 1
    assert np.array_equal(np64(o)[0], np.repeat(want, T, 1))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [2, 6, 12, 40])
@pytest.mark.parametrize("power", [1, 4, 6, 8, 9, 15, 16, 17])
def test_small_weights_beside_one_that_counts_for_nothing(T, power, d):
    """E4M3: one key has nearly all of a row's weight and a value of zero, so the row's result is made of weights 2^-16 to
    2^-22 of the largest, and a few value rows without weight are larger by 2^power.  Column 5 holds E4M3's smallest."""
    for k0, parts in ((8.0, 3), (10.0, 1), (11.0, 1)):
        def edit(name, b, x):
            if name == "k":
                np.clip(x, -0.9, 0.9, out=x)
                x[:, :, 0] = 0.0
                x[:, 7, 0] = k0
                x[:, 30::97, 0] = -448.0
            else:
                x[:] = 1.0 + 0.75 * np.abs(np.sin(np.arange(x.size))).reshape(x.shape)
                x[..., 5] = 3 * 2.0 ** -17
                x[:, 30::97] *= 2.0 ** power
                x[:, 7] = 0.0
        p = Paged(np.random.default_rng(T), [700, 400], 2, d, 32, "e4m3", edit=edit)
        q = np.zeros((2, 8, T, d))
        q[..., 0] = 11.3125
        q = bf16(q).cuda()
        o, lse = fa.decode_tree(q, *p.args(), max_parts=parts, scale=0.125, **p.kw())
        check_tree(o, lse, q, p, [T, T], None, 0.125, heads=[7])


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("scale", [2.0 ** -30, 1e-38])
def test_zero_queries_and_the_smallest_scales(cache, T, scale):
    p = Paged(np.random.default_rng(T), [300, 128 + T, T], 2, 128, 16, cache)
    q = np.random.default_rng(3).standard_normal((3, 8, T, 128))
    q[:, :, 0] = 0.0
    q[:, 3] = 0.0
    q[:, 5] *= 2.0 ** -100
    q = bf16(q).cuda()
    o, lse = fa.decode_tree(q, *p.args(), scale=scale, **p.kw())
    check_tree(o, lse, q, p, [T] * 3, None, scale)


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("power", [100, 120, 122])
def test_the_smallest_values_of_a_long_sequence(T, power):
    """E4M3 rows near the smallest power of two, under a row sum in the tens of thousands."""
    def edit(name, b, x):
        if name == "v":
            x[:] = (1.0 + 0.75 * np.abs(np.sin(np.arange(x.size))).reshape(x.shape)) * 2.0 ** -power
        else:
            x *= 2.0 ** -4
    p = Paged(np.random.default_rng(T), [40000], 1, 64, 128, "e4m3", edit=edit)
    q = bf16(np.random.default_rng(4).standard_normal((1, 2, T, 64))).cuda()
    for parts in (1, 0):
        o, lse = fa.decode_tree(q, *p.args(), max_parts=parts, **p.kw())
        check_tree(o, lse, q, p, [T], None, 0.125, heads=[1])


def test_a_bad_page_is_reported_behind_a_timeout():
    import torch
    kc, vc = (torch.zeros((4, 1, 16, 64), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    x = torch.ones((1, 1, 3, 64), dtype=torch.bfloat16, device="cuda")
    fa.watchdog_selftest()
    fa.cache_append(x, x, kc, vc, _i32([[9]]), _i32([0]))
    with pytest.raises(fa.FAError) as ei:
        fa.device_status()
    assert ei.value.status == fa.FA_ERR_DEVICE_TIMEOUT
    with pytest.raises(fa.FAError, match="paged cache") as ei:
        fa.device_status()
    assert ei.value.status == fa.FA_ERR_INVALID_ARG
    fa.device_status()
    assert not kc.any()


@pytest.mark.parametrize("bad", ["page", "length"])
@pytest.mark.parametrize("Hq", [2, 8])
def test_an_unread_report_of_the_paged_decode_leaves_later_calls_alone(Hq, bad):
    """A bad page or length is one sequence's; the word that it is reported in is not the one that pipeline waits look at:
    a timeout behind it is reported first, and then the page or length."""
    import torch
    p = Paged(np.random.default_rng(Hq), [3000, 700], 2, 128, 16, "bf16")
    q = bf16(np.random.default_rng(1).standard_normal((2, Hq, 1, 128))).cuda()
    want, _ = fa.decode_paged(q, *p.args())
    tree, _ = fa.decode_tree(q, *p.args())
    fa.device_status()
    table, lens = p.table.clone(), p.seq_lens.clone()
    if bad == "page":
        table[1, 3] = -5
    else:
        lens[1] = 0
    got, _ = fa.decode_paged(q, p.k_cache, p.v_cache, table, lens)
    after, _ = fa.decode_paged(q, *p.args())
    tree2, _ = fa.decode_tree(q, *p.args())
    assert torch.equal(got[0], want[0]) and torch.equal(after, want) and torch.equal(tree2, tree)
    fa.watchdog_selftest()
    with pytest.raises(fa.FAError) as ei:
        fa.device_status()
    assert ei.value.status == fa.FA_ERR_DEVICE_TIMEOUT
    with pytest.raises(fa.FAError, match="paged decode") as ei:
        fa.device_status()
    assert ei.value.status == fa.FA_ERR_INVALID_ARG
    fa.device_status()


PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")


@pytest.mark.parametrize("inverse", [False, True])
def test_rope_is_exact_at_any_position_and_frequency(inverse):
    """Against rational arithmetic.  fp32: the angle's fraction of a turn kept to 2^-32 and rounded to 24 bits (π·2^-25
    radians, 2π·2^-32), sine and cosine within 2 ulp (2·2^-24), a product (2^-24): 4.6·2^-24 of |x₁| + |x₂|, and the
    result's rounding."""
    import torch
    w = [1.0, 0.75, 3.3, 100.3, 12345.678, -2.5, 1e-5, 1e-19, 1e15, 1.7e19, 0.0, 5e-324, 2.0 ** -64, 6.283185307179586]
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 3, 1999999973, 16777217, 1, 0, -7, 1048577, 2 ** 30]
    x = torch.randn((1, 3, len(pos), 2 * len(w)), generator=torch.Generator().manual_seed(5)).cuda()
    f = fa.rope_backward if inverse else fa.rope
    y, _ = f(x, None, np.array(w), positions=_i32(pos), interleaved=True)
    x, y = np64(x)[0], np64(y)[0]
    for n, p in enumerate(pos):
        for i, wi in enumerate(w):
            part = Fraction(p) * Fraction(wi) / (2 * PI)
            angle = 2 * math.pi * float(part - math.floor(part)) * (-1 if inverse else 1)
            c, s = math.cos(angle), math.sin(angle)
            a, b = x[:, n, 2 * i], x[:, n, 2 * i + 1]
            for got, ref in ((y[:, n, 2 * i], a * c - b * s), (y[:, n, 2 * i + 1], b * c + a * s)):
                assert np.all(np.abs(got - ref) <= 2.0 ** -24 * (np.abs(ref) + 4.6 * (np.abs(a) + np.abs(b)))), (p, wi)


def test_strides_of_dimensions_of_one_do_not_matter():
    import torch
    d, H = 128, 4
    rng = np.random.default_rng(6)
    p = Paged(rng, [40, 50], 2, d, 16, "bf16")
    def odd(x):  # [B,H,1,d] with strides of the token dimension that no 16-byte access could take
        B, h, _, _ = x.shape
        y = torch.empty((B * (h + 1) * d,), dtype=x.dtype, device="cuda").as_strided(x.shape, ((h + 1) * d, d, 3, 1))
        return y.copy_(x)
    q, k, v = (bf16(rng.standard_normal((2, h, 1, d))).cuda() for h in (H, 2, 2))
    o, lse = fa.decode_tree(q, *p.args())
    o2, lse2 = fa.decode_tree(odd(q), *p.args(), out=odd(torch.zeros_like(q)))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    caches = [[t.clone() for t in (p.k_cache, p.v_cache)] for _ in range(2)]
    fa.cache_append(k, v, *caches[0], p.table, p.seq_lens - 1)
    fa.cache_append(odd(k), odd(v), *caches[1], p.table, p.seq_lens - 1)
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(*caches))
    gk, gv = fa.cache_gather(*p.args(), 1)
    ok, ov = fa.cache_gather(*p.args(), 1, out_k=odd(torch.zeros_like(k)), out_v=odd(torch.zeros_like(k)))
    assert torch.equal(gk, ok) and torch.equal(gv, ov)
