"""Pins of the oracle's four-bit rows, several axes and page pool, and the argument checks of the calls on them (no GPU)."""

import ctypes
import os

import numpy as np
import pytest

from io_aware_exact_11_gb300 import fa
from oracle import serving

FAKE = 1 << 20  # never dereferenced: validation fails first
INV, UNS = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(fa.LIB_PATH):
        from io_aware_exact_11_gb300 import build
        build.build()
    return fa.lib()


def test_e2m1_codes():
    y = np.array([0, 0.24, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 6, 9, -0.75, -5.0, -0.0])
    want = [0, 0, 0, 1, 2, 2, 4, 4, 6, 6, 7, 7, 7, 10, 14, 8]  # halves go to the even code
    assert serving.round_e2m1(y).tolist() == want


def test_groups_take_the_smallest_power_that_holds_them():
    x = np.zeros((5, 64))
    x[0, 0], x[0, 40] = 6.0, 6.0001
    x[1, 3] = 2.0 ** -133
    x[2, :] = np.where(np.arange(64) % 2, -1.0, 0.5)
    x[3, 5] = np.inf
    x[4, 1], x[4, 63] = 3.3e38, -3 * 2.0 ** 126
    codes, scales, values = serving.quantise_groups(x)
    assert scales.tolist() == [[127, 128], [1, 1], [125, 125], [255, 1], [252, 252]]
    assert values[0, 0] == 6 and values[0, 40] == 6 and codes[0, 40] == 5  # 6.0001 / 2 = 3.00005
    assert np.array_equal(values[2], x[2]) and np.isnan(values[3, :32]).all() and (values[3, 32:] == 0).all()
    assert values[4, 1] == 6 * 2.0 ** 125 and values[4, 63] == -6 * 2.0 ** 125  # saturated, and held exactly


def test_one_axis_is_the_plain_rotation():
    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((2, 3, 5, 16)), 10000.0 ** (-np.arange(6) / 6)
    pos = rng.integers(-9, 999, (2, 2, 5))
    for inter in (False, True):
        for inverse in (False, True):
            got = serving.rope_axes(x, pos, [1] * 6, w, 1.25, inter, inverse)
            assert np.allclose(got, serving.rope(x, pos[1], w, 1.25, inter, inverse), rtol=0, atol=1e-13)


def test_pool_shares_copies_and_frees():
    p = serving.Pool([[0, 1, -1], [-1] * 3, [-1] * 3], [20, 0, 0], [1, 1, 0, 0, 0], 16)
    p.fork([0, 0], [1, 2])
    assert p.table == [[0, 1, -1]] * 3 and p.holders == [3, 3, 0, 0, 0] and p.lens == [20, 20, 20]
    # all write into page 1: the last to hold it keeps it; 13 tokens need a page more, for which none is left at the end
    assert p.reserve([1, 13, 1]) == ([1, 1, 1], [1, 1, -1], [2, 3, -1])
    assert p.table == [[0, 2, -1], [0, 3, 4], [0, 1, -1]] and p.holders == [3, 1, 1, 1, 1]
    assert p.reserve([0, 13, 20]) == ([1, 1, 0], [-1] * 3, [-1] * 3)
    p.free([1, 2, 1], [17, 0, 3])
    assert p.lens == [20, 17, 0] and p.table[1] == [0, 3, -1] and p.holders == [2, 0, 1, 1, 0]


# ------------------------------------------------------------------------------------------------ refusals


def _axes(L, **kw):
    a = dict(q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, B=1, Hq=4, Hk=2, N=8, d=128, rot=128, dt=fa.FA_BF16, st=None, pos=FAKE,
             n=3, psa=8, psb=0, axes=np.arange(64, dtype=np.int32) % 3, inv=np.ones(64), mag=1.0, lay=0, back=0)
    a.update(kw)
    ptr = [x.ctypes.data if x is not None else None for x in (a["axes"], a["inv"])]
    return L.fa_rope_axes(a["q"], a["k"], a["qo"], a["ko"], a["B"], a["Hq"], a["Hk"], a["N"], a["d"], a["rot"], a["dt"],
                          a["st"], a["pos"], a["n"], a["psa"], a["psb"], *ptr, a["mag"], a["lay"], a["back"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INV), (dict(qo=None), INV), (dict(k=None), INV), (dict(pos=None), INV), (dict(axes=None), INV),
    (dict(inv=None), INV), (dict(n=0), INV), (dict(n=-1), INV), (dict(n=5), UNS), (dict(n=2), INV), (dict(psa=-1), INV),
    (dict(psb=-1), INV), (dict(pos=FAKE + 2), INV), (dict(axes=np.full(64, -1, dtype=np.int32)), INV), (dict(rot=130), INV),
    (dict(d=258), UNS), (dict(dt=fa.FA_E2M1), INV), (dict(B=0), INV), (dict(lay=2), INV), (dict(back=2), INV),
    (dict(mag=float("nan")), INV), (dict(inv=np.full(64, np.inf)), INV)])
def test_rope_axes_refuses(L, kw, status):
    assert _axes(L, **kw) == status
    assert b"fa_rope_axes" in L.fa_get_last_error()


FOUR_BAD = [(dict(ks=None), INV), (dict(vs=None), INV), (dict(ks=FAKE + 8), INV), (dict(kc=FAKE + 8), INV),
            (dict(kc=None), INV), (dict(d=96), UNS), (dict(d=32), UNS), (dict(bs=8), UNS), (dict(nb=0), INV),
            (dict(dt=4), INV), (dict(dt=fa.FA_FP32), UNS), (dict(Hkv=0), INV), (dict(nb=1 << 30), UNS)]
BASE = dict(kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, table=FAKE, B=2, Hkv=4, nb=100, bs=16, mb=16, d=128, dt=fa.FA_E2M1)


@pytest.mark.parametrize("kw,status", FOUR_BAD)
def test_four_bit_caches_are_checked(L, kw, status):
    a = dict(BASE, **kw)
    tail = (a["B"], a["Hkv"], 8, a["nb"], a["bs"], a["mb"], a["d"], a["dt"], None, None)
    assert L.fa_cache_append(FAKE, FAKE, a["kc"], a["vc"], a["ks"], a["vs"], a["table"], FAKE, None, *tail) == status
    assert L.fa_cache_gather(a["kc"], a["vc"], a["ks"], a["vs"], a["table"], FAKE, FAKE, FAKE, *tail) == status
    assert L.fa_decode_tree(FAKE, a["kc"], a["vc"], a["ks"], a["vs"], a["table"], FAKE, None, None, 0, FAKE, None, a["B"],
                            28, a["Hkv"], 8, a["nb"], a["bs"], a["mb"], a["d"], a["dt"], 0.1, None, 4, FAKE, 1 << 30,
                            None) == status


@pytest.mark.parametrize("kw,status", FOUR_BAD + [
    (dict(first=None), INV), (dict(keep=None), INV), (dict(first=FAKE + 1), INV), (dict(keep=FAKE + 2), INV),
    (dict(lens=FAKE + 2), INV), (dict(N=0), INV), (dict(sb=-1), INV), (dict(table=None), INV), (dict(B=0), INV),
    (dict(B=60000, Hkv=60000, nb=1), UNS), (dict(nb=1 << 25, bs=128, Hkv=1, mb=1), UNS)])
def test_cache_compact_refuses(L, kw, status):
    a = dict(BASE, first=FAKE, keep=FAKE, sb=8, lens=None, N=8)
    a.update(kw)
    assert L.fa_cache_compact(a["kc"], a["vc"], a["ks"], a["vs"], a["table"], a["first"], a["keep"], a["sb"], a["lens"],
                              a["B"], a["Hkv"], a["N"], a["nb"], a["bs"], a["mb"], a["d"], a["dt"], None) == status
    assert b"fa_cache_compact" in L.fa_get_last_error()


@pytest.mark.parametrize("kw,status", FOUR_BAD + [
    (dict(src=None), INV), (dict(dst=None), INV), (dict(src=FAKE + 1), INV), (dict(dst=FAKE + 2), INV), (dict(n=0), INV),
    (dict(n=65536), UNS)])
def test_cache_copy_pages_refuses(L, kw, status):
    a = dict(BASE, src=FAKE, dst=FAKE, n=8)
    a.update(kw)
    assert L.fa_cache_copy_pages(a["kc"], a["vc"], a["ks"], a["vs"], a["src"], a["dst"], a["n"], a["Hkv"], a["nb"], a["bs"],
                                 a["d"], a["dt"], None) == status
    assert b"fa_cache_copy_pages" in L.fa_get_last_error()


PAGES_BAD = [(dict(table=None), INV), (dict(lens=None), INV), (dict(held=None), INV), (dict(one=None), INV), (dict(B=0), INV),
             (dict(nb=0), INV), (dict(bs=0), INV), (dict(mb=0), INV), (dict(bs=24), UNS), (dict(mb=1 << 27), UNS),
             (dict(table=FAKE + 2), INV), (dict(lens=FAKE + 2), INV), (dict(held=FAKE + 1), INV), (dict(one=FAKE + 2), INV)]
PAGES = dict(table=FAKE, lens=FAKE, held=FAKE, one=FAKE, two=FAKE, n=2, B=4, nb=100, bs=16, mb=8)


@pytest.mark.parametrize("kw,status", PAGES_BAD + [(dict(two=None), INV), (dict(two=FAKE + 1), INV), (dict(n=0), INV),
                                                   (dict(n=70000), UNS), (dict(B=70000), UNS)])
def test_pages_fork_refuses(L, kw, status):
    a = dict(PAGES, **kw)
    assert L.fa_pages_fork(a["table"], a["lens"], a["held"], a["one"], a["two"], a["n"], a["B"], a["nb"], a["bs"], a["mb"],
                           None) == status
    assert b"fa_pages_fork" in L.fa_get_last_error()


@pytest.mark.parametrize("kw,status", PAGES_BAD + [(dict(two=FAKE + 1), INV), (dict(n=0), INV), (dict(n=70000), UNS)])
def test_pages_free_refuses(L, kw, status):
    a = dict(PAGES, **kw)
    assert L.fa_pages_free(a["table"], a["lens"], a["held"], a["one"], a["two"], a["n"], a["B"], a["nb"], a["bs"], a["mb"],
                           None) == status
    assert b"fa_pages_free" in L.fa_get_last_error()


@pytest.mark.parametrize("kw,status", PAGES_BAD + [
    (dict(g=None), INV), (dict(src=None), INV), (dict(dst=None), INV), (dict(ws=None), INV), (dict(g=FAKE + 1), INV),
    (dict(ws=FAKE + 2), INV), (dict(wsb=255), INV), (dict(B=4097), UNS), (dict(B=4000, mb=1 << 20), UNS)])
def test_pages_reserve_refuses(L, kw, status):
    a = dict(PAGES, g=FAKE, src=FAKE, dst=FAKE, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    assert L.fa_pages_reserve(a["table"], a["lens"], a["held"], a["one"], a["g"], a["src"], a["dst"], a["B"], a["nb"],
                              a["bs"], a["mb"], a["ws"], a["wsb"], None) == status
    assert b"fa_pages_reserve" in L.fa_get_last_error()


def test_pages_reserve_workspace(L):
    size = L.fa_pages_reserve_workspace_size
    # a word for every 1024 pages, three for every sequence, one more
    assert size(4, 100) == 256 and size(20, 3 * 1024) == 256 and size(20, 3 * 1024 + 1) == 512
    assert size(4096, (1 << 31) - 1) == -(-((1 << 21) + 3 * 4096 + 1) * 4 // 256) * 256
    assert size(0, 5) == 0 and size(5, 0) == 0


def test_binding_refuses_host_tensors_and_shapes():
    torch = pytest.importorskip("torch")
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros((2, 4), dtype=torch.int32)
    c, s = torch.zeros((4, 2, 16, 32), dtype=torch.uint8), torch.zeros((4, 2, 16, 2), dtype=torch.uint8)
    q = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16)
    for call in (lambda: fa.rope_axes(q, None, np.ones(32), np.zeros(32), torch.zeros((1, 3), dtype=torch.int32)),
                 lambda: fa.cache_compact(c, c, t, i, t, k_scale=s, v_scale=s),
                 lambda: fa.cache_copy_pages(c, c, i, i, k_scale=s, v_scale=s), lambda: fa.pages_fork(t, i, i, i, i, 16),
                 lambda: fa.pages_free(t, i, i, i, 16), lambda: fa.pages_reserve(t, i, i, i, 16)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="d/32"):
        fa._cache_args(c, c, s, s[..., :1], t)
    assert fa._cache_args(c, c, s, s, t) == (4, 2, 16, 64, fa.FA_E2M1)
    assert fa._cache_args(c, c, s[..., 0].contiguous(), s[..., 0].contiguous(), t) == (4, 2, 16, 32, fa.FA_E4M3)
    assert ctypes.sizeof(ctypes.c_int) == 4
