"""Argument checks of fa_rope, fa_cache_append, fa_cache_gather and fa_decode_tree (no GPU): every bad call is
refused before anything is queued."""

import ctypes
import os

import numpy as np
import pytest

from io_aware_exact_11_gb300 import fa

FAKE = 1 << 20  # never dereferenced: validation fails first
INV, UNS = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(fa.LIB_PATH):
        from io_aware_exact_11_gb300 import build
        build.build()
    return fa.lib()


def _st(*x):
    return (ctypes.c_int64 * len(x))(*x)


def _rope(L, **kw):
    a = dict(q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, B=1, Hq=4, Hk=2, N=8, d=128, rot=128, dt=fa.FA_BF16, st=None,
             pos=None, psb=0, p0=0, inv=np.ones(128), mag=1.0, lay=fa.FA_ROPE_HALF, back=0)
    a.update(kw)
    inv = a["inv"].ctypes.data if a["inv"] is not None else None
    return L.fa_rope(a["q"], a["k"], a["qo"], a["ko"], a["B"], a["Hq"], a["Hk"], a["N"], a["d"], a["rot"], a["dt"],
                     a["st"], a["pos"], a["psb"], a["p0"], inv, a["mag"], a["lay"], a["back"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INV), (dict(qo=None), INV), (dict(inv=None), INV), (dict(k=None), INV), (dict(ko=None), INV),
    (dict(B=0), INV), (dict(Hq=0), INV), (dict(Hk=-1), INV), (dict(N=0), INV), (dict(d=0), INV), (dict(rot=0), INV),
    (dict(rot=7), INV), (dict(rot=130), INV), (dict(d=127, rot=64), UNS), (dict(d=258, rot=64), UNS),
    (dict(dt=fa.FA_E4M3), INV), (dict(dt=9), INV), (dict(lay=2), INV), (dict(back=2), INV), (dict(mag=0.0), INV),
    (dict(mag=float("nan")), INV), (dict(mag=float("inf")), INV), (dict(B=70000), UNS), (dict(Hq=40000), UNS),
    (dict(q=FAKE + 1), INV), (dict(dt=fa.FA_FP32, k=FAKE + 2), INV), (dict(pos=FAKE + 2), INV),
    (dict(pos=FAKE, psb=-1), INV), (dict(inv=np.array([1.0, np.nan] * 64)), INV),
    (dict(st=_st(*([8192, 1024, 128] * 3 + [8192, 1024, -1]))), INV),
    (dict(qo=FAKE + 64, st=_st(4096, 1024, 128, 4096, 1024, 128, 4096, 512, 128, 4096, 1024, 128)), INV),  # overlaps itself
    (dict(qo=FAKE + 64, ko=FAKE + 64, st=_st(0, 1024, 128, 0, 1024, 128, 0, 1024, 64, 0, 1024, 128)), INV),
    (dict(st=_st(4096, 1024, 128, 4096, 1024, 128, 4096, 128, 512, 4096, 1024, 128)), INV),  # in place, other strides
])
def test_rope_refuses(L, kw, status):
    assert _rope(L, **kw) == status
    assert b"fa_rope" in L.fa_get_last_error()


CACHE_BAD = [
    (dict(kc=None), INV), (dict(vc=None), INV), (dict(table=None), INV), (dict(B=0), INV), (dict(Hkv=0), INV),
    (dict(nb=0), INV), (dict(bs=0), INV), (dict(mb=0), INV), (dict(d=0), INV), (dict(dt=7), INV),
    (dict(dt=fa.FA_FP32), UNS), (dict(d=96), UNS), (dict(d=256), UNS), (dict(bs=8), UNS), (dict(bs=48), UNS),
    (dict(bs=256), UNS), (dict(B=70000), UNS), (dict(mb=1 << 27), UNS), (dict(nb=1 << 30), UNS),
    (dict(dt=fa.FA_E4M3, ks=None), INV), (dict(dt=fa.FA_E4M3, vs=None), INV), (dict(dt=fa.FA_E4M3, ks=FAKE + 8), INV),
    (dict(kc=FAKE + 8), INV), (dict(table=FAKE + 2), INV),
]


def _append(L, **kw):
    a = dict(k=FAKE, v=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, table=FAKE, start=FAKE, lens=None, B=2, Hkv=4, N=8,
             nb=100, bs=16, mb=16, d=128, dt=fa.FA_BF16, st=None)
    a.update(kw)
    return L.fa_cache_append(a["k"], a["v"], a["kc"], a["vc"], a["ks"], a["vs"], a["table"], a["start"], a["lens"],
                             a["B"], a["Hkv"], a["N"], a["nb"], a["bs"], a["mb"], a["d"], a["dt"], a["st"], None)


@pytest.mark.parametrize("kw,status", CACHE_BAD + [
    (dict(k=None), INV), (dict(v=None), INV), (dict(start=None), INV), (dict(N=0), INV), (dict(k=FAKE + 8), INV),
    (dict(start=FAKE + 1), INV), (dict(lens=FAKE + 2), INV), (dict(st=_st(4096, 1024, 128, 4096, 1024, 4)), INV),
    (dict(st=_st(4096, 1024, 128, -8, 1024, 128)), INV)])
def test_cache_append_refuses(L, kw, status):
    assert _append(L, **kw) == status
    assert b"fa_cache_append" in L.fa_get_last_error()


@pytest.mark.parametrize("kw,status", CACHE_BAD + [
    (dict(k=None), INV), (dict(v=None), INV), (dict(lens=None), INV), (dict(N=0), INV), (dict(v=FAKE + 8), INV),
    (dict(st=_st(4096, 1024, 128, 4096, 1024, 4)), INV), (dict(st=_st(4096, 1024, 128, 0, 1024, 128)), INV)])
def test_cache_gather_refuses(L, kw, status):
    a = dict(k=FAKE, v=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, table=FAKE, lens=FAKE, B=2, Hkv=4, N=8, nb=100,
             bs=16, mb=16, d=128, dt=fa.FA_BF16, st=None)
    a.update(kw)
    assert L.fa_cache_gather(a["kc"], a["vc"], a["ks"], a["vs"], a["table"], a["lens"], a["k"], a["v"], a["B"],
                             a["Hkv"], a["N"], a["nb"], a["bs"], a["mb"], a["d"], a["dt"], a["st"], None) == status
    assert b"fa_cache_gather" in L.fa_get_last_error()


@pytest.mark.parametrize("kw,status", CACHE_BAD + [
    (dict(q=None), INV), (dict(o=None), INV), (dict(lens=None), INV), (dict(ws=None), INV), (dict(Hq=0), INV),
    (dict(T=0), INV), (dict(ns=-1), INV), (dict(Hq=30), INV), (dict(Hq=516), UNS), (dict(T=257), UNS),
    (dict(ns=4097), UNS), (dict(scale=0.0), INV), (dict(scale=float("nan")), INV), (dict(q=FAKE + 8), INV),
    (dict(o=FAKE + 8), INV), (dict(ws=FAKE + 8), INV), (dict(lse=FAKE + 2), INV), (dict(dl=FAKE + 2), INV),
    (dict(mask=FAKE, msb=3), INV), (dict(wsb=63), INV), (dict(st=_st(4096, 1024, 128, 4096, 1024, 4)), INV),
    (dict(st=_st(0, 1024, 128, 0, 1024, 128)), INV)])
def test_decode_tree_refuses(L, kw, status):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, table=FAKE, lens=FAKE, dl=None, mask=None, msb=0, o=FAKE,
             lse=None, B=2, Hq=28, Hkv=4, T=8, nb=100, bs=16, mb=64, d=128, dt=fa.FA_BF16, scale=0.1, st=None, ns=4,
             ws=FAKE, wsb=1 << 30)
    a.update(kw)
    assert L.fa_decode_tree(a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["table"], a["lens"], a["dl"], a["mask"],
                            a["msb"], a["o"], a["lse"], a["B"], a["Hq"], a["Hkv"], a["T"], a["nb"], a["bs"], a["mb"],
                            a["d"], a["dt"], a["scale"], a["st"], a["ns"], a["ws"], a["wsb"], None) == status
    assert b"fa_decode_tree" in L.fa_get_last_error()


def test_decode_tree_workspace(L):
    size = L.fa_decode_tree_workspace_size
    # one part: a pair of words per (sequence, key/value head) and no pieces
    assert size(2, 28, 4, 8, 128, 1) == 256
    # three parts of eight pairs: two slots per part beat 8 + 2; of 7·8 rows (o in
    # groups of 32 rows), 128 values and (m, ℓ)
    assert size(2, 28, 4, 8, 128, 3) == 256 + 6 * 64 * 128 * 4 + -(-6 * 56 * 8 // 256) * 256
    # three parts of one pair: slots 0, 1, 2
    assert size(1, 4, 1, 1, 64, 3) == 256 + 3 * 4 * 64 * 4 + 256
    assert size(2, 28, 4, 8, 128, 0) == size(2, 28, 4, 8, 128, 152)         # no device here: 152 SMs
    assert size(1, 8, 1, 64, 128, 0) == size(1, 8, 1, 64, 128, 152 // 2)    # 512 rows: two CTAs of 256 per part
    for bad in ((0, 28, 4, 8, 128, 0), (2, 28, 5, 8, 128, 0), (2, 28, 4, 0, 128, 0), (2, 28, 4, 8, 128, -1)):
        assert size(*bad) == 0


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    q = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fa.rope(q, None, np.ones(32))
    c, t, n = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16), torch.zeros((1, 4), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.cache_append(q, q, c, c, t, n)
    with pytest.raises(ValueError, match="CUDA"):
        fa.cache_gather(c, c, t, n, 3)
    with pytest.raises(ValueError, match="CUDA"):
        fa.decode_tree(q, c, c, t, n)
