"""Calls of the operators around attention that are refused at the edges of their ranges (no GPU)."""

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


def _tree(L, **kw):
    a = dict(q=FAKE, o=FAKE, B=2, Hq=4, Hkv=2, T=4, mb=16, d=64, st=None, wsb=1 << 30)
    a.update(kw)
    return L.fa_decode_tree(a["q"], FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, None, 0, a["o"], None, a["B"], a["Hq"], a["Hkv"],
                            a["T"], 100, 16, a["mb"], a["d"], fa.FA_BF16, 0.1, a["st"], 4, FAKE, a["wsb"], None)


@pytest.mark.parametrize("st", [(1024, 64, 256, 1024, 256, 64), (2048, 256, 64, 1024, 256, 64), (1024, 256, 64, 1024, 64, 256)])
def test_decode_tree_in_place_needs_the_queries_strides(L, st):
    """Rows would be written over queries that other blocks still read."""
    assert _tree(L, st=_st(*st)) == INV
    assert b"in place" in L.fa_get_last_error()
    # Elsewhere these strides are fine, and so are ones that take no step: the next check refuses the workspace.
    assert _tree(L, o=FAKE + (1 << 16), st=_st(*st), wsb=0) == INV
    assert b"workspace" in L.fa_get_last_error()
    assert _tree(L, T=1, st=_st(1024, 256, 64, 1024, 256, 128), wsb=0) == INV
    assert b"workspace" in L.fa_get_last_error()


@pytest.mark.parametrize("w,status", [(2.0 ** 64, UNS), (-1e300, UNS), (float("inf"), INV)])
def test_rope_refuses_frequencies_without_a_fraction(L, w, status):
    inv = np.array([1.0, w])
    assert L.fa_rope(FAKE, None, FAKE, None, 1, 1, 0, 1, 4, 4, fa.FA_FP32, None, None, 0, 0, inv.ctypes.data, 1.0, 0, 0,
                     None) == status
    assert b"inv_freq[1]" in L.fa_get_last_error()


def test_strides_of_dimensions_of_one_are_not_looked_at(L):
    assert _tree(L, T=1, o=FAKE + (1 << 16), st=_st(1024, 256, 3, 1024, 256, -1), wsb=0) == INV
    assert b"workspace" in L.fa_get_last_error()
    assert _tree(L, T=2, o=FAKE + (1 << 16), st=_st(1024, 256, 3, 1024, 256, 64), wsb=0) == INV
    assert b"stride[2]" in L.fa_get_last_error()


@pytest.mark.parametrize("N", [(1 << 31) - 1, (1 << 30) + 1])
@pytest.mark.parametrize("call", ["append", "gather"])
def test_cache_refuses_more_tokens_than_a_table_can_hold(L, call, N):
    """Rounding these up to whole groups of tokens would pass the largest int."""
    st = _st(0, 0, 0, 0, 0, 0) if call == "append" else None
    f = L.fa_cache_append if call == "append" else L.fa_cache_gather
    args = [FAKE] * 8 if call == "gather" else [FAKE] * 9
    assert f(*args, 1, 1, N, 100, 16, 16, 64, fa.FA_BF16, st, None) == UNS
    assert b"N must be" in L.fa_get_last_error()


def test_more_work_than_a_grid_holds_is_refused(L):
    zero = _st(0, 0, 0, 0, 0, 0)
    assert L.fa_cache_append(*[FAKE] * 9, 65535, 65535, 1 << 20, 100, 16, 16, 64, fa.FA_BF16, zero, None) == UNS
    assert b"too large" in L.fa_get_last_error()
    w = np.ones(128)
    assert L.fa_rope(FAKE, None, FAKE + (1 << 20), None, 65535, 1, 0, 1 << 24, 256, 256, fa.FA_FP32, None, None, 0, 0,
                     w.ctypes.data, 1.0, 0, 0, None) == UNS
    assert b"too large" in L.fa_get_last_error()
    assert _tree(L, B=65535, Hq=1024, Hkv=1024, T=256) == UNS
    assert b"too large" in L.fa_get_last_error()
