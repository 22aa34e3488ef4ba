"""Pins of the float64 oracle for rotary positions, E4M3 rows and drafted tokens (no GPU)."""

import math

import numpy as np
import pytest

import oracle
from io_aware_exact_11_gb300 import fa, inputs
from oracle import serving


def test_e4m3_rounding_agrees_with_the_seeded_input_rounding():
    x = np.random.default_rng(0).standard_normal(20000) * np.exp2(np.random.default_rng(1).integers(-14, 9, 20000))
    x = x.astype(np.float32)
    assert np.array_equal(serving.round_e4m3(np.clip(x, -448, 448)), inputs.e4m3_bits_to_f32(inputs.f32_to_e4m3_bits(x)))


def test_e4m3_ties_go_to_the_even_code():
    table = serving.e4m3_values()
    mid = (table[:-1] + table[1:]) / 2
    even = np.where(np.arange(126) % 2 == 0, table[:-1], table[1:])
    assert np.array_equal(serving.round_e4m3(mid), even)


@pytest.mark.parametrize("top,k", [(448.0, 0), (448.0001, 1), (224.0, -1), (224.1, 0), (1.75, -8), (1.76, -7),
                                   (2.0 ** -133, -126), (0.0, -126), (3.3e38, 120)])
def test_row_scale_is_the_smallest_power_of_two_that_holds_the_row(top, k):
    assert serving.quantise_rows(np.array([0.0, -top, top / 3]))[1] == k


def test_tree_attention_with_a_full_lower_mask_is_causal_attention():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((5, 16)), rng.standard_normal((12, 16)), rng.standard_normal((12, 16))
    o, lse, p = serving.tree_attention(q, k, v, 5, None, 0.25)
    ro, rl = oracle.attention_forward(q, k, v, 0.25, causal=True)
    assert np.allclose(o, ro, atol=1e-14) and np.allclose(lse, rl, atol=1e-13)
    assert np.allclose(p.sum(1), 1)


def test_tree_attention_leaves_unseen_keys_out():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((3, 8)), rng.standard_normal((9, 8)), rng.standard_normal((9, 8))
    mask = np.eye(3, dtype=bool)
    mask[1] = False
    k[7], v[7] = np.nan, np.inf                      # drafted token 1, seen by nobody
    o, lse, _ = serving.tree_attention(q, k, v, 3, mask, 0.3)
    keep = [0, 1, 2, 3, 4, 5, 8]
    ro, rl = oracle.attention_forward(q[2:], k[keep], v[keep], 0.3)
    assert np.allclose(o[2], ro[0]) and np.allclose(lse[2], rl[0])
    o0, l0, _ = serving.tree_attention(q, k[6:], v[6:], 3, mask, 0.3)
    assert l0[1] == -np.inf and not o0[1].any()      # no context and no drafts: an empty row


@pytest.mark.parametrize("inter", [False, True])
def test_rope_turns_pairs_and_its_inverse_is_its_transpose(inter):
    rng = np.random.default_rng(5)
    x, g = rng.standard_normal((2, 1, 2, 3, 10))
    w = np.array([1.0, 0.3, 0.01])
    pos = np.array([[0, 7, 100]])
    y = serving.rope(x, pos, w, 1.5, inter)
    assert np.array_equal(y[..., 6:], x[..., 6:])
    assert np.allclose(y[:, :, 0, :6], 1.5 * x[:, :, 0, :6])
    a, b = (1, 0) if inter else (3, 0)               # element b's partner is a: (0, 1) or (0, 3)
    c, s = math.cos(7.0), math.sin(7.0)
    assert np.allclose(y[:, :, 1, b], 1.5 * (x[:, :, 1, b] * c - x[:, :, 1, a] * s))
    # <g, R x> = <Rᵀ g, x> on the turned part
    gb = serving.rope(g, pos, w, 1.5, inter, inverse=True)
    assert np.isclose((g * y)[..., :6].sum(), (gb * x)[..., :6].sum())
    h = 1e-6                                         # and against differences
    dx = np.zeros_like(x)
    dx[0, 1, 2, 4] = h
    assert np.isclose(((serving.rope(x + dx, pos, w, 1.5, inter) - y) * g).sum() / h, gb[0, 1, 2, 4], atol=1e-6)


def test_rope_frequencies():
    w, m = fa.rope_frequencies(128)
    assert m == 1.0 and w.dtype == np.float64 and np.allclose(w, 10000.0 ** (-np.arange(64) / 64))
    lin, _ = fa.rope_frequencies(128, scaling="linear", factor=4)
    assert np.allclose(lin, w / 4)
    base, _ = fa.rope_frequencies(64, scaling="base", factor=8)
    w64, _ = fa.rope_frequencies(64)
    assert base[0] == 1.0 and np.isclose(base[-1], w64[-1] / 8)
    ramp, m = fa.rope_frequencies(128, scaling="ramp", factor=8, original_len=4096)
    turns = 4096 * w / (2 * math.pi)
    assert np.array_equal(ramp[turns >= 32], w[turns >= 32]) and np.allclose(ramp[turns <= 1], w[turns <= 1] / 8)
    assert np.all(np.diff(ramp) < 0) and np.isclose(m, 0.1 * math.log(8) + 1)
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, scaling="cubic"), dict(rot_dim=8, factor=0.5),
                dict(rot_dim=2, scaling="base"), dict(rot_dim=8, base=-1.0),
                dict(rot_dim=8, scaling="ramp", low_turns=5, high_turns=5)):
        with pytest.raises(ValueError):
            fa.rope_frequencies(**bad)
