"""Float64 oracle for the operators around attention: rotary positions, the
paged cache's E4M3 rows, and attention of drafted tokens.

TEST INFRASTRUCTURE ONLY, like ``oracle.attention``: plain definitions in
float64 NumPy, sharing no code with the CUDA path.
"""

from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def rope(x, positions, inv_freq, magnitude: float = 1.0, interleaved: bool = False, inverse: bool = False):
    """x [B,H,N,d], positions [B,N] whole numbers: the first 2·len(inv_freq) elements turned, the rest kept.

    A pair is a complex number z = x₁ + i·x₂; it becomes μ·z·e^{±iθ}.
    """
    x = np.asarray(x, dtype=np.float64)
    w = np.asarray(inv_freq, dtype=np.float64)
    r = 2 * len(w)
    theta = np.asarray(positions, dtype=np.float64)[:, None, :, None] * w
    turn = magnitude * np.exp((-1j if inverse else 1j) * theta)
    out = x.copy()
    if interleaved:
        z = (x[..., 0:r:2] + 1j * x[..., 1:r:2]) * turn
        out[..., 0:r:2], out[..., 1:r:2] = z.real, z.imag
    else:
        z = (x[..., : r // 2] + 1j * x[..., r // 2 : r]) * turn
        out[..., : r // 2], out[..., r // 2 : r] = z.real, z.imag
    return out


def e4m3_values() -> np.ndarray:
    """The 127 non-negative finite E4M3 values in order (code = index)."""
    e, m = np.divmod(np.arange(127), 8)
    return np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))


def round_e4m3(y) -> np.ndarray:
    """Nearest E4M3 value (ties to the even code), by search in the table of values; NaN for what is not finite."""
    y = np.asarray(y, dtype=np.float64)
    table = e4m3_values()
    a = np.minimum(np.abs(np.where(np.isfinite(y), y, 0.0)), E4M3_MAX)
    hi = np.clip(np.searchsorted(table, a), 1, 126)
    lo = hi - 1
    dl, dh = a - table[lo], table[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return np.where(np.isfinite(y), np.copysign(table[code], y), np.nan)


def quantise_rows(x):
    """Rows [..., d] -> (E4M3 values y with x ≈ y·2^k, k): k >= −126 the smallest with max|x| <= 448·2^k over
    the finite entries."""
    x = np.asarray(x, dtype=np.float64)
    top = np.max(np.where(np.isfinite(x), np.abs(x), 0.0), axis=-1)
    k = np.full(top.shape, -126, dtype=np.int64)
    for i in np.ndindex(top.shape):
        while top[i] > E4M3_MAX * 2.0 ** int(k[i]):
            k[i] += 1
    return round_e4m3(x * 2.0 ** (-k[..., None].astype(np.float64))), k


def tree_attention(q, k, v, drafts: int, mask, scale: float):
    """One key/value head of one sequence: q [T, d], k and v [n, d], of which the last ``drafts`` rows are drafted.

    Returns (O [T, d], LSE [T], P [T, n]).  Rows t >= drafts and rows that see
    nothing give 0 and −inf.  A key that a row does not see is left out of its
    sums altogether, whatever it holds.
    """
    q, k, v = (np.asarray(a, dtype=np.float64) for a in (q, k, v))
    T, n = q.shape[0], k.shape[0]
    o, lse, p_all = np.zeros((T, v.shape[1])), np.full((T,), -np.inf), np.zeros((T, n))
    context = n - drafts
    for t in range(min(T, drafts)):
        sees = np.ones((n,), dtype=bool)
        sees[context:] = [u <= t if mask is None else bool(mask[t][u]) for u in range(drafts)]
        if not sees.any():
            continue
        s = scale * (k[sees] @ q[t])
        m = s.max()
        e = np.exp(s - m)
        p = e / e.sum()
        o[t] = p @ v[sees]
        lse[t] = m + np.log(e.sum())
        p_all[t, sees] = p
    return o, lse, p_all
