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


# ------------------------------------------------------------------ several axes, four bits, pages


def rope_axes(x, positions, axes, inv_freq, magnitude: float = 1.0, interleaved: bool = False, inverse: bool = False):
    """x [B,H,N,d], positions [A,B,N]: pair i turns by positions[axes[i]]·inv_freq[i], as in ``rope``."""
    x, w = np.asarray(x, dtype=np.float64), np.asarray(inv_freq, dtype=np.float64)
    r, out = 2 * len(w), np.array(x, dtype=np.float64)
    for i, a in enumerate(axes):
        turn = magnitude * np.exp((-1j if inverse else 1j) * (np.asarray(positions[int(a)], dtype=np.float64) * w[i]))[:, None]
        one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        z = (x[..., one] + 1j * x[..., two]) * turn
        out[..., one], out[..., two] = z.real, z.imag
    return out


E2M1_VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])  # code = index; bit 3 is the sign


def round_e2m1(y):
    """Codes of the nearest E2M1 values (ties to the even code, saturating), by search in the table of values."""
    a = np.minimum(np.abs(np.asarray(y, dtype=np.float64)), 6.0)
    hi = np.clip(np.searchsorted(E2M1_VALUES, a), 1, 7)
    lo = hi - 1
    dl, dh = a - E2M1_VALUES[lo], E2M1_VALUES[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code | np.where(np.signbit(y), 8, 0)).astype(np.uint8)


def quantise_groups(x, group: int = 32):
    """Rows [..., d] -> (codes [..., d], scale bytes [..., d/group], values [..., d]).

    k is the smallest whole number in [−126, 125] with max|x| <= 6·2^k over the
    group; a group with an infinity or NaN is NaN (byte 255, codes 0).
    """
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // group, group)
    fine = np.isfinite(g).all(-1)
    top = np.where(fine, np.abs(np.where(np.isfinite(g), g, 0)).max(-1), 0.0)
    k = np.searchsorted(6.0 * 2.0 ** np.arange(-126.0, 125.0), top) - 126  # the first that is not below
    power = 2.0 ** k[..., None].astype(np.float64)
    codes = np.where(fine[..., None], round_e2m1(np.where(fine[..., None], g, 0.0) / power), 0).astype(np.uint8)
    values = np.where(codes & 8, -1.0, 1.0) * E2M1_VALUES[codes & 7] * power
    values = np.where(fine[..., None], values, np.nan)
    return codes.reshape(x.shape), np.where(fine, k + 127, 255).astype(np.uint8), values.reshape(x.shape)


class Pool:
    """Pages shared, freed and reserved, one sequence after the other with plain lists.

    ``table`` rows are lists of page ids padded with −1, ``holders`` counts the
    sequences that name a page.
    """

    def __init__(self, table, lens, holders, bs: int):
        self.table, self.lens, self.holders, self.bs = [list(r) for r in table], list(lens), list(holders), bs

    def _pages(self, n):
        return -(-n // self.bs)

    def fork(self, src, dst):
        was = list(self.lens), [list(r) for r in self.table]
        for i, (s, t) in enumerate(zip(src, dst)):
            B = len(self.lens)
            if not (0 <= s < B and 0 <= t < B) or t in dst[:i] or s in dst:
                continue
            if was[0][t] != 0 or any(p >= 0 for p in was[1][t]):
                continue
            used = self._pages(self.lens[s])
            self.table[t] = self.table[s][:used] + [-1] * (len(self.table[s]) - used)
            self.lens[t] = self.lens[s]
            for p in self.table[t][:used]:
                self.holders[p] += 1

    def free(self, seqs, keep=None):
        for i, b in enumerate(seqs):
            n = 0 if keep is None else keep[i]
            if not 0 <= b < len(self.lens) or b in seqs[:i] or n < 0:
                continue
            self.lens[b] = min(self.lens[b], n)
            for j in range(self._pages(self.lens[b]), len(self.table[b])):
                if self.table[b][j] >= 0:
                    self.holders[self.table[b][j]] -= 1
                    self.table[b][j] = -1

    def reserve(self, new):
        """After the reservation and its copies, no page that the new tokens go into has another holder.

        Of the entries from the next token's on, those that are missing get a free page, and those whose page others
        hold too get one in its place, which is a copy where tokens of the sequence lie in the page.
        """
        B, held = len(self.lens), list(self.holders)
        granted, src, dst = [0] * B, [-1] * B, [-1] * B
        free = [p for p, n in enumerate(held) if n == 0]
        short = False
        for b in range(B):
            row, n = self.table[b], self.lens[b]
            if new[b] < 0 or n < 0 or n + new[b] > len(row) * self.bs:
                continue
            if new[b] == 0:
                granted[b] = 1
                continue
            entries = range(n // self.bs, self._pages(n + new[b]))
            if any(row[j] >= len(held) or (row[j] < 0 and j * self.bs < n) or (row[j] >= 0 and held[row[j]] < 1)
                   for j in entries):
                continue
            needs = [j for j in entries if row[j] < 0 or self.holders[row[j]] > 1]
            short = short or len(needs) > len(free)
            if short:
                continue
            granted[b] = 1
            for j in needs:
                page = free.pop(0)
                if row[j] >= 0:
                    self.holders[row[j]] -= 1
                    if j * self.bs < n:
                        src[b], dst[b] = row[j], page
                row[j] = page
                self.holders[page] = 1
        return granted, src, dst
