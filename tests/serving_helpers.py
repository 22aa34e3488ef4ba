"""Paged caches, masks and error bounds shared by the tests of the cache and of drafted-token attention."""

from __future__ import annotations

import numpy as np

from oracle import serving


def bf16(x):
    import torch
    return torch.as_tensor(np.asarray(x, dtype=np.float32)).to(torch.bfloat16)


def np64(t):
    return t.detach().double().cpu().numpy()


def codes_of(values) -> np.ndarray:
    """E4M3 codes of values that are exactly E4M3 (NaN gives 0x7F)."""
    v = np.asarray(values, dtype=np.float64)
    c = np.searchsorted(serving.e4m3_values(), np.where(np.isnan(v), 0, np.abs(v))).astype(np.uint8)
    c = np.where(np.isnan(v), 0x7F, c | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)
    return c


class Paged:
    """Sequences of given lengths in a shuffled page pool whose other slots hold NaN, tables padded with −1.

    ``k`` and ``v`` are lists of the live rows [H, len, d] in float64, as the cache holds them.
    """

    def __init__(self, rng, lens, hkv, d, bs, cache, spare=3, edit=None):
        import torch
        self.lens, self.bs, self.d, self.hkv, self.cache = [int(n) for n in lens], bs, d, hkv, cache
        B = len(lens)
        per = max(1, -(-max(self.lens) // bs)) + 1
        used = [-(-n // bs) for n in self.lens]
        nb = sum(used) + spare
        order = rng.permutation(nb)
        table = np.full((B, per), -1, dtype=np.int32)
        pools, scales, self.k, self.v = {}, {}, [], []
        for name in ("k", "v"):
            if cache == "e4m3":
                pools[name] = np.full((nb, hkv, bs, d), 0x7F, dtype=np.uint8)
                scales[name] = np.full((nb, hkv, bs), 0xFF, dtype=np.uint8)
            else:
                pools[name] = np.full((nb, hkv, bs, d), np.nan, dtype=np.float32)
        nxt = 0
        for b, n in enumerate(self.lens):
            table[b, : used[b]] = order[nxt : nxt + used[b]]
            nxt += used[b]
            at = np.arange(n)
            page, slot = table[b][at // bs], at % bs
            for name in ("k", "v"):
                x = np64(bf16(rng.standard_normal((hkv, n, d)) * np.exp2(rng.integers(-2, 3, (hkv, n, 1)))))
                if edit is not None:
                    edit(name, b, x)
                    x = np64(bf16(x))  # the reference holds what the cache holds
                if cache == "e4m3":
                    y, e = serving.quantise_rows(x)
                    pools[name][page, :, slot] = codes_of(y).transpose(1, 0, 2)
                    scales[name][page, :, slot] = (e + 127).astype(np.uint8).T
                    x = y * 2.0 ** e[..., None]
                else:
                    pools[name][page, :, slot] = x.transpose(1, 0, 2)
                getattr(self, name).append(x)
        if cache == "e4m3":
            self.k_cache, self.v_cache = (torch.from_numpy(pools[n]).view(torch.float8_e4m3fn).cuda() for n in "kv")
            self.k_scale, self.v_scale = (torch.from_numpy(scales[n]).cuda() for n in "kv")
        else:
            self.k_cache, self.v_cache = (torch.from_numpy(pools[n]).to(torch.bfloat16).cuda() for n in "kv")
            self.k_scale = self.v_scale = None
        self.table = torch.from_numpy(table).cuda()
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def args(self):
        return (self.k_cache, self.v_cache, self.table, self.seq_lens)

    def kw(self):
        return dict(k_scale=self.k_scale, v_scale=self.v_scale)


def random_tree(rng, B, T, empty=0.0):
    """[B,T,T] bool: each token sees itself and a random ancestor chain; a share ``empty`` of the rows sees no draft."""
    mask = np.zeros((B, T, T), dtype=bool)
    for b in range(B):
        for t in range(T):
            parent = int(rng.integers(-1, t)) if t else -1
            if parent >= 0:
                mask[b, t] = mask[b, parent]
            mask[b, t, t] = True
        mask[b, rng.random(T) < empty] = False
    return mask


def check_tree(o, lse, q, paged, drafts, mask, scale, heads=None):
    """Compare with the oracle, element by element.

    Bounds, from the roundings on the way: O is stored as bf16 (2^-8 |O|); the
    probabilities enter the second product in the cache's matrix type, bf16 or
    fp16 (2^-8 or 2^-11 of Σ p|v|); scores are fp32 sums (and q enters an E4M3
    product as two E4M3 terms, 2^-18 of the row's largest element), so each is
    off by at most 2^-16 of the largest Σ|q||k|·σ plus 2^-18·max|q|·Σ|k|·σ,
    which moves a probability by twice that, relatively; exponential, row sum and
    division are fp32 (2^-18 together).  fp16 probabilities (E4M3 cache) are kept
    relative to a reference at most 2^-3 of the row's largest one, and below
    2^-14 they are multiples of 2^-24: off by half of that, 2^-28 of the largest
    one, and never by more than they are, since 0 is a multiple too.
    """
    o, lse, q = np64(o), np64(lse), np64(q)
    B, Hq, T, d = q.shape
    G = Hq // paged.hkv
    p_type = 2.0 ** -11 if paged.cache == "e4m3" else 2.0 ** -8
    for b in range(B):
        for h in range(Hq) if heads is None else heads:
            k, v = paged.k[b][h // G], paged.v[b][h // G]
            m = int(drafts[b])
            ro, rl, p = serving.tree_attention(q[b, h], k, v, m, None if mask is None else mask[b], scale)
            fin = np.isfinite(rl)
            assert np.array_equal(np.isneginf(lse[b, h]), np.isneginf(rl)), (b, h)
            assert np.array_equal(np.isnan(lse[b, h]), np.isnan(rl)), (b, h)
            assert np.all(o[b, h][np.isneginf(rl)] == 0), (b, h)
            if not fin.any():
                continue
            kf, vf = (np.where(np.isfinite(a), np.abs(a), 0.0) for a in (k, v))
            es = scale * (2.0 ** -16 * (np.abs(q[b, h]) @ kf.T).max(1)
                          + 2.0 ** -18 * np.abs(q[b, h]).max(1) * kf.sum(1).max())
            assert np.all(np.abs(lse[b, h][fin] - rl[fin]) <= (es + 2.0 ** -18 * (1 + np.abs(rl)))[fin]), (b, h)
            bound = 2.0 ** -8 * np.abs(ro) + (p_type + 2 * es[:, None] + 2.0 ** -18) * (p @ vf)
            if paged.cache == "e4m3":
                bound = bound + np.minimum(p, 2.0 ** -28 * p.max(1, keepdims=True)) @ vf
            ok = np.isfinite(ro) & fin[:, None]
            assert np.array_equal(np.isfinite(o[b, h])[fin], np.isfinite(ro)[fin]), (b, h)
            err = np.abs(o[b, h][ok] - ro[ok])
            assert np.all(err <= bound[ok]), (b, h, float((err / np.maximum(bound[ok], 1e-300)).max()))
