"""A paged cache in four bits, shared by its tests (the cache's bounds are those of ``serving_helpers``)."""

from __future__ import annotations

import numpy as np

from oracle import serving
from tests.serving_helpers import bf16, check_tree, np64


def pack(codes):
    """Codes [..., d] -> bytes [..., d/2], the first of two in the low half."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def values(packed, scales):
    """What packed codes and scale bytes [..., d/32] stand for, in float64."""
    c = np.stack((packed & 15, packed >> 4), -1).reshape(*packed.shape[:-1], -1)
    v = np.where(c & 8, -1.0, 1.0) * serving.E2M1_VALUES[c & 7]
    power = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return v * np.repeat(power, 32, axis=-1)


def check_tree4(o, lse, q, paged, drafts, mask, scale, heads=None):
    """``check_tree`` with the bounds of an E4M3 cache, which hold for one in four bits: its weights are fp16 too (off by 2^-11
    of themselves, or below 2^-14 by half of 2^-24 where the row's largest is at least 2^3); up to 32 rows that share a key
    head q goes in as two E4M3 terms, beyond as fp16 with 16 bits below the row's largest (both within 2^-18 of it); and
    values times their groups' powers of two are exact."""
    paged.cache = "e4m3"
    check_tree(o, lse, q, paged, drafts, mask, scale, heads)


class Paged4:
    """Sequences of given lengths in a shuffled page pool in four bits whose other slots are NaN, tables padded with −1.

    ``k`` and ``v`` are lists of the live rows [H, len, d] in float64, as the cache holds them.
    """

    def __init__(self, rng, lens, hkv, d, bs, spare=3, edit=None):
        import torch
        self.lens, self.bs, self.d, self.hkv = [int(n) for n in lens], bs, d, hkv
        per = max(1, -(-max(self.lens) // bs)) + 1
        used = [-(-n // bs) for n in self.lens]
        nb = sum(used) + spare
        order = rng.permutation(nb)
        table = np.full((len(lens), per), -1, dtype=np.int32)
        codes = {n: rng.integers(0, 256, (nb, hkv, bs, d // 2)).astype(np.uint8) for n in "kv"}
        scales = {n: np.full((nb, hkv, bs, d // 32), 255, dtype=np.uint8) for n in "kv"}
        self.k, self.v = [], []
        nxt = 0
        for b, n in enumerate(self.lens):
            table[b, : used[b]] = order[nxt : nxt + used[b]]
            nxt += used[b]
            at = np.arange(n)
            page, slot = table[b][at // bs], at % bs
            for name in "kv":
                x = np64(bf16(rng.standard_normal((hkv, n, d)) * np.exp2(rng.integers(-2, 3, (hkv, n, 1)))))
                if edit is not None:
                    edit(name, b, x)
                    x = np64(bf16(x))
                c, s, y = serving.quantise_groups(x)
                codes[name][page, :, slot] = pack(c).transpose(1, 0, 2)
                scales[name][page, :, slot] = s.transpose(1, 0, 2)
                getattr(self, name).append(y)
        self.k_cache, self.v_cache = (torch.from_numpy(codes[n]).cuda() for n in "kv")
        self.k_scale, self.v_scale = (torch.from_numpy(scales[n]).cuda() for n in "kv")
        self.table = torch.from_numpy(table).cuda()
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def args(self):
        return (self.k_cache, self.v_cache, self.table, self.seq_lens)

    def kw(self):
        return dict(k_scale=self.k_scale, v_scale=self.v_scale)
