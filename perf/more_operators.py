"""Cases of the operators around a paged cache in four bits: rotary positions with several axes, rows written to the
cache and read back, attention of drafted tokens over it, accepted rows moved together, and pages shared, reserved,
copied and freed.

``listed()`` names the cases, ``draw()`` gives more of the same ranges, ``prepare()`` makes what a program has in hand,
``run()`` is one pass (in plain torch operations, or through the library where ``own`` is true), ``exact()`` the same from
the definition in float64.
"""

import math

import torch

own = False

DEV = "cuda"
GROUP = 32  # elements that share a power of two in the four-bit cache


# ------------------------------------------------------------------------------------------------ cases


def listed():
    return [
        # One new token of one sequence, the 28 query / 4 key heads of the grouped decode, three axes: launch latency.
        dict(name="axes_decode", op="axes", B=1, Hq=28, Hk=4, N=1, d=128, rot=128, nt=1, nh=1, nw=1, inter=False, order="blocks",
             dtype="bf16", bnhd=False, backward=False),
        # Gradients of q and k at the training shape: a video of 8 x 32 x 32 patches, its axes interleaved pair by pair.
        dict(name="axes_video_bwd", op="axes", B=2, Hq=16, Hk=16, N=8192, d=128, rot=128, nt=8, nh=32, nw=32, inter=False,
             order="cycle", dtype="bf16", bnhd=True, backward=True),
        # A short chunk of a prompt behind an odd prefix: written in four bits, and all read back.
        dict(name="extend_short", op="extend", B=1, Hkv=4, N=17, d=64, bs=16, start=101, ragged=False, bnhd=True),
        # Chunks of up to 8192 tokens of eight sequences behind a prefix, and prefix and chunk read back for the prefill.
        dict(name="extend_chunk", op="extend", B=8, Hkv=4, N=8192, d=128, bs=64, start=2048, ragged=True, bnhd=True),
        # A small tree on one short sequence: latency.
        dict(name="four_short", op="tree", B=1, Hq=28, Hkv=4, T=5, L=777, d=128, bs=16, ragged=False, padded=False,
             mask=True, bnhd=True),
        # Single tokens of 64 ragged sequences, 16-key pages.
        dict(name="four_single", op="tree", B=64, Hq=28, Hkv=4, T=1, L=8192, d=128, bs=16, ragged=True, padded=False,
             mask=False, bnhd=False),
        # Eight drafted tokens of 16 ragged sequences: 56 rows that share a key head.
        dict(name="four_draft8", op="tree", B=16, Hq=28, Hkv=4, T=8, L=8192, d=128, bs=16, ragged=True, padded=True,
             mask=True, bnhd=True),
        # Wide trees over long contexts.
        dict(name="four_wide", op="tree", B=8, Hq=32, Hkv=8, T=64, L=32768, d=128, bs=64, ragged=False, padded=False,
             mask=True, bnhd=True),
        # Drafted rows of 16 sequences written and the accepted ones moved together.
        dict(name="accept_draft8", op="compact", B=16, Hkv=4, L=1000, first=1000, N=8, d=128, bs=16, cache="bf16", drafts=True),
        # Long sequences cut down to their first rows and some of the last ones.
        dict(name="evict_long", op="compact", B=8, Hkv=8, L=16384, first=257, N=6000, d=128, bs=64, cache="e4m3", drafts=False),
        # Four sequences, each continued in four ways: shared pages, room for one token each.
        dict(name="branch_small", op="branch", roots=4, ways=4, Hkv=4, L=500, N=1, d=128, bs=16, spare=200, cache="bf16"),
        # 64 long sequences continued in eight ways over a large pool, room for 40 tokens each.
        dict(name="branch_large", op="branch", roots=64, ways=8, Hkv=2, L=4000, N=40, d=64, bs=16, spare=40000, cache="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["axes", "extend", "tree", "tree", "tree", "compact", "branch"])
    if op == "axes":
        d = rng.choice([64, 128])
        nt, nh, nw = _log(rng, 1, 16), _log(rng, 1, 24), _log(rng, 1, 24)
        Hk = rng.choice([1, 2, 4, 8, 16])
        return dict(op=op, B=_log(rng, 1, 4), Hq=Hk * rng.choice([1, 2, 4, 7]) if nt * nh * nw < 2000 else Hk, Hk=Hk,
                    N=nt * nh * nw, d=d, rot=rng.choice([d, d // 2]), nt=nt, nh=nh, nw=nw, inter=rng.random() < 0.5,
                    order=rng.choice(["blocks", "cycle"]), dtype=rng.choice(["bf16", "bf16", "fp32"]), bnhd=rng.random() < 0.5,
                    backward=rng.random() < 0.5)
    if op == "extend":
        return dict(op=op, B=_log(rng, 1, 32), Hkv=rng.choice([1, 2, 4, 8]), N=_log(rng, 1, 2048), d=rng.choice([64, 128]),
                    bs=rng.choice([16, 32, 64, 128]), start=rng.randrange(0, 2000), ragged=rng.random() < 0.6,
                    bnhd=rng.random() < 0.5)
    if op == "tree":
        B, T, Hkv = _log(rng, 1, 24), _log(rng, 1, 64), rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 7, 8])
        most = min(16384, (1 << 29) // (B * T * Hq))  # no more score entries than the largest listed case has
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, T=T, L=max(T, _log(rng, 16, most)), d=rng.choice([64, 128]),
                    bs=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.6, padded=rng.random() < 0.4,
                    mask=rng.random() < 0.7, bnhd=rng.random() < 0.5)
    if op == "compact":
        drafts = rng.random() < 0.5
        N = _log(rng, 1, 64) if drafts else _log(rng, 1, 2000)
        first = rng.randrange(0, 2000)
        return dict(op=op, B=_log(rng, 1, 32), Hkv=rng.choice([1, 2, 4, 8]), L=first if drafts else first + 4 * N + 3, first=first,
                    N=N, d=rng.choice([64, 128]), bs=rng.choice([16, 32, 64, 128]), cache=rng.choice(["bf16", "e4m3"]),
                    drafts=drafts)
    return dict(op="branch", roots=_log(rng, 1, 64), ways=rng.randrange(2, 9), Hkv=rng.choice([1, 2, 4]), L=_log(rng, 1, 2000),
                N=_log(rng, 1, 100), d=rng.choice([64, 128]), bs=rng.choice([16, 32, 64, 128]), spare=_log(rng, 1, 4000),
                cache=rng.choice(["bf16", "e4m3"]))


def _lens(n, B, ragged, least):
    """Length of each of B sequences: the longest has n; ragged ones spread over the upper half."""
    return [max(least, n - (b * 1237) % (n // 2 + 1)) if ragged else n for b in range(B)]


def _kept(c):
    """Rows that a compaction keeps of each sequence: what is accepted of its drafts, or most of what it may keep."""
    return [(b * 5 + c["N"]) % (c["N"] + 1) if c["drafts"] else c["N"] - (b * 7) % (c["N"] // 3 + 1) for b in range(c["B"])]


def work(c):
    if c["op"] == "axes":
        n = c["B"] * (c["Hq"] + c["Hk"]) * c["N"] * c["d"]
        return {"bytes": 2 * n * (4 if c["dtype"] == "fp32" else 2) + 12 * c["B"] * c["N"], "flops": 3 * n * c["rot"] // c["d"]}
    four = c["d"] // 2 + c["d"] // GROUP  # bytes of a row in four bits
    if c["op"] == "extend":
        new, pre = _lens(c["N"], c["B"], c["ragged"], 1), [max(0, c["start"] - 3 * b) for b in range(c["B"])]
        rows, full = 2 * c["Hkv"] * sum(new), 2 * c["Hkv"] * c["B"] * (c["start"] + c["N"])
        read = 2 * c["Hkv"] * (sum(new) + sum(pre))
        return {"bytes": rows * (2 * c["d"] + four) + read * four + full * 2 * c["d"], "flops": (2 * rows + read) * c["d"]}
    if c["op"] == "tree":
        lens = _lens(c["L"], c["B"], c["ragged"], c["T"])
        qo = c["B"] * c["Hq"] * c["T"] * (4 * c["d"] + 4)
        return {"bytes": 2 * c["Hkv"] * sum(lens) * four + qo, "flops": 4 * c["Hq"] * c["T"] * sum(lens) * c["d"]}
    row = 2 * c["d"] if c["cache"] == "bf16" else c["d"] + 1
    if c["op"] == "compact":
        moved = 2 * c["Hkv"] * sum(_kept(c))
        wrote = 2 * c["Hkv"] * c["B"] * c["N"] if c["drafts"] else 0
        return {"bytes": 2 * moved * row + wrote * (2 * c["d"] + row) + 4 * sum(_kept(c)), "flops": 0}
    # Entries of the tables that change hands, and the last page of every continued sequence but one of each kind.
    pages = c["roots"] * c["ways"] * (-(-c["L"] // c["bs"]))
    copied = c["roots"] * c["ways"] * c["bs"] * row * 2 * c["Hkv"] if c["L"] % c["bs"] else 0
    return {"bytes": 24 * pages + 2 * copied, "flops": 0}


# ------------------------------------------------------------------------------------------------ inputs


def _quantise8(x):
    """E4M3 codes and E8M0 scale bytes of the rows of x (last dimension): the smallest power of two that holds the row."""
    x = x.float()
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)
    k = torch.where(amax > 0, e - 9 + (m > 0.875).int(), -126).clamp(-126, 127)
    return torch.ldexp(x, -k[..., None]).to(torch.float8_e4m3fn), (k + 127).to(torch.uint8)


def _quantise4(x):
    """Packed E2M1 codes (two to a byte, the first in the low half) and E8M0 bytes of groups of 32: the smallest power of
    two that holds the group's largest finite magnitude, from 2^-126 to 2^125; a group with others in it is NaN."""
    g = x.float().unflatten(-1, (-1, GROUP))
    fine = g.isfinite()
    amax = torch.where(fine, g.abs(), 0.0).amax(-1)
    m, e = torch.frexp(amax)
    k = torch.where(amax > 0, e - 3 + (m > 0.75).int(), -126).clamp(-126, 125)
    whole = fine.all(-1)
    y = torch.where(whole[..., None], torch.ldexp(g, -k[..., None]), 0.0)
    a = y.abs()
    # Values 0, 0.5, 1, 1.5, 2, 3, 4, 6: steps of 0.5, 1 and 2; halves go to the even code.
    code = torch.where(a < 2, torch.round(a * 2), torch.where(a < 4, torch.round(a) + 2, torch.round(a / 2) + 4)).clamp(max=7)
    code = (code.to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.where(whole, k + 127, 255).to(torch.uint8)


def _values4(code, scale):
    """What packed codes and scale bytes stand for, in float32."""
    c = torch.stack((code & 15, code >> 4), -1).flatten(-2)
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=c.device)
    v = torch.ldexp(table[c.int()].unflatten(-1, (-1, GROUP)), (scale.int() - 127)[..., None])
    return torch.where((scale == 255)[..., None], math.nan, v).flatten(-2)


def _layout(x, bnhd):
    """[B,H,N,d] in its own layout, or as a view of [B,N,H,d]."""
    return x.transpose(1, 2).contiguous().transpose(1, 2) if bnhd else x


def _pool(c, g, nb):
    """A page pool of nb pages filled with normal rows, the keys with a few strong channels."""
    kind, s = c.get("cache", "e2m1"), {}
    for n in ("k", "v"):
        x = torch.randn((nb, c["Hkv"], c["bs"], c["d"]), generator=g, device=DEV, dtype=torch.bfloat16)
        if n == "k":
            x[..., ::17] *= 3
        if kind == "bf16":
            s[n + "_cache"], s[n + "_scale"] = x, None
        else:
            x = x * torch.exp2(torch.randint(-1, 2, x.shape[:-1], generator=g, device=DEV))[..., None]
            s[n + "_cache"], s[n + "_scale"] = (_quantise8 if kind == "e4m3" else _quantise4)(x)
    return s


def _cache(c, g, most, lens):
    """A pool for sequences of up to `most` keys, its pages handed out in a random order."""
    per = -(-most // c["bs"])
    nb = c["B"] * per + 3
    s = _pool(c, g, nb)
    table = torch.randperm(nb, generator=g, device=DEV)[: c["B"] * per].view(c["B"], per).int()
    used = (torch.tensor(lens, device=DEV) + c["bs"] - 1) // c["bs"]
    s["table"] = torch.where(torch.arange(per, device=DEV)[None] < used[:, None], table, -1).int()
    return s


def _ints(x):
    return torch.tensor(x, device=DEV, dtype=torch.int32)


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    gc = torch.Generator().manual_seed(seed)
    d, s = c["d"], {"case": c}

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device=DEV, dtype=dtype)

    if c["op"] == "axes":
        B, r, nh, nw = c["B"], c["rot"], c["nh"], c["nw"]
        dt = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16
        s["q"] = _layout(normal(B, c["Hq"], c["N"], d, dtype=dt), c["bnhd"])
        s["k"] = _layout(normal(B, c["Hk"], c["N"], d, dtype=dt), c["bnhd"])
        # Time, height and width of every patch, behind a text of some length.
        n = torch.arange(c["N"], device=DEV)
        where = torch.stack((n // (nh * nw), n // nw % nh, n % nw))[:, None]
        s["positions"] = (where + torch.randint(0, 30000, (1, B, 1), generator=g, device=DEV)).int()
        i = torch.arange(r // 2)
        # A quarter of the pairs for time and the rest for height and width in blocks, or the three in turn.
        s["axes"] = (i % 3 if c["order"] == "cycle" else (i >= r // 8).int() + (i >= r // 8 + (r // 2 - r // 8) // 2).int()).int()
        s["inv_freq"] = 10000.0 ** (-2 * i.double() / r)
        s["inv_freq_dev"], s["axes_dev"] = s["inv_freq"].to(DEV), s["axes"].to(DEV).long()
        return s
    if c["op"] == "extend":
        lens = _lens(c["N"], c["B"], c["ragged"], 1)
        start = [max(0, c["start"] - 3 * b) for b in range(c["B"])]
        s.update(_cache(c, g, c["start"] + c["N"], [a + n for a, n in zip(start, lens)]))
        s["k"], s["v"] = (_layout(normal(c["B"], c["Hkv"], c["N"], d), c["bnhd"]) for _ in range(2))
        s["start"], s["new_lens"] = _ints(start), _ints(lens)
        s["lens"] = s["start"] + s["new_lens"]
        return s
    if c["op"] == "tree":
        B, T = c["B"], c["T"]
        lens = _lens(c["L"], B, c["ragged"], T)
        s.update(_cache(c, g, max(lens), lens))
        s["lens"] = _ints(lens)
        s["q"] = _layout(normal(B, c["Hq"], T, d), c["bnhd"])
        s["draft_lens"] = _ints([max(1, T - b % 3) for b in range(B)]) if c["padded"] else None
        s["mask"] = None
        if c["mask"]:  # each token follows a random earlier one, or starts a branch of its own
            mask = torch.zeros((B, T, T), dtype=torch.bool)
            for t in range(T):
                parent = torch.randint(-1, max(t, 1), (B,), generator=gc) if t else torch.full((B,), -1)
                mask[:, t] = mask[torch.arange(B), parent.clamp_min(0)] & (parent >= 0)[:, None]
                mask[:, t, t] = True
            s["mask"] = mask.to(DEV)
        # Scratch that a serving loop keeps: partial results of up to 64 splits.
        s["workspace"] = torch.empty(max(1 << 22, 64 * min(B * c["Hq"] * T, 4096) * (d + 2) * 4), dtype=torch.uint8, device=DEV)
        return s
    if c["op"] == "compact":
        B, N, kept = c["B"], c["N"], _kept(c)
        most = c["L"] + (N if c["drafts"] else 0)
        s.update(_cache(c, g, most, [most] * B))
        keep = torch.zeros((B, N), dtype=torch.int32)
        for b in range(B):  # rising positions: drafted rows, or rows of the last part, behind all that is written
            if c["drafts"]:
                pick = torch.randperm(N, generator=gc)[: kept[b]].sort().values + c["first"]
            else:
                lo = c["first"] + N
                pick = torch.randperm(c["L"] - lo, generator=gc)[: kept[b]].sort().values + lo
            keep[b, : kept[b]] = pick
        s["keep"], s["keep_lens"], s["first"] = keep.to(DEV), _ints(kept), _ints([c["first"]] * B)
        if c["drafts"]:
            s["k"], s["v"] = (normal(B, c["Hkv"], N, d) for _ in range(2))
        return s
    # branch: the last rows of the table are sequences, the first ones their continuations, empty so far.
    S, W = c["roots"], c["ways"]
    B, per = S * (W + 1), -(-(c["L"] + c["N"]) // c["bs"])
    lens = [max(1, c["L"] - (b * 37) % (c["L"] // 2 + 1)) for b in range(S)]
    nb = sum(-(-n // c["bs"]) for n in lens) + S * W + c["spare"]
    s.update(_pool(c, g, nb))
    order, at = torch.randperm(nb, generator=gc), 0
    table = torch.full((B, per), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        m = -(-n // c["bs"])
        table[S * W + b, :m] = order[at : at + m].int()
        at += m
    refs = torch.zeros(nb, dtype=torch.int32)
    refs[order[:at]] = 1
    s["table"], s["refs"] = table.to(DEV), refs.to(DEV)
    s["lens"] = _ints([0] * (S * W) + lens)
    s["all"] = torch.arange(B, device=DEV, dtype=torch.int32)
    s["back_to"] = s["lens"].clone()
    s["dst"] = torch.arange(S * W, device=DEV, dtype=torch.int32)
    s["src"] = (S * W + s["dst"] // W).int()
    s["new"] = _ints([1 + (b * 11 + c["N"] - 1) % c["N"] for b in range(B)])
    return s


# ------------------------------------------------------------------------------------------------ one pass


def run(s):
    return globals()[("own_" if own else "plain_") + s["case"]["op"]](s)


def own_axes(s):
    from io_aware_exact_11_gb300 import fa
    f = fa.rope_axes_backward if s["case"]["backward"] else fa.rope_axes
    return f(s["q"], s["k"], s["inv_freq"], s["axes"], s["positions"], interleaved=s["case"]["inter"])


def own_extend(s):
    from io_aware_exact_11_gb300 import fa
    scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
    fa.cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["start"], new_lens=s["new_lens"], **scales)
    return fa.cache_gather(s["k_cache"], s["v_cache"], s["table"], s["lens"], s["case"]["start"] + s["case"]["N"], **scales)


def own_tree(s):
    from io_aware_exact_11_gb300 import fa
    return fa.decode_tree(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], tree_mask=s["mask"],
                          draft_lens=s["draft_lens"], k_scale=s["k_scale"], v_scale=s["v_scale"], workspace=s["workspace"])


def own_compact(s):
    from io_aware_exact_11_gb300 import fa
    scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
    if s["case"]["drafts"]:
        fa.cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["first"], **scales)
    fa.cache_compact(s["k_cache"], s["v_cache"], s["table"], s["first"], s["keep"], keep_lens=s["keep_lens"], **scales)
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def own_branch(s):
    from io_aware_exact_11_gb300 import fa
    bs = s["case"]["bs"]
    fa.pages_free(s["table"], s["lens"], s["refs"], s["all"], bs, keep_lens=s["back_to"])
    fa.pages_fork(s["table"], s["lens"], s["refs"], s["src"], s["dst"], bs)
    granted, old, new = fa.pages_reserve(s["table"], s["lens"], s["refs"], s["new"], bs)
    fa.cache_copy_pages(s["k_cache"], s["v_cache"], old, new, k_scale=s["k_scale"], v_scale=s["v_scale"])
    return (s["table"], s["lens"], s["refs"], granted, old, new, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])


def plain_axes(s):
    c = s["case"]
    r = c["rot"]
    angle = s["positions"][s["axes_dev"]].permute(1, 2, 0).double() * s["inv_freq_dev"]  # [B, N, pairs]
    if c["backward"]:
        angle = -angle
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def rotate(x):
        y = x.float()
        if c["inter"]:
            a, b = y[..., 0:r:2], y[..., 1:r:2]
            turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = y[..., : r // 2], y[..., r // 2 : r]
            turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((turned, y[..., r:]), -1).to(x.dtype)

    return rotate(s["q"]), rotate(s["k"])


def _write(s, name, quantise):
    """The new rows of `name` to their places in the cache."""
    c = s["case"]
    n = torch.arange(c["N"], device=DEV)
    count = s["new_lens"] if "new_lens" in s else torch.full((c["B"],), c["N"], device=DEV)
    b, n = torch.nonzero(n[None] < count[:, None], as_tuple=True)
    at = (s["start"] if "start" in s else s["first"]).long()[b] + n
    page, slot = s["table"].long()[b, at // c["bs"]], at % c["bs"]
    x, cache = s[name].transpose(1, 2)[b, n], s[name + "_cache"]
    if quantise is None:
        cache[page, :, slot] = x
    else:
        code, scale = quantise(x)
        cache.view(torch.uint8)[page, :, slot] = code.view(torch.uint8)
        s[name + "_scale"][page, :, slot] = scale


def _paged(s, name, L):
    """The first L rows of each sequence in float32 [B,H,L,d]; rows past a sequence are some page's."""
    pages = s["table"][:, : -(-L // s["case"]["bs"])].long().clamp_min(0)
    return _values4(s[name + "_cache"][pages], s[name + "_scale"][pages]).transpose(1, 2).flatten(2, 3)[:, :, :L]


def plain_extend(s):
    _write(s, "k", _quantise4)
    _write(s, "v", _quantise4)
    L = s["case"]["start"] + s["case"]["N"]
    live = (torch.arange(L, device=DEV)[None] < s["lens"][:, None])[:, None, :, None]
    return (torch.where(live, _paged(s, "k", L), 0.0).to(torch.bfloat16), torch.where(live, _paged(s, "v", L), 0.0).to(torch.bfloat16))


def plain_tree(s):
    c = s["case"]
    B, Hq, Hkv, T, d = c["B"], c["Hq"], c["Hkv"], c["T"], c["d"]
    L = s["table"].shape[1] * c["bs"]
    k, v = _paged(s, "k", L), _paged(s, "v", L)
    drafts = s["draft_lens"] if s["draft_lens"] is not None else torch.full((B,), T, device=DEV)
    context = (s["lens"] - drafts).long()
    j, t = torch.arange(L, device=DEV), torch.arange(T, device=DEV)
    mask = s["mask"] if s["mask"] is not None else (t[None] <= t[:, None]).expand(B, T, T)
    u = (j[None] - context[:, None]).clamp(0, T - 1)
    seen = mask.gather(2, u[:, None].expand(B, T, L)) & (j[None] < s["lens"][:, None])[:, None]
    seen = (seen | (j[None] < context[:, None])[:, None]) & (t[None] < drafts[:, None])[..., None]
    q = s["q"].float().reshape(B, Hkv, Hq // Hkv * T, d)
    score = (q @ k.transpose(-1, -2)).view(B, Hq, T, L) * (1 / math.sqrt(d))
    score = score.masked_fill(~seen[:, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, -1, L) @ v).view(B, Hq, T, d) / torch.where(total == 0, 1.0, total)
    return o.to(torch.bfloat16), (top + torch.log(total))[..., 0]


def plain_compact(s):
    c = s["case"]
    if c["drafts"]:
        _write(s, "k", _quantise8 if c["cache"] == "e4m3" else None)
        _write(s, "v", _quantise8 if c["cache"] == "e4m3" else None)
    b, i = torch.nonzero(torch.arange(c["N"], device=DEV)[None] < s["keep_lens"][:, None], as_tuple=True)
    src, dst = s["keep"].long()[b, i], s["first"].long()[b] + i
    at = s["table"].long()
    page, slot, to_page, to_slot = at[b, src // c["bs"]], src % c["bs"], at[b, dst // c["bs"]], dst % c["bs"]

    def move(x):
        if x is not None:
            x[to_page, :, to_slot] = x[page, :, slot]

    move(s["k_cache"].view(torch.int16 if c["cache"] == "bf16" else torch.uint8))
    move(s["v_cache"].view(torch.int16 if c["cache"] == "bf16" else torch.uint8))
    move(s["k_scale"])
    move(s["v_scale"])
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def plain_branch(s):
    c = s["case"]
    bs, table, lens, refs = c["bs"], s["table"], s["lens"], s["refs"]
    B, per = table.shape
    col = torch.arange(per, device=DEV)
    # Back to the sequences alone: pages behind what is kept lose a holder.
    lens.copy_(torch.minimum(lens, s["back_to"]))
    gone = (col[None] >= ((lens + bs - 1) // bs)[:, None]) & (table >= 0)
    refs.index_add_(0, table.clamp_min(0).flatten().long(), -gone.flatten().int())
    table.masked_fill_(gone, -1)
    # Continuations hold their sequence's pages too.
    src, dst = s["src"].long(), s["dst"].long()
    rows = torch.where(col[None] < ((lens[src] + bs - 1) // bs)[:, None], table[src], -1)
    table[dst] = rows
    lens[dst] = lens[src]
    refs.index_add_(0, rows.clamp_min(0).flatten().long(), (rows >= 0).flatten().int())
    # A page for every token to come; who writes into a page that others hold too gets one of its own.
    n = s["new"]
    have, need = (lens + bs - 1) // bs, (lens + n + bs - 1) // bs
    last = torch.where((n > 0) & (lens % bs != 0), table.gather(1, (lens // bs).clamp(max=per - 1).long()[:, None])[:, 0], -1)
    before = ((last[None] == last[:, None]) & (s["all"][None] < s["all"][:, None])).sum(1)
    copies = (last >= 0) & (refs[last.clamp_min(0).long()] - before > 1)
    missing = (col[None] >= have[:, None]) & (col[None] < need[:, None]) & (table < 0) & (n > 0)[:, None]
    wanted = torch.cat((copies[:, None], missing), 1)
    free = torch.nonzero(refs == 0)[:, 0].int()
    short = ((wanted.sum(1).cumsum(0) > free.numel()) & (wanted.sum(1) > 0)).cumsum(0) > 0
    granted = ~short | (n == 0)
    wanted &= granted[:, None]
    b, j = torch.nonzero(wanted, as_tuple=True)
    got = torch.full((B, per + 1), -1, dtype=torch.int32, device=DEV)
    got[b, j] = free[: b.numel()]
    refs[free[: b.numel()].long()] = 1
    table.copy_(torch.where(got[:, 1:] >= 0, got[:, 1:], table))
    new = got[:, 0].contiguous()
    old = torch.where(new >= 0, last, -1).int()
    at = torch.nonzero(new >= 0)[:, 0]
    refs.index_add_(0, old[at].long(), torch.full_like(old[at], -1))
    table[at, (lens[at] // bs).long()] = new[at]
    of, to = old[at].long(), new[at].long()

    def copy(x):
        if x is not None:
            x[to] = x[of]

    copy(s["k_cache"].view(torch.int16 if c["cache"] == "bf16" else torch.uint8))
    copy(s["v_cache"].view(torch.int16 if c["cache"] == "bf16" else torch.uint8))
    copy(s["k_scale"])
    copy(s["v_scale"])
    return (table, lens, refs, granted.int(), old, new, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])


# ------------------------------------------------------------------------------------------------ in 64 bits


def exact(c, seed):
    s = prepare(c, seed)
    return {"axes": _exact_axes, "extend": _exact_extend, "tree": _exact_tree, "compact": _exact_compact,
            "branch": _exact_branch}[c["op"]](s)


def _exact_axes(s):
    c = s["case"]
    r, out = c["rot"], []
    where = torch.stack([s["positions"][int(a)] for a in s["axes"]], -1).double()
    theta = where * s["inv_freq"].to(DEV) * (-1 if c["backward"] else 1)
    turn = torch.polar(torch.ones_like(theta), theta)[:, None]
    for x in (s["q"].double(), s["k"].double()):
        pairs = x[..., :r].unflatten(-1, (r // 2, 2) if c["inter"] else (2, r // 2))
        if not c["inter"]:
            pairs = pairs.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z if c["inter"] else z.transpose(-1, -2)
        out.append(torch.cat((z.flatten(-2), x[..., r:]), -1))
    return tuple(out)


def _rows(s, name, b, n):
    """The n live rows of sequence b: [H, n, d] in float64."""
    at = torch.arange(n, device=DEV)
    bs = s["case"]["bs"]
    page, slot = s["table"][b].long()[at // bs], at % bs
    code = s[name + "_cache"][page, :, slot].int()
    nibble = torch.stack((code % 16, code // 16), -1).flatten(-2)
    e, m = nibble % 8 // 2, nibble % 2
    value = torch.where(e == 0, m * 0.5, (1 + m * 0.5) * torch.exp2(e.double() - 1)) * (1 - 2 * (nibble // 8))
    power = torch.exp2(s[name + "_scale"][page, :, slot].double() - 127)
    return (value * power.repeat_interleave(GROUP, -1)).transpose(0, 1)


def _nearest4(x):
    """Rows in four bits by search among the values a group can hold."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    g = x.double().unflatten(-1, (-1, GROUP))
    most = g.abs().amax(-1, keepdim=True)
    k = torch.ceil(torch.log2(most / 6)).clamp(-126, 125)
    k = torch.where(most > 6 * torch.exp2(k), k + 1, torch.where(most <= 6 * torch.exp2(k - 1), k - 1, k)).clamp(-126, 125)
    far = ((g.abs() * torch.exp2(-k))[..., None] - table).abs()
    # The nearest; of two as near, the even one.
    code = (far + (torch.arange(8, device=DEV) % 2) * 1e-9).argmin(-1)
    return (table[code] * torch.exp2(k) * g.sign()).flatten(-2)


def _exact_extend(s):
    c = s["case"]
    if c["B"] * c["Hkv"] * (c["start"] + c["N"]) > 1 << 19:
        return None
    out = []
    for name in ("k", "v"):
        y = torch.zeros((c["B"], c["Hkv"], c["start"] + c["N"], c["d"]), dtype=torch.float64, device=DEV)
        for b in range(c["B"]):
            first, n = int(s["start"][b]), int(s["new_lens"][b])
            y[b, :, :first] = _rows(s, name, b, first)
            y[b, :, first : first + n] = _nearest4(s[name][b, :, :n])
        out.append(y)
    return tuple(out)


def _exact_tree(s):
    c = s["case"]
    B, T, G = c["B"], c["T"], c["Hq"] // c["Hkv"]
    o = torch.zeros((B, c["Hq"], T, c["d"]), dtype=torch.float64, device=DEV)
    lse = torch.full((B, c["Hq"], T), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(B):
        n = int(s["lens"][b])
        m = T if s["draft_lens"] is None else int(s["draft_lens"][b])
        sees = torch.ones((m, n), dtype=torch.bool, device=DEV)
        sees[:, n - m :] = s["mask"][b, :m, :m] if s["mask"] is not None else torch.ones((m, m), dtype=torch.bool, device=DEV).tril()
        k, v = _rows(s, "k", b, n), _rows(s, "v", b, n)
        for h in range(c["Hq"]):
            z = s["q"][b, h, :m].double() @ k[h // G].T / math.sqrt(c["d"])
            z = torch.where(sees, z, -math.inf)
            lse[b, h, :m] = torch.logsumexp(z, -1)
            o[b, h, :m] = torch.softmax(z, -1) @ v[h // G]
    return o, lse


def _exact_compact(s):
    c = s["case"]
    out = []
    for name in ("k", "v"):
        cache = s[name + "_cache"].double()
        for b in range(c["B"]):
            at, m = s["table"][b].long(), int(s["keep_lens"][b])
            if c["drafts"]:
                rows = s[name][b].double()  # [H, N, d]
                if c["cache"] == "e4m3":
                    most = rows.abs().amax(-1, keepdim=True)
                    k = torch.ceil(torch.log2(most / 448)).clamp_min(-126)
                    k = torch.where(most > 448 * torch.exp2(k), k + 1, torch.where(most <= 448 * torch.exp2(k - 1), k - 1, k))
                    y = rows * torch.exp2(-k)
                    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0**-6))) - 3)
                    rows = torch.round(y / step) * step
                to = c["first"] + torch.arange(c["N"], device=DEV)
                cache[at[to // c["bs"]], :, to % c["bs"]] = rows.transpose(0, 1)
            of, to = s["keep"][b, :m].long(), c["first"] + torch.arange(m, device=DEV)
            cache[at[to // c["bs"]], :, to % c["bs"]] = cache[at[of // c["bs"]], :, of % c["bs"]]
        out.append(cache)
    return out[0], out[1], None, None


def _exact_branch(s):
    """One sequence after another, as a program on the host would do it: the caches that come out of it."""
    c = s["case"]
    bs, S, W = c["bs"], c["roots"], c["ways"]
    table, refs, lens, new = ([x.tolist() for x in (s["table"], s["refs"], s["lens"], s["new"])])
    for j in range(S * W):
        b = S * W + j // W
        used = -(-lens[b] // bs)
        table[j] = table[b][:used] + [-1] * (len(table[b]) - used)
        lens[j] = lens[b]
        for page in table[j][:used]:
            refs[page] += 1
    free = [page for page, n in enumerate(refs) if n == 0]
    pairs, at = [], 0
    for b in range(len(table)):
        last = lens[b] // bs if lens[b] % bs else -1
        own_page = last >= 0 and refs[table[b][last]] > 1
        missing = [j for j in range(-(-lens[b] // bs), -(-(lens[b] + new[b]) // bs)) if table[b][j] < 0]
        if at + own_page + len(missing) > len(free):
            break
        if own_page:
            pairs.append((table[b][last], free[at]))
            refs[table[b][last]] -= 1
            at += 1
        at += len(missing)
    k, v = s["k_cache"].double(), s["v_cache"].double()
    if pairs:
        of, to = (torch.tensor(x, device=DEV) for x in zip(*pairs))
        k[to], v[to] = k[of], v[of]
    return None, None, None, None, None, None, k, v, None, None
