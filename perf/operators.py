"""Cases of the operators around attention: rotary positions, writing and reading back a paged key/value cache
(bf16 or E4M3 codes with a power-of-two scale per row), and attention of drafted tokens over that cache.

``listed()`` names the cases, ``draw()`` gives more of the same ranges, ``prepare()`` makes what a program has in hand,
``run()`` is one pass (in plain torch operations, or through the library where ``own`` is true), ``exact()`` the same from
the definition in float64.
"""

import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------------ cases


def listed():
    return [
        # One new token of one sequence, the 28 query / 4 key heads of the grouped decode: launch latency.
        dict(name="rope_decode", op="rope", B=1, Hq=28, Hk=4, N=1, d=128, rot=128, dtype="bf16", inter=False,
             scaling="none", factor=1.0, far=8191, bnhd=False, backward=False),
        # Long positions in float32, an odd length, half of the head rotated, pairs side by side, scaled by parts.
        dict(name="rope_far_fp32", op="rope", B=3, Hq=8, Hk=8, N=1001, d=128, rot=64, dtype="fp32", inter=True,
             scaling="ramp", factor=8.0, far=1000003, bnhd=True, backward=False),
        # Gradients of q and k at the training shape.
        dict(name="rope_train_bwd", op="rope", B=2, Hq=16, Hk=16, N=8192, d=128, rot=128, dtype="bf16", inter=False,
             scaling="none", factor=1.0, far=0, bnhd=False, backward=True),
        # One new token for each of 64 sequences, quantised as it is written.
        dict(name="append_decode_e4m3", op="append", B=64, Hkv=4, N=1, d=128, bs=16, cache="e4m3", start=8191, ragged=False,
             bnhd=True),
        # Prompts of up to 8192 tokens written in one call, quantised; a padded batch.
        dict(name="append_prefill_e4m3", op="append", B=8, Hkv=4, N=8192, d=128, bs=16, cache="e4m3", start=0, ragged=True,
             bnhd=True),
        # A chunk of a prompt written as bf16 behind an odd prefix.
        dict(name="append_chunk_bf16", op="append", B=16, Hkv=8, N=513, d=64, bs=32, cache="bf16", start=259, ragged=True,
             bnhd=False),
        # A long quantised prefix read back for a prefill over it.
        dict(name="gather_e4m3", op="gather", B=4, Hkv=8, L=32768, d=128, bs=64, cache="e4m3", ragged=False),
        # Short ragged prefixes of a bf16 cache.
        dict(name="gather_bf16", op="gather", B=16, Hkv=4, L=2049, d=128, bs=16, cache="bf16", ragged=True),
        # A small tree on one short sequence: latency.
        dict(name="tree_short", op="tree", B=1, Hq=28, Hkv=4, T=5, L=777, d=128, bs=16, cache="e4m3", ragged=False,
             padded=False, mask=True, bnhd=True),
        # Eight drafted tokens over the paged decode's shape, bf16 cache with 16-key pages.
        dict(name="tree_draft8_bf16", op="tree", B=16, Hq=28, Hkv=4, T=8, L=8192, d=128, bs=16, cache="bf16", ragged=True,
             padded=True, mask=True, bnhd=True),
        # Single tokens of 64 sequences over a quantised cache.
        dict(name="tree_single_e4m3", op="tree", B=64, Hq=28, Hkv=4, T=1, L=8192, d=128, bs=64, cache="e4m3", ragged=True,
             padded=False, mask=False, bnhd=False),
        # Wide trees over long quantised contexts.
        dict(name="tree_wide_e4m3", op="tree", B=8, Hq=32, Hkv=8, T=64, L=32768, d=128, bs=64, cache="e4m3", ragged=False,
             padded=False, mask=True, bnhd=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "gather", "tree", "tree"])
    if op == "rope":
        d = rng.choice([64, 128])
        B, N = _log(rng, 1, 8), _log(rng, 1, 4096)
        Hk = rng.choice([1, 2, 4, 8, 16])
        return dict(op=op, B=B, Hq=Hk * rng.choice([1, 2, 4, 7]), Hk=Hk, N=N, d=d, rot=rng.choice([d, d // 2, d // 4]),
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), inter=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "base", "ramp"]), factor=float(rng.choice([2, 4, 8])),
                    far=_log(rng, 1, 2000000), bnhd=rng.random() < 0.5, backward=rng.random() < 0.4)
    if op == "append":
        return dict(op=op, B=_log(rng, 1, 64), Hkv=rng.choice([1, 2, 4, 8]), N=_log(rng, 1, 1024), d=rng.choice([64, 128]),
                    bs=rng.choice([16, 32, 64, 128]), cache=rng.choice(["bf16", "e4m3"]), start=rng.randrange(0, 3000),
                    ragged=rng.random() < 0.6, bnhd=rng.random() < 0.5)
    if op == "gather":
        return dict(op=op, B=_log(rng, 1, 32), Hkv=rng.choice([1, 2, 4, 8]), L=_log(rng, 1, 4096), d=rng.choice([64, 128]),
                    bs=rng.choice([16, 32, 64, 128]), cache=rng.choice(["bf16", "e4m3"]), ragged=rng.random() < 0.6)
    B, T, Hkv = _log(rng, 1, 24), _log(rng, 1, 64), rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 7, 8])
    most = min(16384, (1 << 29) // (B * T * Hq))  # no more score entries than the largest listed case has
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, T=T, L=max(T, _log(rng, 16, most)), d=rng.choice([64, 128]),
                bs=rng.choice([16, 32, 64, 128]), cache=rng.choice(["bf16", "e4m3"]), ragged=rng.random() < 0.6,
                padded=rng.random() < 0.4, mask=rng.random() < 0.7, bnhd=rng.random() < 0.5)


def _lens(n, B, ragged, least):
    """Length of each of B sequences: the longest has n; ragged ones spread over the upper half."""
    return [max(least, n - (b * 1237) % (n // 2 + 1)) if ragged else n for b in range(B)]


def work(c):
    esz = 4 if c.get("dtype") == "fp32" else 2
    if c["op"] == "rope":
        n = c["B"] * (c["Hq"] + c["Hk"]) * c["N"] * c["d"]
        return {"bytes": 2 * n * esz + c["B"] * c["N"] * 4, "flops": 3 * n * c["rot"] // c["d"]}
    row = 2 * c["d"] if c["cache"] == "bf16" else c["d"] + 1
    if c["op"] == "append":
        rows = 2 * c["Hkv"] * sum(_lens(c["N"], c["B"], c["ragged"], 1))
        return {"bytes": rows * (2 * c["d"] + row), "flops": 0 if c["cache"] == "bf16" else 2 * rows * c["d"]}
    if c["op"] == "gather":
        rows = 2 * c["Hkv"] * sum(_lens(c["L"], c["B"], c["ragged"], 1))
        full = 2 * c["Hkv"] * c["L"] * c["B"]
        return {"bytes": rows * row + full * 2 * c["d"], "flops": 0 if c["cache"] == "bf16" else rows * c["d"]}
    lens = _lens(c["L"], c["B"], c["ragged"], c["T"])
    qo = c["B"] * c["Hq"] * c["T"] * (4 * c["d"] + 4)
    return {"bytes": 2 * c["Hkv"] * sum(lens) * row + qo, "flops": 4 * c["Hq"] * c["T"] * sum(lens) * c["d"]}


# ------------------------------------------------------------------------------------------------ inputs


def _inv_freq(c):
    """Inverse frequencies in float64 and the magnitude, for the three usual ways to stretch a context."""
    r, base, f = c["rot"], 10000.0, c["factor"]
    i = torch.arange(r // 2, dtype=torch.float64)
    if c["scaling"] == "base":
        base *= f ** (r / (r - 2))
    w = base ** (-2 * i / r)
    if c["scaling"] == "linear":
        w = w / f
    if c["scaling"] == "ramp":
        keep = ((w * 4096 / (2 * math.pi) - 1) / 31).clamp(0, 1)
        return w * keep + w / f * (1 - keep), 0.1 * math.log(f) + 1
    return w, 1.0


def _quantise(x):
    """E4M3 codes and E8M0 scale bytes of the rows of x (last dimension): the smallest power of two that holds the row."""
    x = x.float()
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)
    k = torch.where(amax > 0, e - 9 + (m > 0.875).int(), -126).clamp(-126, 127)
    code = torch.ldexp(x, -k[..., None]).to(torch.float8_e4m3fn)
    return code, (k + 127).to(torch.uint8)


def _values(code, scale):
    """What codes and scale bytes stand for, in float32."""
    return torch.ldexp(code.float(), (scale.int() - 127)[..., None])


def _layout(x, bnhd):
    """[B,H,N,d] in its own layout, or as a view of [B,N,H,d]."""
    return x.transpose(1, 2).contiguous().transpose(1, 2) if bnhd else x


def _cache(c, g, most, lens):
    """A page pool for sequences of up to `most` keys, filled with normal rows, its pages in a random order."""
    per = -(-most // c["bs"])
    nb = c["B"] * per + 3
    s = {}
    for n in ("k", "v"):
        x = torch.randn((nb, c["Hkv"], c["bs"], c["d"]), generator=g, device=DEV, dtype=torch.bfloat16)
        if n == "k":  # keys have a few strong channels
            x[..., ::17] *= 3
        if c["cache"] == "e4m3":
            code, s[n + "_scale"] = _quantise(x * torch.exp2(torch.randint(-1, 2, x.shape[:-1], generator=g, device=DEV))[..., None])
            s[n + "_cache"] = code
        else:
            s[n + "_cache"], s[n + "_scale"] = x, None
    table = torch.randperm(nb, generator=g, device=DEV)[: c["B"] * per].view(c["B"], per).int()
    used = (torch.tensor(lens, device=DEV) + c["bs"] - 1) // c["bs"]
    s["table"] = torch.where(torch.arange(per, device=DEV)[None] < used[:, None], table, -1).int()
    return s


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    B, d = c["B"], c["d"]
    s = {"case": c}

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device=DEV, dtype=dtype)

    if c["op"] == "rope":
        dt = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16
        s["q"] = _layout(normal(B, c["Hq"], c["N"], d, dtype=dt), c["bnhd"])
        s["k"] = _layout(normal(B, c["Hk"], c["N"], d, dtype=dt), c["bnhd"])
        first = torch.randint(0, c["far"] + 1, (B, 1), generator=g, device=DEV)
        s["positions"] = (first + torch.arange(c["N"], device=DEV)[None]).int()
        s["inv_freq"], s["magnitude"] = _inv_freq(c)
        s["inv_freq_dev"] = s["inv_freq"].to(DEV)
        return s
    if c["op"] == "append":
        lens = _lens(c["N"], B, c["ragged"], 1)
        start = [max(0, c["start"] - 3 * b) for b in range(B)]
        s.update(_cache(c, g, c["start"] + c["N"], [a + n for a, n in zip(start, lens)]))
        s["k"], s["v"] = (_layout(normal(B, c["Hkv"], c["N"], d), c["bnhd"]) for _ in range(2))
        s["start"] = torch.tensor(start, device=DEV, dtype=torch.int32)
        s["new_lens"] = torch.tensor(lens, device=DEV, dtype=torch.int32)
        return s
    if c["op"] == "gather":
        lens = _lens(c["L"], B, c["ragged"], 1)
        s.update(_cache(c, g, c["L"], lens))
        s["lens"] = torch.tensor(lens, device=DEV, dtype=torch.int32)
        return s
    T = c["T"]
    lens = _lens(c["L"], B, c["ragged"], T)
    s.update(_cache(c, g, max(lens), lens))
    s["lens"] = torch.tensor(lens, device=DEV, dtype=torch.int32)
    s["q"] = _layout(normal(B, c["Hq"], T, d), c["bnhd"])
    s["draft_lens"] = None
    if c["padded"]:
        s["draft_lens"] = torch.tensor([max(1, T - b % 3) for b in range(B)], device=DEV, dtype=torch.int32)
    s["mask"] = None
    if c["mask"]:  # each token follows a random earlier one, or starts a branch of its own
        gc = torch.Generator().manual_seed(seed)
        mask = torch.zeros((B, T, T), dtype=torch.bool)
        for t in range(T):
            parent = torch.randint(-1, max(t, 1), (B,), generator=gc) if t else torch.full((B,), -1)
            mask[:, t] = mask[torch.arange(B), parent.clamp_min(0)] & (parent >= 0)[:, None]
            mask[:, t, t] = True
        s["mask"] = mask.to(DEV)
    # Scratch that a serving loop keeps: partial results of up to 64 splits.
    s["workspace"] = torch.empty(max(1 << 22, 64 * min(B * c["Hq"] * T, 4096) * (d + 2) * 4), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------------------------------------ one pass


def run(s):
    return globals()[("own_" if own else "plain_") + s["case"]["op"]](s)


def own_rope(s):
    from io_aware_exact_11_gb300 import fa
    c = s["case"]
    f = fa.rope_backward if c["backward"] else fa.rope
    return f(s["q"], s["k"], s["inv_freq"], positions=s["positions"], magnitude=s["magnitude"], interleaved=c["inter"])


def own_append(s):
    from io_aware_exact_11_gb300 import fa
    fa.cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["start"], new_lens=s["new_lens"],
                    k_scale=s["k_scale"], v_scale=s["v_scale"])
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def own_gather(s):
    from io_aware_exact_11_gb300 import fa
    return fa.cache_gather(s["k_cache"], s["v_cache"], s["table"], s["lens"], s["case"]["L"], k_scale=s["k_scale"],
                           v_scale=s["v_scale"])


def own_tree(s):
    from io_aware_exact_11_gb300 import fa
    return fa.decode_tree(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], tree_mask=s["mask"],
                          draft_lens=s["draft_lens"], k_scale=s["k_scale"], v_scale=s["v_scale"], workspace=s["workspace"])


def plain_rope(s):
    c = s["case"]
    r = c["rot"]
    angle = s["positions"].double()[..., None] * s["inv_freq_dev"]
    if c["backward"]:
        angle = -angle
    cos, sin = ((f(angle) * s["magnitude"]).float()[:, None] for f in (torch.cos, torch.sin))

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


def plain_append(s):
    c = s["case"]
    n = torch.arange(c["N"], device=DEV)
    b, n = torch.nonzero(n[None] < s["new_lens"][:, None], as_tuple=True)
    at = s["start"].long()[b] + n
    page, slot = s["table"].long()[b, at // c["bs"]], at % c["bs"]
    for name in ("k", "v"):
        x, cache, scale = s[name].transpose(1, 2)[b, n], s[name + "_cache"], s[name + "_scale"]
        if c["cache"] == "e4m3":
            code, k = _quantise(x)
            cache.view(torch.uint8)[page, :, slot] = code.view(torch.uint8)
            scale[page, :, slot] = k
        else:
            cache[page, :, slot] = x
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _paged(s, name, L):
    """The first L keys (or values) of each sequence in float32 [B,H,L,d]; rows past a sequence are some page's."""
    c = s["case"]
    pages = s["table"][:, : -(-L // c["bs"])].long().clamp_min(0)
    if s[name + "_scale"] is not None:
        x = _values(s[name + "_cache"].view(torch.uint8)[pages].view(torch.float8_e4m3fn), s[name + "_scale"][pages])
    else:
        x = s[name + "_cache"][pages].float()
    return x.transpose(1, 2).flatten(2, 3)[:, :, :L]


def plain_gather(s):
    c = s["case"]
    live = (torch.arange(c["L"], device=DEV)[None] < s["lens"][:, None])[:, None, :, None]
    return tuple((_paged(s, n, c["L"]) * live).to(torch.bfloat16) for n in ("k", "v"))


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


# ------------------------------------------------------------------------------------------------ in 64 bits


def exact(c, seed):
    s = prepare(c, seed)
    return {"rope": _exact_rope, "append": _exact_append, "gather": _exact_gather, "tree": _exact_tree}[c["op"]](s)


def _exact_rope(s):
    c = s["case"]
    r = c["rot"]
    angle = s["positions"].double()[:, None, :, None] * s["inv_freq"].to(DEV)
    turn = torch.polar(torch.full_like(angle, s["magnitude"]), -angle if c["backward"] else angle)
    out = []
    for x in (s["q"].double(), s["k"].double()):
        pairs = x[..., :r].unflatten(-1, (r // 2, 2) if c["inter"] else (2, r // 2))
        if not c["inter"]:
            pairs = pairs.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z if c["inter"] else z.transpose(-1, -2)
        out.append(torch.cat((z.flatten(-2), x[..., r:]), -1))
    return tuple(out)


def _exact_append(s):
    c = s["case"]
    out = []
    for name in ("k", "v"):
        cache, x = s[name + "_cache"].double(), s[name].double()
        for b in range(c["B"]):
            for n0 in range(0, n := int(s["new_lens"][b]), 4096):
                at = int(s["start"][b]) + torch.arange(n0, min(n, n0 + 4096), device=DEV)
                rows = x[b][:, n0 : min(n, n0 + 4096)].transpose(0, 1)
                if c["cache"] == "e4m3":
                    most = rows.abs().amax(-1, keepdim=True)
                    k = torch.ceil(torch.log2(most / E4M3_MAX)).clamp_min(-126)
                    k = torch.where(most > E4M3_MAX * torch.exp2(k), k + 1, torch.where(most <= E4M3_MAX * torch.exp2(k - 1), k - 1, k))
                    y = rows * torch.exp2(-k)
                    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0**-6))) - 3)
                    rows = torch.round(y / step) * step
                cache[s["table"][b].long()[at // c["bs"]], :, at % c["bs"]] = rows
        out.append(cache)
    return out[0], out[1], None, None


def _rows(s, name, b, n):
    """The n live rows of sequence b: [H, n, d] in float64."""
    c = s["case"]
    at = torch.arange(n, device=DEV)
    page, slot = s["table"][b].long()[at // c["bs"]], at % c["bs"]
    x = s[name + "_cache"].view(torch.uint8)[page, :, slot].view(s[name + "_cache"].dtype).double()
    if s[name + "_scale"] is not None:
        x = x * torch.exp2(s[name + "_scale"][page, :, slot].double() - 127)[..., None]
    return x.transpose(0, 1)


def _exact_gather(s):
    c = s["case"]
    out = []
    for name in ("k", "v"):
        y = torch.zeros((c["B"], c["Hkv"], c["L"], c["d"]), dtype=torch.float64, device=DEV)
        for b in range(c["B"]):
            n = int(s["lens"][b])
            y[b, :, :n] = _rows(s, name, b, n)
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
