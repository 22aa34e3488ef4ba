"""The operators around attention run together, as a serving loop and a training step use them, and the calls that a
program makes beside the plain one: captured and replayed, on other streams, two at once, with little workspace, into
buffers with neighbours, and beyond 32-bit offsets."""

import math

import numpy as np
import pytest

import oracle
from io_aware_exact_11_gb300 import fa
from oracle import serving
from tests.gpu_helpers import Guarded, rel_l2
from tests.serving_helpers import Paged, bf16, check_tree, np64, random_tree
from tests.test_gpu_parity import TOL_GRAD

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.lib()
    yield
    fa.device_status()


def _i32(a):
    import torch
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def _pools(nb, hkv, bs, d, cache):
    """Two empty pools (NaN everywhere) and, for E4M3, their scales."""
    import torch
    dt = torch.float8_e4m3fn if cache == "e4m3" else torch.bfloat16
    esz = 1 if cache == "e4m3" else 2
    raw = [torch.full((nb, hkv, bs, d * esz), 0x7F if cache == "e4m3" else 0xFF, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scale = [torch.full((nb, hkv, bs), 0xFF, dtype=torch.uint8, device="cuda") if cache == "e4m3" else None for _ in "kv"]
    return [r.view(dt) for r in raw], dict(k_scale=scale[0], v_scale=scale[1])


class _Cached:
    """What the oracle sees of a cache: the rows of each sequence as read back."""

    def __init__(self, k, v, lens, cache):
        self.hkv, self.cache = k.shape[1], cache
        self.k, self.v = ([np64(t[b, :, :n]) for b, n in enumerate(lens)] for t in (k, v))


def _rope_bound(x, pos, w):
    """Bound of a bf16 rotation: the rounding of the result and 13·2^-24 of |x₁| + |x₂| for the fp32 work."""
    ref = serving.rope(np64(x), pos, w)
    a = np.abs(np64(x))
    h = x.shape[-1] // 2
    return ref, 2.0 ** -8 * np.abs(ref) + 13 * 2.0 ** -24 * np.tile(a[..., :h] + a[..., h:], 2)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_serving_loop(cache):
    """Prompts of different lengths, then two rounds of drafted trees of which a path is accepted: rotate, append,
    attend, read the accepted path's rows back, write them behind the context, go on."""
    import torch
    rng = np.random.default_rng(21)
    B, Hq, hkv, d, bs, T = 3, 8, 2, 128, 16, 5
    w, _ = fa.rope_frequencies(d)
    (kc, vc), sc = _pools(B * 14, hkv, bs, d, cache)
    table = _i32(rng.permutation(B * 14).reshape(B, 14).tolist())
    have = [0, 0, 0]  # rows in the cache
    draw = lambda H, N: bf16(rng.standard_normal((B, H, N, d))).cuda()  # noqa: E731

    def step(N, new, depth, mask):
        """Append N tokens (new[b] of them real) behind what is there, with positions there + depth, and attend."""
        q, k, v = draw(Hq, N), draw(hkv, N), draw(hkv, N)
        pos = np.asarray(have)[:, None] + depth
        q2, k2 = fa.rope(q, k, w, positions=_i32(pos.tolist()))
        for x, y in ((q, q2), (k, k2)):
            ref, bound = _rope_bound(x, pos, w)
            assert np.all(np.abs(np64(y) - ref) <= bound)
        fa.cache_append(k2, v, kc, vc, table, _i32(have), new_lens=_i32(new), **sc)
        lens = [h + n for h, n in zip(have, new)]
        gk, gv = fa.cache_gather(kc, vc, table, _i32(lens), max(lens), **sc)
        for rows, got in ((k2, gk), (v, gv)):
            for b in range(B):
                x = np64(rows[b, :, : new[b]])
                if cache == "e4m3":
                    y, e = serving.quantise_rows(x)
                    x = y * 2.0 ** e[..., None]
                assert np.array_equal(np64(got[b, :, have[b] : lens[b]]), x) and not got[b, :, lens[b] :].any()
        o, lse = fa.decode_tree(q2, kc, vc, table, _i32(lens), draft_lens=_i32(new),
                                tree_mask=None if mask is None else torch.from_numpy(mask).cuda(), **sc)
        check_tree(o, lse, q2, _Cached(gk, gv, lens, cache), new, mask, d ** -0.5, heads=[0, 3, 7])
        return lens, gk, gv

    have, _, _ = step(40, [40, 1, 17], np.arange(40), None)
    for paths in ([[0, 1, 4], [0], [0, 2, 3]], [[0, 3], [0, 1, 2, 4], [0]]):
        mask = np.zeros((B, T, T), dtype=bool)
        for b, path in enumerate(paths):
            mask[b, np.arange(T), np.arange(T)] = True
            mask[b, :, 0] = True
            for i, t in enumerate(path):
                mask[b, t, path[:i]] = True
        lens, gk, gv = step(T, [T] * B, mask.sum(2) - 1, mask)
        # The accepted rows, in order, over the drafted ones.
        n = max(len(p) for p in paths)
        pick = torch.tensor([[h + p[min(i, len(p) - 1)] for i in range(n)] for h, p in zip(have, paths)], device="cuda")
        at = pick[:, None, :, None].expand(B, hkv, n, d)
        ak, av = gk.gather(2, at), gv.gather(2, at)
        new = [len(p) for p in paths]
        fa.cache_append(ak, av, kc, vc, table, _i32(have), new_lens=_i32(new), **sc)
        lens = [h + m for h, m in zip(have, new)]
        bk, bv = fa.cache_gather(kc, vc, table, _i32(lens), max(lens), **sc)
        for b in range(B):  # what came out of the cache goes back in as it was, E4M3 too
            assert torch.equal(bk[b, :, have[b] : lens[b]], ak[b, :, : new[b]])
            assert torch.equal(bv[b, :, have[b] : lens[b]], av[b, :, : new[b]])
        have = lens
    fa.device_status()


def test_training_step_with_rotary_positions():
    """rope → forward → backward → rope_backward against the formula's gradient and against differences.

    The rotation is orthogonal, so the gradients of the attention keep their relative error (TOL_GRAD) through it; the
    rotated gradients are rounded to bf16 once more (2^-8)."""
    rng = np.random.default_rng(22)
    B, H, N, d = 1, 2, 150, 128
    w, _ = fa.rope_frequencies(d)
    q, k, v, do = (bf16(rng.standard_normal((B, H, N, d))).cuda() for _ in range(4))
    q2, k2 = fa.rope(q, k, w)
    o, lse = fa.forward(q2, k2, v, causal=True)
    dq2, dk2, dv = fa.backward(q2, k2, v, o, lse, do, causal=True)
    dq, dk = fa.rope_backward(dq2, dk2, w)
    pos, sigma, tol = np.arange(N)[None], d ** -0.5, TOL_GRAD + 2.0 ** -8
    for h in range(H):
        a = [np64(t[0, h]) for t in (q2, k2, v, do)]
        want = oracle.attention_backward(*a, sigma, causal=True)
        for got, ref, x in ((dq, want[0], 0), (dk, want[1], 1)):
            ref = serving.rope(ref[None, None], pos, w, inverse=True)[0, 0]
            got = np64(got[0, h])
            assert rel_l2(got, ref) <= tol
            u = rng.standard_normal((N, d))
            turned, f = serving.rope(u[None, None], pos, w)[0, 0], []
            for eps in (1e-4, -1e-4):
                b = list(a)
                b[x] = b[x] + eps * turned
                f.append((oracle.attention_forward(*(t[None, None] for t in b[:3]), sigma, causal=True)[0][0, 0] * a[3]).sum())
            # 1e-6: what central differences leave of the third derivative at steps of 1e-4, and float64 rounding.
            slack = tol * np.linalg.norm(ref) * np.linalg.norm(u) + 1e-6 * np.linalg.norm(ref) * np.linalg.norm(u)
            assert abs((got * u).sum() - (f[0] - f[1]) / 2e-4) <= slack
        assert rel_l2(np64(dv[0, h]), want[2]) <= TOL_GRAD
    fa.device_status()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,T", [(1, 15), (1, 16), (1, 17), (1, 32), (1, 33), (2, 32), (1, 65), (4, 32), (3, 43), (1, 256),
                                  (8, 32), (2, 129), (4, 65), (128, 256)])
def test_row_counts_around_the_tiles(cache, d, Hq, T):
    """Rows of a pair (heads that share keys × drafted tokens) on both sides of every tile of rows."""
    rng = np.random.default_rng(T * Hq)
    lens = [T + 70, T]
    p = Paged(rng, lens, 1, d, 32, cache)
    q = bf16(rng.standard_normal((2, Hq, T, d))).cuda()
    o, lse = fa.decode_tree(q, *p.args(), **p.kw())
    check_tree(o, lse, q, p, [T, T], None, d ** -0.5, heads=sorted({0, Hq - 1}))


class _Step:
    """rope, append and tree attention of one decode step, on buffers of its own."""

    def __init__(self, seed, cache, lens, T=4, hkv=2, Hq=8, d=128, bs=32):
        import torch
        rng = np.random.default_rng(seed)
        self.w, _ = fa.rope_frequencies(d)
        self.p = Paged(rng, lens, hkv, d, bs, cache)
        new = lambda H: bf16(rng.standard_normal((len(lens), H, T, d))).cuda()  # noqa: E731
        self.q, self.k, self.v = new(Hq), new(hkv), new(hkv)
        self.q2, self.k2, self.o = torch.empty_like(self.q), torch.empty_like(self.k), torch.empty_like(self.q)
        self.lse = torch.empty((len(lens), Hq, T), device="cuda")
        self.start = self.p.seq_lens - T
        self.mask = torch.from_numpy(random_tree(rng, len(lens), T, 0.2)).cuda()
        self.gk, self.gv = (torch.empty((len(lens), hkv, max(lens), d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
        self.ws = torch.empty(fa.decode_tree_workspace_size(len(lens), Hq, hkv, T, d), dtype=torch.uint8, device="cuda")

    def __call__(self, stream=None):
        p, s = self.p, dict(stream=stream)
        fa.rope(self.q, self.k, self.w, positions=None, position0=77, out_q=self.q2, out_k=self.k2, **s)
        fa.cache_append(self.k2, self.v, p.k_cache, p.v_cache, p.table, self.start, **p.kw(), **s)
        fa.decode_tree(self.q2, *p.args(), tree_mask=self.mask, out=self.o, lse=self.lse, workspace=self.ws, **p.kw(), **s)
        fa.cache_gather(*p.args(), self.gk.shape[2], out_k=self.gk, out_v=self.gv, **p.kw(), **s)

    def results(self):
        import torch
        torch.cuda.synchronize()
        return [t.clone() for t in (self.q2, self.k2, self.o, self.lse, self.gk, self.gv)]

    def wipe(self):
        import torch
        for t in (self.q2, self.k2, self.o, self.lse, self.gk, self.gv):
            t.fill_(float("nan"))
        torch.cuda.synchronize()


def _same(a, b):
    import torch
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_captured_steps_follow_their_inputs(cache):
    """A step is captured once; lengths, tokens and masks then change in place and every replay agrees with a plain call."""
    import torch
    step = _Step(31, cache, [700, 130, 40])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for lens, token in (([700, 130, 40], 0), ([698, 4, 33], 1), ([0, 129, 36], 2)):
        step.q.copy_(bf16(np.random.default_rng(token).standard_normal(step.q.shape)).cuda())
        step.mask.copy_(torch.roll(step.mask, 1, 1))
        step.p.seq_lens.copy_(_i32(lens))
        step.start.copy_(_i32([max(n - 4, 0) for n in lens]))
        step.wipe()
        g.replay()
        got = step.results()
        step.wipe()
        step()
        assert _same(got, step.results()), lens
        assert torch.isfinite(got[2]).all()
    fa.device_status()


def test_two_graphs_share_a_workspace_in_turn():
    """Nothing that a call leaves in the workspace matters to the next."""
    import torch
    a, b = _Step(32, "bf16", [900, 300]), _Step(33, "e4m3", [64, 1200, 5, 700], Hq=16)
    want = []
    for s in (a, b):
        s()
        want.append(s.results())
    a.ws = b.ws = max(a.ws, b.ws, key=lambda t: t.numel())
    graphs = []
    for s in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s()
        graphs.append(g)
    for s in (a, b):
        s.wipe()
    for _ in range(3):
        for g in graphs:
            g.replay()
    assert _same(a.results(), want[0]) and _same(b.results(), want[1])


@pytest.mark.parametrize("wide", [False, True])
def test_two_calls_at_once_and_other_streams(wide):
    import torch
    T = 20 if wide else 4  # rows of a pair: 80 or 16
    steps = [_Step(41, "bf16", [3000, 200], T=T), _Step(42, "e4m3", [2500, 900, 33], T=T)]
    want = []
    for s in steps:
        s()
        want.append(s.results())
    streams = [torch.cuda.Stream() for _ in steps]
    for s in steps:
        s.wipe()
    for _ in range(20):
        for s, st in zip(steps, streams):
            s(stream=st)
    for s, r in zip(steps, want):
        assert _same(s.results(), r)
    with torch.cuda.stream(streams[0]):  # the current stream, its outputs allocated by the call
        o, lse = fa.decode_tree(steps[0].q2, *steps[0].p.args(), tree_mask=steps[0].mask, **steps[0].p.kw())
    torch.cuda.synchronize()
    assert torch.equal(o, want[0][2]) and torch.equal(lse, want[0][3])
    fa.device_status()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("T", [3, 24])
def test_little_workspace_means_fewer_parts(cache, T):
    import torch
    rng = np.random.default_rng(T)
    lens, Hq, d = [2000, 77, 900], 8, 128
    p = Paged(rng, lens, 2, d, 16, cache)
    q = bf16(rng.standard_normal((3, Hq, T, d))).cuda()
    for parts in (1, 2, 9, 0):
        n = fa.decode_tree_workspace_size(3, Hq, 2, T, d, parts)
        ws = Guarded((n,), torch.uint8)
        o, lse = fa.decode_tree(q, *p.args(), workspace=ws.t, **p.kw())
        assert ws.intact()
        check_tree(o, lse, q, p, [T] * 3, None, d ** -0.5, heads=[0, 7])
    with pytest.raises(fa.FAError, match="workspace"):
        fa.decode_tree(q, *p.args(), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"), **p.kw())


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("T", [1, 7, 40])
def test_writes_stay_inside_their_tensors(cache, T):
    import torch
    step = _Step(51, cache, [300, T, 129 + T], T=T)
    g = {n: Guarded(tuple(getattr(step, n).shape), getattr(step, n).dtype) for n in ("q2", "k2", "o", "lse", "gk", "gv", "ws")}
    p = step.p
    for n in ("k_cache", "v_cache", "k_scale", "v_scale"):
        t = getattr(p, n)
        if t is not None:
            g[n] = Guarded(tuple(t.shape), t.dtype)
            g[n].t.view(torch.uint8).copy_(t.view(torch.uint8))
    step()
    want = step.results()
    for n, x in g.items():
        setattr(p if n in ("k_cache", "v_cache", "k_scale", "v_scale") else step, n, x.t)
    step()
    assert all(x.intact() for x in g.values())
    assert _same(step.results(), want)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("T", [6, 40])
@pytest.mark.parametrize("value", [3e38, -3e38])
def test_a_drafted_key_that_nobody_sees_may_hold_the_largest_numbers(cache, T, value):
    import torch
    mask = np.tril(np.ones((1, T, T), dtype=bool))
    mask[:, :, 2] = False

    def huge(name, b, x):
        x[:, x.shape[1] - T + 2] = value
    for n in (T, 131, 128 + T):
        p = Paged(np.random.default_rng(n), [n], 2, 128, 16, cache, edit=huge)
        q = bf16(np.random.default_rng(9).standard_normal((1, 4, T, 128))).cuda()
        o, lse = fa.decode_tree(q, *p.args(), tree_mask=torch.from_numpy(mask).cuda(), max_parts=2, **p.kw())
        p.k[0][:, n - T + 2] = p.v[0][:, n - T + 2] = 0.0  # (what it holds is no part of the bounds either)
        check_tree(o, lse, q, p, [T], mask, 128 ** -0.5)
    fa.device_status()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [2, 6, 12, 40, 70])
@pytest.mark.parametrize("power", [12, 30, 90])
def test_value_rows_that_are_large_where_they_hardly_count(T, power, d):
    """E4M3: some value rows are larger than the others by 2^power, but rows either do not see them or give them next to
    no weight.  The bounds are relative to Σ p|v|, so the small rows have to come through."""
    import torch
    rng = np.random.default_rng(T + power)
    mask = random_tree(rng, 2, T)
    mask[:, 1:, 0] = False                       # drafted token 0 is seen by itself only
    n = [T + 300, T + 128]

    def far(name, b, x):
        if name == "v":
            x[:, n[b] - T] *= 2.0 ** power       # its value row
            x[:, [3, 90, 120]] *= 2.0 ** power  # and three of the context
            x[:, 40:60] *= 2.0 ** -20
            x[:, 61] = 0.0
        else:
            x[:, [3, 90, 120], 0] = -1000.0     # whose scores lie far below all others
    p = Paged(rng, n, 2, d, 32, "e4m3", edit=far)
    q = rng.standard_normal((2, 8, T, d))
    q[..., 0] = 8.0
    q = bf16(q).cuda()
    for parts in (1, 3):
        o, lse = fa.decode_tree(q, *p.args(), tree_mask=torch.from_numpy(mask).cuda(), max_parts=parts, **p.kw())
        fa.device_status()
        check_tree(o, lse, q, p, [T, T], mask, d ** -0.5)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("T", [2, 40])
def test_output_in_place_of_the_queries(cache, T):
    import torch
    p = Paged(np.random.default_rng(T), [900, 50, 0, 300], 2, 128, 32, cache)
    for parts in (1, 5):
        q = bf16(np.random.default_rng(1).standard_normal((4, 8, T, 128))).cuda()
        want, lse = fa.decode_tree(q, *p.args(), max_parts=parts, **p.kw())
        got, lse2 = fa.decode_tree(q, *p.args(), max_parts=parts, out=q, **p.kw())
        assert got is q and torch.equal(got, want) and torch.equal(lse2, lse)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_sequences_that_share_pages(cache):
    """A common prefix is stored once: two rows of the table name the same pages."""
    import torch
    rng = np.random.default_rng(61)
    p = Paged(rng, [96, 96], 2, 128, 16, cache)
    q = bf16(rng.standard_normal((2, 4, 1, 128))).cuda()
    table = p.table[:1].expand(2, -1).contiguous()
    o, lse = fa.decode_tree(q, p.k_cache, p.v_cache, table, p.seq_lens, **p.kw())
    p.k[1], p.v[1] = p.k[0], p.v[0]
    check_tree(o, lse, q, p, [1, 1], None, 128 ** -0.5)
    gk, gv = fa.cache_gather(p.k_cache, p.v_cache, table, p.seq_lens, 96, **p.kw())
    assert torch.equal(gk[0], gk[1]) and torch.equal(gv[0], gv[1])


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_pages_beyond_32_bit_offsets(cache):
    """The same sequences in a small pool and at the end of one with over 2^32 elements agree bit for bit."""
    import torch
    rng = np.random.default_rng(62)
    hkv, d, bs, lens, T = 8, 128, 128, [390, 130], 3
    nb = (1 << 32) // (hkv * d * bs) + 9
    dt, kw = (torch.float8_e4m3fn, {}) if cache == "e4m3" else (torch.bfloat16, {})
    far = [torch.empty((nb, hkv, bs, d), dtype=dt, device="cuda") for _ in "kv"]
    near = [torch.empty((9, hkv, bs, d), dtype=dt, device="cuda") for _ in "kv"]
    scales = lambda n: ({f"{x}_scale": torch.empty((n, hkv, bs), dtype=torch.uint8, device="cuda") for x in "kv"}  # noqa: E731
                        if cache == "e4m3" else kw)
    table = rng.permutation(9)[:8].reshape(2, 4).astype(np.int32)
    k, v = (bf16(rng.standard_normal((2, hkv, 390, d))).cuda() for _ in "kv")
    q = bf16(rng.standard_normal((2, 16, T, d))).cuda()
    got = []
    for pools, first in ((far, nb - 9), (near, 0)):
        t, sc = _i32((table + first).tolist()), scales(pools[0].shape[0])
        for x in sc.values():
            x[first:] = 127  # (scales of slots that nothing is written to are never used)
        fa.cache_append(k, v, *pools, t, _i32([0, 0]), new_lens=_i32(lens), **sc)
        got.append([*fa.decode_tree(q, *pools, t, _i32(lens), **sc), *fa.cache_gather(*pools, t, _i32(lens), 390, **sc)])
        torch.cuda.synchronize()
    assert _same(*got)
    del far, got
    torch.cuda.empty_cache()
    fa.device_status()


def test_numbers_beyond_int32_are_refused():
    import torch
    p = Paged(np.random.default_rng(3), [20], 1, 64, 16, "bf16")
    q = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16, device="cuda")
    for position0 in (1 << 31, -(1 << 31) - 1):
        with pytest.raises(ValueError, match="int32"):
            fa.rope(q, None, [1.0], position0=position0)
    with pytest.raises(ValueError, match="int32"):
        fa.decode_tree(q, *p.args(), max_parts=1 << 32)
    with pytest.raises(ValueError, match="int32"):
        fa.cache_gather(*p.args(), 1 << 32)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_rope_beyond_32_bit_offsets(dt):
    import torch
    t = torch.float32 if dt == "fp32" else torch.bfloat16
    rng = np.random.default_rng(63)
    x = torch.from_numpy(rng.standard_normal((2, 2, 3, 64)).astype(np.float32)).to(t).cuda()
    big = torch.empty(((1 << 32) + 4096,), dtype=t, device="cuda")
    far = big.as_strided((2, 2, 3, 64), (1 << 32, 1024, 64, 1))
    far.copy_(x)
    w, _ = fa.rope_frequencies(64)
    want, _ = fa.rope(x, None, w, position0=5)
    got, _ = fa.rope(far, None, w, position0=5, out_q=far)
    assert torch.equal(got, want)
    del big, far, got
    torch.cuda.empty_cache()


def test_largest_grids_of_small_work():
    """Many sequences of one token, up to the 65535 that the cache operators take (more is refused)."""
    import torch
    rng = np.random.default_rng(64)
    B, d, bs = 65535, 64, 16
    w, _ = fa.rope_frequencies(d)
    q, k, v = (bf16(rng.standard_normal((B, 1, 1, d))).cuda() for _ in range(3))
    (kc, vc), sc = _pools(B, 1, bs, d, "bf16")
    table = torch.randperm(B, device="cuda").int()[:, None]
    fa.cache_append(k, v, kc, vc, table, torch.zeros(B, dtype=torch.int32, device="cuda"))
    one = torch.ones(B, dtype=torch.int32, device="cuda")
    more = torch.cat([table, table[:1]])
    with pytest.raises(fa.FAError, match="65535"):
        fa.cache_append(q.new_zeros((B + 1, 1, 1, d)), q.new_zeros((B + 1, 1, 1, d)), kc, vc, more, more[:, 0] * 0)
    with pytest.raises(fa.FAError, match="65535"):
        fa.cache_gather(kc, vc, more, more[:, 0] * 0 + 1, 1)
    gk, gv = fa.cache_gather(kc, vc, table, one, 1)
    assert torch.equal(gk, k) and torch.equal(gv, v)
    o, lse = fa.decode_tree(q, kc, vc, table, one)
    assert torch.equal(o, v)  # one key: its weight is 1
    s = (np64(q) * np64(k)).sum(-1) / math.sqrt(d)
    assert np.abs(np64(lse) - s).max() <= 2.0 ** -16 * (np.abs(np64(q)) * np.abs(np64(k))).sum(-1).max() / math.sqrt(d)
    y, _ = fa.rope(q, None, w, position0=1)
    ref, bound = _rope_bound(q, np.ones((B, 1)), w)
    assert np.all(np.abs(np64(y) - ref) <= bound)
    fa.device_status()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
def test_large_calls_agree_with_small_ones(cache, d):
    """Large calls give each thread several tokens; the same tokens in small calls, bit for bit, and the same report of a
    page that is none."""
    import torch
    rng = np.random.default_rng(d)
    hkv, bs, N = 8, 16, 1801
    starts = [0, 5, 31, 14, 2, 1] * (1 if d == 128 else 2)
    B = len(starts)
    lens = [N, 1800, 0, 1, 1799, 777] * (B // 6)
    per = (31 + N + bs - 1) // bs
    table = _i32(rng.permutation(B * per).reshape(B, per).tolist())
    table[0, 50] = -1
    k, v = (torch.randn((B, hkv, N, d), device="cuda").bfloat16() for _ in "kv")
    k *= torch.exp2(torch.randint(-9, 9, (B, hkv, N, 1), device="cuda").float()).bfloat16()
    k[1, 0, 7, 3], v[1, 2, 100, 5], v[4, 3, 9] = float("nan"), float("inf"), -float("inf")
    assert B * N * hkv * d // 8 >= 4 * 152 * 2048  # where a call counts as large
    got = []
    for step in (N, 150):
        pools, sc = _pools(B * per, hkv, bs, d, cache)
        for x in sc.values():
            if x is not None:
                x.zero_()
        for n in range(0, N, step):
            part = slice(n, min(n + step, N))
            fa.cache_append(k[:, :, part], v[:, :, part], *pools, table, _i32([s + n for s in starts]),
                            new_lens=_i32([min(max(m - n, 0), part.stop - n) for m in lens]), **sc)
        with pytest.raises(fa.FAError, match="block-table"):
            fa.device_status()
        got.append([x.view(torch.uint8) for x in (*pools, *sc.values()) if x is not None])
    assert _same(*got)
    table[0, 50] = int(table[0, 49])
    ends = [s + m for s, m in zip(starts, lens)]
    n = max(ends)
    many = fa.cache_gather(*pools, table, _i32(ends), n, **sc)
    for b in range(B):
        one = fa.cache_gather(*pools, table[b : b + 1], _i32(ends[b : b + 1]), n, **sc)
        assert all(torch.equal(x[b : b + 1].view(torch.int16), y.view(torch.int16)) for x, y in zip(many, one))
    fa.device_status()


def test_first_calls_of_a_process_may_be_captured():
    """Nothing needs a call before the capture: a fresh process captures every kernel's first launch."""
    import os
    import subprocess
    import sys
    code = """
import torch
from io_aware_exact_11_gb300 import fa
torch.zeros(1, device="cuda")
table = torch.arange(64, dtype=torch.int32, device="cuda").view(2, 32)
lens = torch.full((2,), 300, dtype=torch.int32, device="cuda")
w, _ = fa.rope_frequencies(128)
q, k = (torch.ones((2, h, 40, 128), device="cuda", dtype=torch.bfloat16) for h in (8, 2))
for dt, sc in ((torch.bfloat16, {}), (torch.float8_e4m3fn, {n: torch.full((64, 2, 16), 127, dtype=torch.uint8, device="cuda")
                                                              for n in ("k_scale", "v_scale")})):
    kc, vc = (torch.zeros((64, 2, 16, 128), device="cuda").to(dt) for _ in "kv")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q2, k2 = fa.rope(q, k, w)
        fa.cache_append(k2, k, kc, vc, table, lens - 40, **sc)
        few, _ = fa.decode_tree(q2[:, :, :2], kc, vc, table, lens, **sc)
        many, _ = fa.decode_tree(q2, kc, vc, table, lens, **sc)
        gk, gv = fa.cache_gather(kc, vc, table, lens, 300, **sc)
    g.replay()
    torch.cuda.synchronize()
    fa.device_status()
    assert (gv[:, :, 260:] == 1).all() and torch.isfinite(many).all() and many.any() and few.any()
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=280,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
