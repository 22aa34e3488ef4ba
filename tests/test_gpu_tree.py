"""Attention of drafted tokens over a paged cache against the float64 oracle."""

import math

import numpy as np
import pytest

from io_aware_exact_11_gb300 import fa
from tests.serving_helpers import Paged, bf16, check_tree, np64, random_tree

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


def _mask(m):
    import torch
    return None if m is None else torch.from_numpy(m).cuda()


def _run(seed, lens, Hq, hkv, T, d, bs, cache, mask=None, drafts=None, parts=0, heads=None, q_scale=1.0, edit=None, **kw):
    rng = np.random.default_rng(seed)
    p = Paged(rng, lens, hkv, d, bs, cache, edit=edit)
    q = bf16(rng.standard_normal((len(lens), Hq, T, d)) * q_scale).cuda()
    if isinstance(mask, str):
        mask = random_tree(rng, len(lens), T, empty={"tree": 0.0, "holes": 0.4}[mask])
    scale = kw.pop("scale", 1 / math.sqrt(d))
    o, lse = fa.decode_tree(q, *p.args(), tree_mask=_mask(mask), draft_lens=None if drafts is None else _i32(drafts),
                            max_parts=parts, scale=scale, **p.kw(), **kw)
    fa.device_status()
    real = drafts if drafts is not None else [T if n else 0 for n in lens]
    check_tree(o, lse, q, p, real, mask, scale, heads)
    return o, lse, q, p


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,Hq,hkv,T,bs,mask,drafts", [
    ([1], 1, 1, 1, 16, None, None),
    ([5, 128, 129, 127], 7, 1, 1, 16, None, None),
    ([130, 64, 300], 28, 4, 5, 16, "tree", None),
    ([8, 9, 260], 4, 2, 8, 64, "holes", None),
    ([33, 0, 700], 8, 2, 3, 32, "tree", None),
    ([40, 500, 3, 0], 8, 1, 12, 128, "tree", [12, 3, 3, 0]),
    ([100, 257], 16, 2, 64, 64, "tree", [64, 50]),
    ([300], 2, 1, 130, 16, "holes", None),
    ([256], 1, 1, 256, 128, None, None)])
def test_tree(cache, d, lens, Hq, hkv, T, bs, mask, drafts):
    for parts in (0, 1, 3):
        _run(T * d, lens, Hq, hkv, T, d, bs, cache, mask, drafts, parts, heads=sorted({0, Hq // 2, Hq - 1}))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("parts", [1, 2, 7, 64, 256])
def test_parts_of_a_long_sequence(cache, parts):
    _run(5, [4000, 1, 2047], 8, 2, 2, 128, 16, cache, None, [2, 1, 2], parts, heads=[0, 7])


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_one_group_of_128_heads_and_many_row_tiles(cache):
    _run(6, [190], 128, 1, 3, 128, 64, cache, "tree", heads=[0, 1, 63, 64, 127])


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_large_scores_and_rising_maxima(cache):
    """Scores with a standard deviation of about 20 whose maximum keeps moving along the keys."""
    def rising(name, b, x):
        if name == "k":
            x *= np.linspace(0.1, 3, x.shape[1])[None, :, None]
    _run(7, [1500, 1000], 4, 2, 4, 128, 32, cache, "tree", parts=2, q_scale=8.0, edit=rising)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_value_rows_of_very_different_size(cache):
    def spread(name, b, x):
        if name == "v":
            x *= np.exp2((np.arange(x.shape[1]) * 37 % 41) - 20.0)[None, :, None]
            x[:, 3] = 0.0
    _run(8, [700, 513], 4, 2, 3, 128, 16, cache, "tree", parts=3, edit=spread)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_what_unseen_drafted_keys_hold_does_not_matter(cache, value):
    """Drafted token 2's key and value hold NaN or infinities; only rows that see it may show it."""
    T = 6
    mask = np.tril(np.ones((1, T, T), dtype=bool))
    mask[:, :, 2] = False
    mask[0, 4, 2] = True
    mask[0, 5] = False

    def poison(name, b, x):
        x[:, x.shape[1] - T + 2] = value
    for n in (T, 131, 128 + T):
        rng = np.random.default_rng(9)
        p = Paged(rng, [n], 1, 128, 16, cache, edit=poison)
        q = bf16(rng.standard_normal((1, 2, T, 128))).cuda()
        o, lse = (np64(x) for x in fa.decode_tree(q, *p.args(), tree_mask=_mask(mask), max_parts=2, **p.kw()))
        assert np.isnan(o[:, :, 4]).all() and not np.isfinite(lse[:, :, 4]).any()
        mask2 = mask.copy()
        mask2[0, 4, 2] = False
        clean = Paged(np.random.default_rng(9), [n], 1, 128, 16, cache,
                      edit=lambda name, b, x: x.__setitem__((slice(None), x.shape[1] - T + 2), 0.0))
        ro, rl = (np64(x) for x in fa.decode_tree(q, *clean.args(), tree_mask=_mask(mask2), max_parts=2, **clean.kw()))
        rows = [0, 1, 2, 3, 5]
        assert np.array_equal(o[:, :, rows], ro[:, :, rows]) and np.array_equal(lse[:, :, rows], rl[:, :, rows])


def test_an_infinite_value_shows_in_its_columns_only():
    def poison(name, b, x):
        if name == "v":
            x[:, -1, 5] = np.inf
    o, _, _, _ = _run(10, [140], 2, 1, 2, 64, 16, "bf16", np.array([[[1, 0], [0, 1]]], dtype=bool), edit=poison)
    o = np64(o)
    assert np.isposinf(o[:, :, 1, 5]).all() and np.isfinite(np.delete(o, 5, 3)).all() and np.isfinite(o[:, :, 0]).all()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_what_is_not_finite_in_the_context_shows_in_every_row(cache):
    def poison(name, b, x):
        if b == 0:
            x[:, 70, 9 if name == "v" else slice(None)] = np.nan if name == "v" else x[:, 70]
        elif name == "k":
            x[:, 3, 7] = np.nan
    rng = np.random.default_rng(17)
    p = Paged(rng, [300, 200, 250], 2, 128, 16, cache, edit=lambda n, b, x: poison(n, b, x) if b < 2 else None)
    q = bf16(rng.standard_normal((3, 8, 3, 128))).cuda()
    o, lse = (np64(t) for t in fa.decode_tree(q, *p.args(), **p.kw()))
    assert np.isnan(o[0, :, :, 9]).all() and np.isfinite(np.delete(o[0], 9, 2)).all() and np.isfinite(lse[0]).all()
    assert np.isnan(o[1]).all() and np.isnan(lse[1]).all()
    assert np.isfinite(o[2]).all() and np.isfinite(lse[2]).all()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_layouts_masks_and_buffers_agree_bitwise(cache):
    import torch
    T, Hq, lens = 6, 8, [150, 77, 300]
    rng = np.random.default_rng(12)
    mask = random_tree(rng, 1, T)[0]
    o, lse, q, p = _run(13, lens, Hq, 2, T, 128, 32, cache, np.stack([mask] * 3), parts=3)
    kw = dict(max_parts=3, **p.kw())
    qs = q.transpose(1, 2).contiguous().transpose(1, 2)
    out = torch.full((3, T, Hq, 128), 9.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    a, b = fa.decode_tree(qs, *p.args(), tree_mask=_mask(mask), out=out, **kw)          # one mask for the batch
    assert a is out and torch.equal(a, o) and torch.equal(b, lse)
    a, b = fa.decode_tree(q, *p.args(), tree_mask=_mask(mask).to(torch.uint8) * 7, **kw)
    assert torch.equal(a, o) and torch.equal(b, lse)
    ws = torch.full((fa.decode_tree_workspace_size(3, Hq, 2, T, 128, 3),), 0xFF, dtype=torch.uint8, device="cuda")
    a, b = fa.decode_tree(q, *p.args(), tree_mask=_mask(mask), workspace=ws, **kw)      # NaN bits in the workspace
    assert torch.equal(a, o) and torch.equal(b, lse)
    if cache == "e4m3":
        a, b = fa.decode_tree(q, p.k_cache.view(torch.uint8), p.v_cache.view(torch.uint8), p.table, p.seq_lens,
                              tree_mask=_mask(mask), **kw)
        assert torch.equal(a, o) and torch.equal(b, lse)


def test_chain_of_one_is_the_paged_decode():
    import torch
    o, lse, q, p = _run(14, [700, 33, 1], 28, 4, 1, 128, 16, "bf16", parts=2)
    ro, rl = fa.decode_paged(q, *p.args(), n_splits=2)
    # two roundings of the same number to bf16, and both kernels' bf16 probabilities: 2·2^-8 relative each
    assert (o.float() - ro.float()).abs().max() <= 4 * 2.0 ** -8 * ro.float().abs().max()
    assert (lse[..., 0] - rl).abs().max() < 1e-4
    assert torch.isfinite(lse).all()


def test_bad_lengths_and_pages_are_reported():
    import torch
    rng = np.random.default_rng(15)
    p = Paged(rng, [40, 50], 1, 64, 16, "bf16")
    q = bf16(rng.standard_normal((2, 2, 4, 64))).cuda()
    good, _ = fa.decode_tree(q, *p.args())
    for lens, drafts in (([40, 3], None), ([40, 1000], None), ([40, -1], None), ([40, 50], [4, 5]), ([40, 50], [4, -1]),
                         ([40, 2], [4, 3])):
        o, lse = fa.decode_tree(q, p.k_cache, p.v_cache, p.table, _i32(lens), draft_lens=None if drafts is None else _i32(drafts))
        with pytest.raises(fa.FAError) as ei:
            fa.device_status()
        assert ei.value.status == fa.FA_ERR_INVALID_ARG and "decode tree" in str(ei.value)
        assert torch.equal(o[0], good[0]) and not o[1].any() and torch.isneginf(lse[1]).all()
    for page in (-1, p.k_cache.shape[0]):
        table = p.table.clone()
        table[1, 2] = page
        o, _ = fa.decode_tree(q, p.k_cache, p.v_cache, table, p.seq_lens)
        with pytest.raises(fa.FAError, match="block-table"):
            fa.device_status()
        assert torch.equal(o[0], good[0])
    fa.device_status()


def test_decode_tree_refuses():
    import torch
    p = Paged(np.random.default_rng(16), [40, 50], 2, 64, 16, "e4m3")
    q = torch.zeros((2, 4, 3, 64), dtype=torch.bfloat16, device="cuda")
    one = torch.ones((3, 3), dtype=torch.bool, device="cuda")
    good = dict(q=q, k_cache=p.k_cache, v_cache=p.v_cache, block_table=p.table, seq_lens=p.seq_lens, **p.kw())
    for bad, err in ((dict(q=q.float()), TypeError), (dict(q=q[:1]), ValueError), (dict(q=q[..., :32]), ValueError),
                     (dict(k_scale=None), ValueError), (dict(seq_lens=p.seq_lens.long()), TypeError),
                     (dict(draft_lens=p.seq_lens[:1]), TypeError), (dict(tree_mask=one.float()), TypeError),
                     (dict(tree_mask=one[:2]), ValueError), (dict(tree_mask=one.t().contiguous().t()), ValueError),
                     (dict(out=q.float()), ValueError), (dict(lse=torch.empty((2, 4), device="cuda")), ValueError),
                     (dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), fa.FAError),
                     (dict(q=q[:, :3]), fa.FAError), (dict(max_parts=-1), fa.FAError), (dict(max_parts=5000), fa.FAError),
                     (dict(scale=-1.0), fa.FAError), (dict(q=q.cpu()), ValueError),
                     (dict(k_cache=p.k_cache[:, :, ::2]), ValueError)):
        with pytest.raises(err):
            fa.decode_tree(**{**good, **bad})
