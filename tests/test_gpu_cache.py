"""Writing and reading the paged cache on the GPU: every value and every untouched byte, exactly."""

import numpy as np
import pytest

from io_aware_exact_11_gb300 import fa
from oracle import serving
from tests.serving_helpers import Paged, codes_of, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.lib()
    yield
    fa.device_status()


def _pool(nb, hkv, bs, d, cache, fill=0x5A):
    import torch
    esz = 1 if cache == "e4m3" else 2
    raw = [torch.full((nb, hkv, bs, d * esz), fill, dtype=torch.uint8, device="cuda") for _ in range(2)]
    dt = torch.float8_e4m3fn if cache == "e4m3" else torch.bfloat16
    scales = [torch.full((nb, hkv, bs), fill, dtype=torch.uint8, device="cuda") for _ in range(2)]
    return [r.view(dt) for r in raw], scales if cache == "e4m3" else [None, None]


def _expect(pool, scale, x, table, start, lens, bs, cache):
    """The pool's bytes with rows x[b, :, n] at their slots (host arrays)."""
    import torch
    pool = pool.view(torch.uint8).cpu().numpy().copy()
    scale = None if scale is None else scale.cpu().numpy().copy()
    for b in range(x.shape[0]):
        for n in range(lens[b]):
            t = start[b] + n
            page, slot = table[b][t // bs], t % bs
            if cache == "e4m3":
                y, k = serving.quantise_rows(np64(x[b, :, n]))
                pool[page, :, slot] = codes_of(y)
                scale[page, :, slot] = k + 127
            else:
                pool[page, :, slot] = x[b, :, n].cpu().contiguous().view(torch.uint8).numpy()
    return pool, scale


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,hkv,N,d,bs,start,lens,strided", [
    (1, 1, 1, 128, 16, [0], None, False), (3, 4, 1, 128, 64, [15, 63, 64], [1, 0, 1], True),
    (2, 3, 37, 64, 16, [5, 31], [37, 20], False), (4, 2, 130, 128, 32, [0, 1, 100, 31], [130, 1, 0, 129], True),
    (2, 5, 70, 64, 128, [127, 3], None, True)])
def test_append(cache, B, hkv, N, d, bs, start, lens, strided):
    import torch
    rng = np.random.default_rng(N * d + B)
    per = -(-(max(start) + N) // bs)
    nb = B * per + 2
    table = rng.permutation(nb)[: B * per].reshape(B, per).astype(np.int32)
    kc, ks = _pool(nb, hkv, bs, d, cache)
    x = [torch.from_numpy((rng.standard_normal((B, hkv, N, d)) * np.exp2(rng.integers(-20, 20, (B, hkv, N, 1))))
                          .astype(np.float32)).to(torch.bfloat16).cuda() for _ in range(2)]
    x[0][0, 0, 0] = 0.0
    if N > 1:
        x[1][0, 0, 1, 3:6] = torch.tensor([float("inf"), float("nan"), -float("inf")])
        x[0][0, 0, 1] = torch.finfo(torch.bfloat16).max
        x[1][-1, -1, 0] = 2.0 ** -133
    if strided:
        x = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in x]
    n = lens if lens is not None else [N] * B
    want = [_expect(kc[i], ks[i], x[i], table, start, n, bs, cache) for i in range(2)]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    fa.cache_append(x[0], x[1], kc[0], kc[1], torch.from_numpy(table).cuda(), i32(start),
                    new_lens=None if lens is None else i32(lens), k_scale=ks[0], v_scale=ks[1])
    for i in range(2):
        got = kc[i].view(torch.uint8).cpu().numpy()
        if cache == "bf16":
            assert np.array_equal(got, want[i][0])
        else:
            # a NaN code's sign is not specified
            nan = (want[i][0] & 0x7F) == 0x7F
            assert np.array_equal((got & 0x7F) == 0x7F, nan) and np.array_equal(got[~nan], want[i][0][~nan])
            assert np.array_equal(ks[i].cpu().numpy(), want[i][1])
    fa.device_status()


def test_every_bf16_magnitude_quantises_as_the_oracle():
    """All 65536 bf16 values, in rows whose scale another element sets and in rows of their own."""
    import torch
    bits = np.arange(65536, dtype=np.uint16)
    x = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).view(1, 1, 512, 128).cuda()
    w = x.clone()
    w[..., 0] = torch.exp2(torch.arange(512, device="cuda") % 200 - 100.0).to(torch.bfloat16)
    (kc, vc), (ks, vs) = _pool(4, 1, 128, 128, "e4m3")
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    fa.cache_append(x, w, kc, vc, table, torch.zeros(1, dtype=torch.int32, device="cuda"), k_scale=ks, v_scale=vs)
    for src, code, scale in ((x, kc, ks), (w, vc, vs)):
        y, k = serving.quantise_rows(np64(src)[0, 0])
        assert np.array_equal(scale.cpu().numpy().reshape(-1), k + 127)
        got = np64(code.float()).reshape(512, 128)
        assert np.array_equal(got, y, equal_nan=True)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,n,hkv,d,bs", [([1], 1, 1, 128, 16), ([0, 5, 40], 40, 2, 64, 16), ([200, 129, 128], 131, 3, 128, 64),
                                             ([77, 300], 512, 4, 64, 128)])
def test_gather(cache, lens, n, hkv, d, bs):
    import torch
    p = Paged(np.random.default_rng(n), lens, hkv, d, bs, cache)
    strided = torch.full((len(lens), n, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    k, v = fa.cache_gather(*p.args(), n, **p.kw(), out_v=strided)
    assert v is strided
    for b, ln in enumerate(lens):
        m = min(n, ln)
        for got, rows in ((k, p.k), (v, p.v)):
            assert np.array_equal(np64(got[b, :, :m]), rows[b][:, :m])      # a code times its power of two is a bf16
            assert not np64(got[b, :, m:]).any()
    fa.device_status()


def test_append_then_gather_then_forward_is_prefill_over_a_cached_prefix():
    import torch
    import oracle
    rng = np.random.default_rng(11)
    B, H, n0, n1, d, bs = 2, 3, 100, 57, 128, 32
    k, v = (torch.from_numpy(rng.standard_normal((B, H, n0 + n1, d)).astype(np.float32)).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((B, H, n1, d)).astype(np.float32)).to(torch.bfloat16).cuda()
    (kc, vc), _ = _pool(16, H, bs, d, "bf16")
    table = torch.from_numpy(rng.permutation(16)[:10].reshape(2, 5).astype(np.int32)).cuda()
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    fa.cache_append(k[:, :, :n0], v[:, :, :n0], kc, vc, table, zero)
    fa.cache_append(k[:, :, n0:], v[:, :, n0:], kc, vc, table, zero + n0)
    gk, gv = fa.cache_gather(kc, vc, table, zero + n0 + n1, n0 + n1)
    assert torch.equal(gk, k) and torch.equal(gv, v)
    o, lse = fa.forward(q, gk, gv, causal=True)
    ro, rl = oracle.attention_forward(np64(q), np64(k), np64(v), d ** -0.5, causal=True)
    assert np.abs(np64(o) - ro).max() < 1e-2 and np.abs(np64(lse) - rl).max() < 1e-3


def test_bad_pages_and_positions_are_reported_and_write_nothing():
    import torch
    (kc, vc), (ks, vs) = _pool(6, 2, 16, 128, "e4m3")
    before = kc.view(torch.uint8).clone()
    x = torch.ones((2, 2, 20, 128), dtype=torch.bfloat16, device="cuda")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    for table, start, lens in (([[6, -1], [-7, 99]], [0, 0], None), ([[0, 1], [2, 3]], [40, -30], None),
                               ([[0, 1], [2, 3]], [0, 0], [21, -1])):
        fa.cache_append(x, x, kc, vc, i32(table), i32(start), new_lens=None if lens is None else i32(lens), k_scale=ks, v_scale=vs)
        with pytest.raises(fa.FAError) as ei:
            fa.device_status()
        assert ei.value.status == fa.FA_ERR_INVALID_ARG and "paged cache" in str(ei.value)
        assert torch.equal(kc.view(torch.uint8), before)
    for table, lens in (([[6, 0], [0, 0]], [20, 0]), ([[0, 1], [2, 3]], [33, -1])):
        k, _ = fa.cache_gather(kc, vc, i32(table), i32(lens), 16, k_scale=ks, v_scale=vs)
        assert not k.any()
        with pytest.raises(fa.FAError):
            fa.device_status()
    fa.device_status()


def test_cache_refuses():
    import torch
    (kc, vc), (ks, vs) = _pool(6, 2, 16, 64, "e4m3")
    x = torch.ones((2, 2, 20, 64), dtype=torch.bfloat16, device="cuda")
    table, start = torch.zeros((2, 2), dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    good = dict(k=x, v=x, k_cache=kc, v_cache=vc, block_table=table, start=start, k_scale=ks, v_scale=vs)
    for bad, err in ((dict(k_scale=None), ValueError), (dict(v_scale=vs[:5]), ValueError), (dict(k=x[:1]), ValueError),
                     (dict(v=x.float()), TypeError), (dict(k=x[:, :1]), ValueError), (dict(block_table=table.long()), TypeError),
                     (dict(start=start.long()), TypeError), (dict(new_lens=start[:1]), TypeError),
                     (dict(k_cache=kc.float()), TypeError), (dict(k_cache=kc.float(), v_cache=vc.float()), TypeError),
                     (dict(k=x.cpu()), ValueError), (dict(block_table=table.t()[:, :2].t()[:, ::2]), ValueError)):
        with pytest.raises(err):
            fa.cache_append(**{**good, **bad})
    with pytest.raises(ValueError):
        fa.cache_gather(kc, vc, table, start, 0, k_scale=ks, v_scale=vs)
    with pytest.raises(ValueError):
        fa.cache_gather(kc, vc, table, start, 4, k_scale=ks, v_scale=vs, out_k=x)
