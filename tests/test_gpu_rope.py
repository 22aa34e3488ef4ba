"""Rotary positions on the GPU against the float64 oracle, forward and backward."""

import numpy as np
import pytest

from io_aware_exact_11_gb300 import fa
from oracle import serving
from tests.serving_helpers import np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.lib()
    yield
    fa.device_status()


def _dt(name):
    import torch
    return torch.float32 if name == "fp32" else torch.bfloat16


def _check(y, x, pos, w, mag, inter, inverse):
    """One rounding to the output type, and fp32 work: the angle's fraction rounded to 24 bits (π·2^-24), sine and
    cosine within 2 ulp (4·2^-24), the magnitude twice, two products and a sum (5·2^-24): 13·2^-24 of μ(|x₁| + |x₂|)."""
    x, y = np64(x), np64(y)
    ref = serving.rope(x, pos, w, mag, inter, inverse)
    r = 2 * len(w)
    assert np.array_equal(y[..., r:], x[..., r:])
    a = np.abs(x[..., :r])
    pair = (np.repeat(a[..., 0::2] + a[..., 1::2], 2, -1) if inter
            else np.tile(a[..., : r // 2] + a[..., r // 2 :], 2))
    half_step = 2.0 ** -8 if _check.dt == "bf16" else 2.0 ** -24
    bound = half_step * np.abs(ref[..., :r]) + 13 * 2.0 ** -24 * mag * pair
    assert np.all(np.abs(y - ref)[..., :r] <= bound)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,Hq,Hk,N,d,rot", [
    (1, 28, 4, 1, 128, 128), (2, 3, 1, 7, 128, 64), (1, 1, 1, 333, 64, 64), (3, 5, 5, 33, 64, 20), (2, 2, 0, 5, 80, 2),
    (1, 4, 2, 9, 256, 256), (5, 2, 1, 3, 34, 34), (2, 16, 16, 513, 128, 128)])
def test_rope(dt, inter, B, Hq, Hk, N, d, rot):
    import torch
    _check.dt = dt
    g = torch.Generator().manual_seed(d * N + Hq)
    q, k = (torch.randn((B, H, N, d), generator=g).to(_dt(dt)).cuda() for H in (Hq, max(Hk, 1)))
    pos = torch.randint(-5, 1 << 20, (B, N), generator=g).int()
    w, mag = fa.rope_frequencies(rot, scaling="ramp", factor=4.0)
    for f, inverse in ((fa.rope, False), (fa.rope_backward, True)):
        yq, yk = f(q, k if Hk else None, w, positions=pos.cuda(), magnitude=mag, interleaved=inter)
        _check(yq, q, pos.numpy(), w, mag, inter, inverse)
        if Hk:
            _check(yk, k, pos.numpy(), w, mag, inter, inverse)
        else:
            assert yk is None


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_rope_far_positions(dt):
    import torch
    _check.dt = dt
    q = torch.randn((1, 2, 4, 64), generator=torch.Generator().manual_seed(1)).to(_dt(dt)).cuda()
    w, _ = fa.rope_frequencies(64)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 123456789, 0], dtype=torch.int32)
    y, _ = fa.rope(q, None, w, positions=pos.cuda())
    # float64's own products are off by up to 2^31·2^-53 radians here, far below the bound's 2^-24.
    _check(y, q, pos.numpy()[None], w, 1.0, False, False)
    y0, _ = fa.rope(q, None, w, position0=1000)
    _check(y0, q, 1000 + np.arange(4)[None], w, 1.0, False, False)
    y1, _ = fa.rope(q, None, w, positions=torch.arange(4, dtype=torch.int32).cuda(), position0=1000)
    assert torch.equal(y0, y1)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [128, 32, 36])
def test_rope_layouts_and_in_place_agree_bitwise(inter, rot):
    import torch
    g = torch.Generator().manual_seed(2)
    w, _ = fa.rope_frequencies(rot)
    qkv = torch.randn((2, 17, 12, 128), generator=g).to(torch.bfloat16).cuda()      # packed [B, N, Hq + 2 Hk, d]
    q, k = qkv[:, :, :8].transpose(1, 2), qkv[:, :, 8:10].transpose(1, 2)
    v = qkv[:, :, 10:].clone()
    yq, yk = fa.rope(q.contiguous(), k.contiguous(), w, interleaved=inter)
    sq, sk = fa.rope(q, k, w, interleaved=inter)
    assert torch.equal(sq, yq) and torch.equal(sk, yk)
    odd = torch.empty((2, 8, 17, 129), dtype=torch.bfloat16, device="cuda")[..., 1:]  # no 16-byte alignment
    odd.copy_(q)
    oq, _ = fa.rope(odd, None, w, interleaved=inter)
    assert torch.equal(oq, yq)
    fa.rope(odd, None, w, interleaved=inter, out_q=odd)
    assert torch.equal(odd, yq)
    wide = q.expand(2, 8, 17, 128)[:1].expand(2, 8, 17, 128)                          # a broadcast batch
    bq, _ = fa.rope(wide, None, w, interleaved=inter)
    assert torch.equal(bq[1], yq[0])
    fa.rope(q, k, w, interleaved=inter, out_q=q, out_k=k)                             # in place, inside the packed buffer
    assert torch.equal(q, yq) and torch.equal(k, yk) and torch.equal(qkv[:, :, 10:], v)


def test_rope_gradient_against_differences():
    import torch
    g = torch.Generator().manual_seed(3)
    x, gy, dx = (torch.randn((1, 2, 6, 64), generator=g).cuda() for _ in range(3))
    w, mag = fa.rope_frequencies(48, scaling="ramp", factor=2.0)
    kw = dict(position0=70000, magnitude=mag, interleaved=True)
    gx, _ = fa.rope_backward(gy, None, w, **kw)
    # the map is linear, so one difference with a whole step is the derivative: 2·768 terms, each a few 2^-24 off
    d = (fa.rope(x + dx, None, w, **kw)[0].double() - fa.rope(x, None, w, **kw)[0].double())
    lhs, rhs = (gy.double() * d).sum(), (gx.double() * dx.double()).sum()
    size = (gy.double().abs() * (x.double().abs() + dx.double().abs())).sum()
    assert abs(float(lhs - rhs)) <= 64 * 2.0 ** -24 * float(size)


def test_rope_refuses():
    import torch
    q = torch.zeros((2, 4, 8, 64), dtype=torch.bfloat16, device="cuda")
    w, _ = fa.rope_frequencies(64)
    for bad in (dict(k=q[:1]), dict(k=q[..., :32]), dict(out_q=q[:, :, :4]), dict(out_k=q),
                dict(positions=torch.zeros((3,), dtype=torch.int32, device="cuda")),
                dict(positions=torch.zeros((8,), dtype=torch.int32)), dict(out_q=q.float())):
        kw = dict(k=None)
        kw.update(bad)
        with pytest.raises(ValueError):
            fa.rope(q, kw.pop("k"), w, **kw)
    with pytest.raises(TypeError):
        fa.rope(q, q.float(), w)
    with pytest.raises(TypeError):
        fa.rope(q, None, w, positions=torch.zeros((8,), dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError):
        fa.rope(q.half(), None, w)
    with pytest.raises(ValueError, match="contiguous"):
        fa.rope(q.transpose(-1, -2).contiguous().transpose(-1, -2), None, w)
    with pytest.raises(fa.FAError):
        fa.rope(q, None, np.ones(33))
    with pytest.raises(fa.FAError):
        fa.rope(q, None, w, out_q=q[:1, :1, :1].expand(2, 4, 8, 64))
