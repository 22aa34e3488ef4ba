"""Rotary positions with several axes on the GPU against the float64 oracle, forward and backward."""

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


def _check(y, x, pos, axes, w, mag, inter, inverse, dt):
    """One rounding to the output type, and fp32 work: the angle's fraction rounded to 24 bits (π·2^-24), sine and
    cosine within 2 ulp (4·2^-24), the magnitude twice, two products and a sum (5·2^-24): 13·2^-24 of μ(|x₁| + |x₂|)."""
    x, y = np64(x), np64(y)
    ref = serving.rope_axes(x, pos, axes, w, mag, inter, inverse)
    r = 2 * len(w)
    assert np.array_equal(y[..., r:], x[..., r:])
    a = np.abs(x[..., :r])
    pair = np.repeat(a[..., 0::2] + a[..., 1::2], 2, -1) if inter else np.tile(a[..., : r // 2] + a[..., r // 2 :], 2)
    half_step = 2.0 ** -8 if dt == "bf16" else 2.0 ** -24
    bound = half_step * np.abs(ref[..., :r]) + 13 * 2.0 ** -24 * mag * pair
    assert np.all(np.abs(y - ref)[..., :r] <= bound)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("A,B,Hq,Hk,N,d,rot", [
    (3, 1, 28, 4, 1, 128, 128), (3, 2, 3, 1, 7, 128, 64), (1, 1, 1, 1, 333, 64, 64), (2, 3, 5, 5, 33, 64, 20),
    (4, 2, 2, 0, 5, 80, 2), (4, 1, 4, 2, 9, 256, 256), (3, 5, 2, 1, 3, 34, 34), (3, 2, 16, 16, 513, 128, 128)])
def test_axes(dt, inter, A, B, Hq, Hk, N, d, rot):
    import torch
    g = torch.Generator().manual_seed(d * N + Hq)
    q, k = (torch.randn((B, H, N, d), generator=g).to(_dt(dt)).cuda() for H in (Hq, max(Hk, 1)))
    pos = torch.randint(-5, 1 << 20, (A, B, N), generator=g).int()
    axes = torch.randint(0, A, (rot // 2,), generator=g).int()
    w, mag = fa.rope_frequencies(rot, scaling="ramp", factor=4.0)
    for f, inverse in ((fa.rope_axes, False), (fa.rope_axes_backward, True)):
        for positions, p in ((pos.cuda(), pos.numpy()), (pos[:, 0].contiguous().cuda(), np.repeat(pos[:, :1].numpy(), B, 1))):
            yq, yk = f(q, k if Hk else None, w, axes, positions, magnitude=mag, interleaved=inter)
            _check(yq, q, p, axes, w, mag, inter, inverse, dt)
            if Hk:
                _check(yk, k, p, axes, w, mag, inter, inverse, dt)
            else:
                assert yk is None


def test_the_same_position_on_all_axes_is_the_plain_rotation():
    import torch
    q, k = (torch.randn((2, H, 65, 128), device="cuda").bfloat16() for H in (4, 2))
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (2, 65), device="cuda").int()
    w, _ = fa.rope_frequencies(128)
    for f, g in ((fa.rope_axes, fa.rope), (fa.rope_axes_backward, fa.rope_backward)):
        got = f(q, k, w, np.arange(64) % 3, pos[None].expand(3, 2, 65))
        want = g(q, k, w, positions=pos)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradient_is_the_slope():
    """<dy, f(x + h e) − f(x − h e)> / 2h against the gradient; the map is linear in x, so differences are exact but for
    fp32's roundings (2^-24 of values of size up to 8 in each, twice, over 2h = 2: below 2^-20 per element of dy)."""
    import torch
    g = torch.Generator().manual_seed(5)
    x, dy = (torch.randn((1, 2, 6, 32), generator=g).clamp(-3, 3).cuda() for _ in range(2))
    pos = torch.randint(0, 4000, (3, 6), generator=g).int().cuda()
    axes, w = np.arange(12) % 3, fa.rope_frequencies(24)[0]
    dx, _ = fa.rope_axes_backward(dy, None, w, axes, pos)
    for _ in range(20):
        e = torch.zeros_like(x)
        at = tuple(int(torch.randint(0, s, (1,), generator=g)) for s in x.shape)
        e[at] = 1.0
        up, down = (fa.rope_axes(x + h * e, None, w, axes, pos)[0].double() for h in (1.0, -1.0))
        slope = float(((up - down) / 2 * dy.double()).sum())
        assert abs(slope - float(dx[at])) <= 2.0 ** -20 * float(dy.abs().max()) * 4


def test_strides_in_place_and_refusals():
    import torch
    q = torch.randn((2, 9, 4, 128), device="cuda").bfloat16().transpose(1, 2)  # [B, H, N, d] over [B, N, H, d]
    k = torch.randn((2, 3, 9, 256), device="cuda").bfloat16()[..., 64:192]
    pos = torch.randint(0, 99, (3, 2, 9), device="cuda").int()
    w, axes = fa.rope_frequencies(64)[0], torch.arange(32).int() % 3
    want = fa.rope_axes(q.contiguous(), k.contiguous(), w, axes, pos)
    got = fa.rope_axes(q, k, w, axes, pos.transpose(0, 1).contiguous().transpose(0, 1))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    fa.rope_axes(q, k, w, axes, pos, out_q=q, out_k=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    q2, k2 = (x.clone() for x in want)
    for same in (axes.tolist(), axes.long().numpy(), axes.numpy().astype(np.uint8)):
        again = fa.rope_axes(q2, k2, w, same, pos)
        assert all(torch.equal(a, b) for a, b in zip(again, fa.rope_axes(q2, k2, w, axes, pos)))
    for bad in ([0.5] * 32, axes.double().numpy(), [1 << 32] * 32, np.full(32, 1 << 32), [-1] * 32):
        with pytest.raises(ValueError):
            fa.rope_axes(q, k, w, bad, pos)
    with pytest.raises(TypeError):
        fa.rope_axes(q, k, w, axes, None)
    with pytest.raises(TypeError):
        fa.rope_axes(q, k, w, axes, pos.long())
    with pytest.raises(ValueError):
        fa.rope_axes(q, k, w, axes[:-1], pos)
    with pytest.raises(ValueError):
        fa.rope_axes(q, k, w, axes, pos[:, :, :-1])
    with pytest.raises(ValueError):
        fa.rope_axes(q, k, w, axes, pos[0, 0])
    with pytest.raises(fa.FAError):
        fa.rope_axes(q, k, w, axes, pos[:2])  # axis 2 has no positions
    with pytest.raises(fa.FAError):
        fa.rope_axes(q, k, w, axes, pos[:1].expand(5, 2, 9))
