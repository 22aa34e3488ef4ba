"""Queries whose scores come from elements far below their row's largest one, over a cache in four bits, on the GPU against
the float64 oracle, with bounds that leave the queries no error of their own."""

import math

import numpy as np
import pytest

from io_aware_exact_11_gb300 import fa
from oracle import serving
from tests.four_bit_helpers import Paged4
from tests.serving_helpers import bf16, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.lib()
    yield
    fa.device_status()


def bounds(q, k, v, scale):
    """Oracle's results and how far a call's may be off: ``serving_helpers.check_tree``'s bounds for weights in fp16, with
    scores that are off by their fp32 sums alone (2^-16 of the largest Σ|q||k|·σ)."""
    ro, rl, p = serving.tree_attention(q, k, v, len(q), None, scale)
    es = scale * 2.0 ** -16 * (np.abs(q) @ np.abs(k).T).max(1)
    off = 2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 2 * es[:, None] + 2.0 ** -18) * (p @ np.abs(v))
    return ro, rl, off + np.minimum(p, 2.0 ** -28 * p.max(1, keepdims=True)) @ np.abs(v), es + 2.0 ** -18 * (1 + np.abs(rl))


def small_queries(rng, shape, below):
    """Rows whose first 32 elements hold the largest, 1, and the others ±2^-3 to ±4 times 2^-below."""
    q = rng.choice([-1, 1], shape) * np.clip(np.abs(rng.standard_normal(shape)), 2.0 ** -3, 4) * 2.0 ** -below
    q[..., :32] = 0
    q[..., 5] = 1
    return np64(bf16(q))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,below", [(2, 5), (2, 10), (8, 10), (16, 10), (17, 20), (24, 5), (24, 26), (64, 20), (80, 26), (128, 20)])
def test_small_elements_of_a_query_decide(G, below, d):
    """Two tokens, so 2 G rows: up to 32 take q as two E4M3 terms, exact down to 2^-14 of the largest element (here 2^-13),
    more take it as fp16, exact down to 2^-31 of it (here 2^-29).  Keys are zero where that element is, and as much larger
    elsewhere."""
    def keys(name, b, x):
        if name == "k":
            x *= 2.0 ** below
            x[..., :32] = 0
    rng = np.random.default_rng(G + below)
    p = Paged4(rng, [300, 129], 2, d, 16, edit=keys)
    q = small_queries(rng, (2, 2 * G, 2, d), below)
    scale = 1 / math.sqrt(d)
    o, lse = (np64(x) for x in fa.decode_tree(bf16(q).cuda(), *p.args(), **p.kw()))
    fa.device_status()
    for b in range(2):
        for h in sorted({0, G - 1, G, 2 * G - 1}):
            ro, rl, off, off_lse = bounds(q[b, h], p.k[b][h // G], p.v[b][h // G], scale)
            assert np.all(np.abs(lse[b, h] - rl) <= off_lse), (b, h)
            assert np.all(np.abs(o[b, h] - ro) <= off), (b, h)
