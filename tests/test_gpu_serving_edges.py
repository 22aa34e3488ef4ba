"""The operators around attention at the edges of their ranges."""

import numpy as np
import pytest

from io_aware_exact_11_gb300 import fa
from tests.serving_helpers import Paged, bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.lib()
    fa.device_status()
    yield
    fa.device_status()


def _i32(a):
    import torch
    return torch.tensor(a, dtype=torch.int32, device="cuda")


# Drafted tokens with 4 query heads a key/value head: 4, 12, 32, 80 and 256 rows, on every kernel's side.
TOKENS = [1, 3, 8, 20, 64]


@pytest.mark.parametrize("cache,T", [("bf16", 2), ("bf16", 20), ("bf16", 64), ("e4m3", 2), ("e4m3", 20), ("e4m3", 64)])
def test_calls_behind_an_unread_timeout_end(cache, T):
    """A timeout that nobody has read makes the waits of later calls give up early, each for itself.  Such calls end, and
    the ones after the report are right.  (4 query heads a key/value head: 8, 80 and 256 rows.)"""
    import torch
    p = Paged(np.random.default_rng(T), [3000, 500, T], 2, 128, 16, cache)
    q = bf16(np.random.default_rng(1).standard_normal((3, 8, T, 128))).cuda()
    want, lse = fa.decode_tree(q, *p.args(), **p.kw())
    fa.device_status()
    fa.watchdog_selftest()
    for parts in (0, 1, 7):
        fa.decode_tree(q, *p.args(), max_parts=parts, **p.kw())
    with pytest.raises(fa.FAError) as ei:
        fa.device_status()
    assert ei.value.status == fa.FA_ERR_DEVICE_TIMEOUT
    got, lse2 = fa.decode_tree(q, *p.args(), **p.kw())
    assert torch.equal(got, want) and torch.equal(lse, lse2)
    fa.device_status()


def test_output_over_the_queries_needs_their_strides():
    import torch
    p = Paged(np.random.default_rng(7), [40, 50], 2, 64, 16, "bf16")
    q = torch.zeros((2, 4, 4, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fa.FAError, match="in place"):
        fa.decode_tree(q, *p.args(), out=q.transpose(1, 2))
    with pytest.raises(fa.FAError, match="in place"):
        fa.decode_tree(q.transpose(1, 2), *p.args(), out=q)
