"""Cross attention on the GPU where a result could be lost or stale: expanded tables."""
import math

import pytest
import torch

from streaming_sinkhorn_solver_gb300 import binding as fs
from tests.test_gpu_attention import BF, HF, check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    fs.load_library()


@pytest.fixture(autouse=True)
def _no_wait_gave_up():
    yield
    fs.fs_check()


def dirty(shape, dtype):
    """Leaves NaN in the memory that the next results of this shape take."""
    x = [torch.full(shape, math.nan, dtype=dtype, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    del x


@pytest.mark.parametrize("n,m", [(1, 300), (140, 300), (0, 5), (3, 0)])
@pytest.mark.parametrize("side", [False, True])
def test_an_expanded_row_has_a_gradient_for_each_head(n, m, side):
    """One row expanded to all heads is a table of equal rows, not the shared row of
    shape (1, buckets)."""
    c, how, dout = make(2, n, m, 4, 2, 64, BF, nb=16, far=50, shared=True, seed=41)
    row = how["bias"]
    stored = dict(how, bias=row.repeat(4, 1))
    a = fs.fs_cross_attention(c["q"], c["k"], c["v"], **stored)
    ga = fs.fs_cross_attention_grad(c["q"], c["k"], c["v"], *a, dout, **stored)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream() if side else None
    spread = dict(how, bias=row.expand(4, -1))
    dirty((4, 16), BF)
    b = fs.fs_cross_attention(c["q"], c["k"], c["v"], stream=stream, **spread)
    gb = fs.fs_cross_attention_grad(c["q"], c["k"], c["v"], *b, dout, stream=stream, **spread)
    torch.cuda.synchronize()
    for x, y in zip((*a, *ga), (*b, *gb)):
        assert x.shape == y.shape and torch.equal(x, y)
    if n and m:
        check(c, stored, dout)
        check(c, how, dout)
