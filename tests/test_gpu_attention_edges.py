"""Cross attention on the GPU where a result could be lost or stale: expanded tables, results
that overlap, streams of other libraries, arguments of other kinds, lowest values."""
import math

import numpy as np
import pytest
import torch

from streaming_sinkhorn_solver_gb300 import binding as fs
from tests.test_gpu_attention import BF, HF, check, make, reference

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


# (batch, token, head) strides of (2, 3, 4, 64) tensors
OVERLAPS = [(2048, 64, 64), (2048, 192, 64), (2048, 256, 32), (256, 256, 64), (64, 256, 128), (700, 256, 64),
            (0, 256, 64), (2048, 64, 0), (1024, 63, 2048)]
APART = [(768, 256, 64), (2048, 256, 64), (64, 512, 128), (64, 128, 384), (768, 64, 192), (256, 512, 64),
         (5000, 1000, 101)]


@pytest.mark.parametrize("name", ["out", "dq", "dk", "dv"])
def test_results_that_overlap_are_refused(name):
    c, how, dout = make(2, 3, 3, 4, 4, 64, BF, seed=42)
    a = fs.fs_cross_attention(c["q"], c["k"], c["v"], **how)
    want = dict(zip(("out", "lse", "dq", "dk", "dv"),
                    (*a, *fs.fs_cross_attention_grad(c["q"], c["k"], c["v"], *a, dout, **how))))

    def call(strides):
        store = torch.zeros(20000, dtype=BF, device="cuda")
        x = store.as_strided((2, 3, 4, 64), strides + (1,))
        if name == "out":
            fs.fs_cross_attention(c["q"], c["k"], c["v"], out=x, **how)
        else:
            fs.fs_cross_attention_grad(c["q"], c["k"], c["v"], *a, dout, **{name: x}, **how)
        return x

    for strides in OVERLAPS:
        with pytest.raises(fs.FlashSinkhornError, match="overlap"):
            call(strides)
    for strides in APART:
        assert torch.equal(call(strides), want[name])


def test_a_result_of_one_entry_may_have_any_stride_there():
    c, how, _ = make(1, 3, 5, 1, 1, 64, BF, seed=43)
    store = torch.zeros(1000, dtype=BF, device="cuda")
    x = store.as_strided((1, 3, 1, 64), (0, 64, 0, 1))
    want, _ = fs.fs_cross_attention(c["q"], c["k"], c["v"], **how)
    assert torch.equal(fs.fs_cross_attention(c["q"], c["k"], c["v"], out=x, **how)[0], want)


class Foreign:
    """What other libraries' stream objects have in common with torch's."""

    def __init__(self, stream):
        self.cuda_stream = stream.cuda_stream


@pytest.mark.parametrize("kind", [lambda s: s, lambda s: s.cuda_stream, Foreign])
def test_results_belong_to_the_stream_that_writes_them(kind):
    """Memory that pending work of the current stream still writes to, although it was freed
    there, is not handed to a call on another stream."""
    c, how, dout = make(2, 150, 300, 4, 2, 64, BF, nb=16, far=50, seed=44)
    a = fs.fs_cross_attention(c["q"], c["k"], c["v"], **how)
    want = [*a, *fs.fs_cross_attention_grad(c["q"], c["k"], c["v"], *a, dout, **how)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    pending = [torch.empty_like(x) for x in want for _ in range(4)]
    torch.cuda._sleep(200_000_000)         # 0.1 s of the current stream
    for x in pending:
        x.fill_(math.nan)
    del pending, x
    b = fs.fs_cross_attention(c["q"], c["k"], c["v"], stream=kind(side), **how)
    got = [*b, *fs.fs_cross_attention_grad(c["q"], c["k"], c["v"], *b, dout, stream=kind(side), **how)]
    torch.cuda.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x, y)


@pytest.mark.parametrize("handle", [0, 1])
def test_the_default_stream_by_its_handle(handle):
    c, how, _ = make(1, 20, 40, 2, 2, 64, BF, seed=45)
    want = fs.fs_cross_attention(c["q"], c["k"], c["v"], **how)
    got = fs.fs_cross_attention(c["q"], c["k"], c["v"], stream=handle, **how)
    torch.cuda.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


class Tagged(torch.Tensor):
    """A tensor of a user's own class."""


@pytest.mark.parametrize("n", [2, 150])
def test_tensors_of_a_subclass_are_read_and_not_written(n):
    c, how, dout = make(2, n, 300, 4, 2, 64, BF, nb=16, far=50, seed=46)
    a = fs.fs_cross_attention(c["q"], c["k"], c["v"], **how)
    want = [*a, *fs.fs_cross_attention_grad(c["q"], c["k"], c["v"], *a, dout, **how)]
    own = {x: y.clone().as_subclass(Tagged) for x, y in c.items()}
    b = fs.fs_cross_attention(own["q"], own["k"], own["v"], **how)
    got = [*b, *fs.fs_cross_attention_grad(own["q"], own["k"], own["v"], *b, dout, **how)]
    for x, y in zip(want, got):
        assert torch.equal(x, y)
    for x, y in c.items():
        assert torch.equal(y, own[x].as_subclass(torch.Tensor))
    assert b[0].data_ptr() != own["q"].data_ptr()


def test_arguments_of_other_kinds_are_refused():
    c, how, dout = make(2, 3, 5, 4, 2, 64, BF, nb=8, far=9)
    q, k, v = c["q"], c["k"], c["v"]
    out, lse = fs.fs_cross_attention(q, k, v, **how)
    for other in (np.zeros((2, 5, 2, 64), np.float16), [1.0], None):
        for args in ((other, k, v), (q, other, v), (q, k, other)):
            with pytest.raises(TypeError):
                fs.fs_cross_attention(*args, **how)
            with pytest.raises(TypeError):
                fs.fs_cross_attention_grad(*args, out, lse, dout, **how)
    for name, other in (("key_mask", np.ones((2, 5), bool)), ("key_mask", [[1] * 5] * 2),
                        ("bias", np.zeros((4, 8), np.float16)), ("bias_buckets", [0] * 19),
                        ("kv_len", [5, 5]), ("q_pos", 3)):
        with pytest.raises(TypeError):
            fs.fs_cross_attention(q, k, v, **dict(how, **{name: other}))
    with pytest.raises(TypeError):
        fs.fs_cross_attention_grad(q, k, v, out, lse, dout, dbias=np.zeros((4, 8), np.float16), **how)
    for shape in ((2, 3, 4, 0), (3, 4, 64)):
        with pytest.raises(ValueError):
            fs.fs_cross_attention(q.new_zeros(shape), k, v, **how)


@pytest.mark.parametrize("n", [2, 150])
def test_rows_that_have_nothing_but_the_lowest_bias(n):
    """In bfloat16 they are empty.  In float16 -65504 is a finite bias: a softmax of the scores,
    which next to -94503 in base 2 are rounded to multiples of 2^-7.  p is then off by a
    factor of up to 2^(4 * 2^-8) (its score, its row's, lse and its product with log2 e), 1.1 %,
    ds too, and delta by as much of sum |dout v|; lse by its own rounding, 2^-8, twice."""
    for dtype in (BF, HF):
        c, how, dout = make(2, n, 300, 2, 2, 64, dtype, nb=8, far=20, seed=47)
        how["bias"][1] = torch.finfo(dtype).min
        out, lse = fs.fs_cross_attention(c["q"], c["k"], c["v"], **how)
        dq, dk, dv, dbias = fs.fs_cross_attention_grad(c["q"], c["k"], c["v"], out, lse, dout, **how)
        if dtype == BF:
            assert bool((out[:, :, 1] == 0).all()) and bool((lse[:, 1] == -math.inf).all())
            assert all(bool((x[:, :, 1] == 0).all()) for x in (dq, dk, dv)) and bool((dbias[1] == 0).all())
            continue
        ref = reference(c, how, dout)
        p, do = 0.011, dout.cpu().double()
        v = c["v"].cpu().double()[:, :, 1]
        z = how["scale"] * torch.einsum("bic,bjc->bij", c["q"].cpu().double()[:, :, 1], c["k"].cpu().double()[:, :, 1])
        w = z.softmax(-1)
        tol = ref["tol"]["out"][:, :, 1] + p * 2 * torch.einsum("bij,bjc->bic", w, v.abs())
        assert float(((out.cpu().double() - ref["out"])[:, :, 1].abs() - tol).max()) <= 0
        assert float((lse.cpu().double() - ref["lse"])[:, 1].abs().max()) <= 2 * 2.0 ** -8
        tol = ref["tol"]["dv"][:, :, 1] + p * torch.einsum("bij,bic->bjc", w, do[:, :, 1].abs())
        assert float(((dv.cpu().double() - ref["dv"])[:, :, 1].abs() - tol).max()) <= 0
        ds = p * 4 * w * torch.einsum("bic,bijc->bij", do[:, :, 1].abs(),
                                      v.abs()[:, None] + (w @ v.abs())[:, :, None])
        for name, x, tol in (("dq", dq, torch.einsum("bij,bjc->bic", ds, c["k"].cpu().double()[:, :, 1].abs())),
                             ("dk", dk, torch.einsum("bij,bic->bjc", ds, c["q"].cpu().double()[:, :, 1].abs()))):
            tol = ref["tol"][name][:, :, 1] + how["scale"] * tol
            assert float(((x.cpu().double() - ref[name])[:, :, 1].abs() - tol).max()) <= 0, name
