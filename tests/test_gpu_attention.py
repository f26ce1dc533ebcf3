"""Cross attention on the GPU against the 64-bit reference, forward and
gradients, at the sizes, masks, strides and types where it can go wrong.  Each
result is within the bound that tests/attention_ref.py derives for it."""
import math

import pytest
import torch

from streaming_sinkhorn_solver_gb300 import binding as fs
from tests.attention_ref import attention64

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    fs.load_library()


@pytest.fixture(autouse=True)
def _no_wait_gave_up():
    yield
    fs.fs_check()


def make(B, n, m, H, G, d, dtype=BF, lens=None, drop=0.0, nb=0, far=0, pos=None, shared=False,
         seed=0, gain=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=g, device="cuda")

    c = dict(q=(gain * r(B, n, H, d)).to(dtype), k=r(B, m, G, d).to(dtype), v=r(B, m, G, d).to(dtype))
    how = dict(scale=d ** -0.5)
    if lens is not None:
        how["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if drop:
        how["key_mask"] = torch.rand(B, m, generator=g, device="cuda") >= drop
    if nb:
        how["bias"] = r(1 if shared else H, nb).to(dtype)
        how["bias_buckets"] = torch.from_numpy(fs.fs_relative_buckets(nb, far)).cuda()
        if pos is not None:
            how["q_pos"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
    return c, how, r(B, n, H, d).to(dtype)


def reference(c, how, dout=None):
    h = dict(how)
    h["buckets"] = h.pop("bias_buckets", None)
    return attention64(c["q"], c["k"], c["v"], dout=dout, **h)


def within(got, ref, name):
    x, want, tol = got.detach().cpu().double(), ref[name], ref["tol"][name]
    assert x.shape == want.shape, name
    fine = torch.isfinite(want)
    assert torch.equal(x[~fine], want[~fine]), name
    over = ((x - want).abs() - tol)[fine]
    assert over.numel() == 0 or float(over.max()) <= 0, \
        f"{name}: {float(over.max()):.3g} over the bound at {int((over > 0).sum())} places"


def check(c, how, dout=None):
    ref = reference(c, how, dout)
    out, lse = fs.fs_cross_attention(c["q"], c["k"], c["v"], **how)
    within(out, ref, "out")
    within(lse, ref, "lse")
    if dout is not None:
        dq, dk, dv, db = fs.fs_cross_attention_grad(c["q"], c["k"], c["v"], out, lse, dout, **how)
        within(dq, ref, "dq")
        within(dk, ref, "dk")
        within(dv, ref, "dv")
        assert (db is None) == ("bias" not in how)
        if db is not None:
            within(db, ref, "dbias")


# one token to several tiles, sizes around the tile edges, odd head dimensions
SIZES = [(1, 1, 1, 1, 1, 64), (1, 1, 128, 2, 2, 128), (2, 3, 129, 2, 1, 64), (1, 127, 128, 2, 2, 64),
         (1, 128, 127, 2, 2, 128), (2, 129, 257, 3, 3, 64), (1, 256, 384, 2, 1, 128),
         (1, 300, 700, 4, 2, 80), (2, 65, 200, 6, 2, 96), (1, 40, 90, 2, 2, 8), (1, 33, 70, 2, 1, 33),
         (1, 20, 50, 2, 2, 1), (3, 17, 1000, 8, 1, 64), (1, 513, 130, 2, 2, 112), (1, 5, 3, 4, 4, 127)]


@pytest.mark.parametrize("B,n,m,H,G,d", SIZES)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_sizes(B, n, m, H, G, d, dtype):
    check(*make(B, n, m, H, G, d, dtype, seed=n + m))


@pytest.mark.parametrize("lens", [[300, 1, 0], [128, 129, 127], [299, 400, -3]])
@pytest.mark.parametrize("drop", [0.0, 0.4, 1.1])
@pytest.mark.parametrize("n", [1, 140])
def test_masks(lens, drop, n):
    """Lengths of zero and beyond m, random masks, and masks that leave nothing."""
    check(*make(3, n, 300, 4, 2, 64, HF if drop else BF, lens=lens, drop=drop, seed=7))


@pytest.mark.parametrize("n,m", [(1, 500), (3, 40), (150, 300), (260, 900)])
@pytest.mark.parametrize("nb,far,shared", [(8, 5, False), (32, 128, False), (16, 700, True),
                                           (32, 2048, False)])
def test_bias(n, m, nb, far, shared):
    check(*make(2, n, m, 4, 2, 64, BF, nb=nb, far=far, shared=shared, pos=[m // 2, 3], seed=11))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("drop", [0.0, 0.2])
def test_many_key_tiles_with_partial_ones(d, drop):
    """Sequences of more key tiles than the kernels keep in flight, with masked tiles."""
    check(*make(2, 130, 2300, 2, 1, d, BF, lens=[2300, 1900], drop=drop, seed=22))
    fs.fs_check()


def test_bias_with_masks_and_wide_heads():
    check(*make(3, 200, 333, 6, 3, 128, HF, lens=[333, 130, 0], drop=0.3, nb=48, far=300, seed=3))


def test_widest_bias_with_wide_heads():
    """The largest max_distance, where the gradient's shared memory is tightest."""
    check(*make(1, 300, 900, 2, 1, 128, BF, nb=64, far=2048, pos=[400], seed=23))


def test_positions_far_outside_the_keys():
    check(*make(2, 70, 260, 2, 2, 64, BF, nb=32, far=128, pos=[100000, -2000], seed=4))


@pytest.mark.parametrize("value", [-math.inf, -3.0e38])
def test_forbidding_bias(value):
    """Buckets forbidden by -inf or the type's lowest value; rows whose every
    pair is forbidden are empty rows."""
    c, how, dout = make(1, 150, 200, 2, 2, 64, BF, nb=8, far=16, seed=5)
    how["bias"][:, 4:] = value            # keys after the query
    check(c, how, dout)
    how["bias"][1] = value
    check(c, how, dout)
    out, lse = fs.fs_cross_attention(c["q"], c["k"], c["v"], **how)
    assert bool((out[:, :, 1] == 0).all()) and bool((lse[:, 1] == -math.inf).all())


def test_large_finite_bias_of_float16():
    c, how, dout = make(1, 30, 80, 2, 2, 64, HF, nb=8, far=16, seed=6)
    how["bias"][:, 2] = -65504.0
    check(c, how, dout)


@pytest.mark.parametrize("n", [1, 200])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_masked_places_may_hold_anything(n, bad):
    c, how, dout = make(2, n, 400, 4, 2, 64, BF, lens=[390, 150], drop=0.3, nb=8, far=20, seed=8)
    gone = ~how["key_mask"] | (torch.arange(400, device="cuda")[None] >= how["kv_len"][:, None])
    dirty = {x: c[x].clone() for x in ("k", "v")}
    for x in dirty.values():
        x[gone] = bad
    a = fs.fs_cross_attention(c["q"], c["k"], c["v"], **how)
    b = fs.fs_cross_attention(c["q"], dirty["k"], dirty["v"], **how)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga = fs.fs_cross_attention_grad(c["q"], c["k"], c["v"], *a, dout, **how)
    gb = fs.fs_cross_attention_grad(c["q"], dirty["k"], dirty["v"], *a, dout, **how)
    for x, y in zip(ga, gb):
        assert torch.equal(x, y)
    assert bool((ga[1][gone] == 0).all()) and bool((ga[2][gone] == 0).all())


@pytest.mark.parametrize("n", [1, 130])
def test_nan_in_counted_places_is_not_hidden(n):
    c, how, _ = make(2, n, 300, 2, 2, 64, BF, seed=9)
    c["k"][0, 7, 1, 3] = math.nan
    out, lse = fs.fs_cross_attention(c["q"], c["k"], c["v"], **how)
    assert bool(torch.isnan(out[0, :, 1]).all()) and bool(torch.isnan(lse[0, 1]).all())
    assert bool(torch.isfinite(out[1]).all()) and bool(torch.isfinite(out[0, :, 0]).all())


@pytest.mark.parametrize("B,n,m", [(0, 3, 5), (2, 0, 5), (2, 3, 0), (1, 200, 0)])
def test_empty_sizes(B, n, m):
    c, how, dout = make(B, n, m, 2, 1, 64, BF, nb=8, far=9)
    out, lse = fs.fs_cross_attention(c["q"], c["k"], c["v"], **how)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    dq, dk, dv, db = fs.fs_cross_attention_grad(c["q"], c["k"], c["v"], out, lse, dout, **how)
    for x in (dq, dk, dv, db):
        assert bool((x == 0).all())


@pytest.mark.parametrize("gain", [0.01, 30.0])
@pytest.mark.parametrize("n", [2, 140])
def test_flat_and_peaked_scores(gain, n):
    """Nearly equal weights, and rows dominated by one key (scores of about 30
    standard deviations, which move the running maximum far)."""
    check(*make(1, n, 600, 2, 2, 64, BF, gain=gain, seed=10))


def test_growing_scores_move_the_maximum_every_tile():
    c, how, dout = make(1, 140, 900, 2, 2, 64, HF, seed=12, gain=1.0)
    ramp = torch.linspace(0.0, 6.0, 900, device="cuda")[None, :, None, None]
    c["k"] = (c["k"] * 0.1 + ramp * c["q"][:, :1].mean(2, keepdim=True)).to(HF)
    check(c, how, dout)
    c["k"] = c["k"].flip(1).contiguous()
    check(c, how, dout)


def layouts(x, kind):
    B, t, h, d = x.shape
    if kind == "heads-first":
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    if kind == "tokens-first":
        return x.permute(1, 0, 2, 3).contiguous().permute(1, 0, 2, 3)
    if kind == "padded":                # rows of d + 8 elements
        y = torch.full((B, t, h, d + 8), math.nan, dtype=x.dtype, device=x.device)
        y[..., :d] = x
        return y[..., :d]
    if kind == "odd":                   # neither address nor strides a multiple of 16 bytes
        y = torch.full((B * t * h * (d + 3) + 1,), math.nan, dtype=x.dtype, device=x.device)[1:]
        y = y.view(B, t, h, d + 3)
        y[..., :d] = x
        return y[..., :d]
    raise ValueError(kind)


@pytest.mark.parametrize("kind", ["heads-first", "tokens-first", "padded", "odd"])
@pytest.mark.parametrize("n", [2, 150])
def test_strides_change_nothing(kind, n):
    c, how, dout = make(2, n, 333, 4, 2, 72, BF, lens=[333, 200], nb=8, far=30, seed=13)
    a = fs.fs_cross_attention(c["q"], c["k"], c["v"], **how)
    ga = fs.fs_cross_attention_grad(c["q"], c["k"], c["v"], *a, dout, **how)
    s = {x: layouts(c[x], kind) for x in c}
    out = layouts(torch.zeros_like(c["q"]), kind)
    b = fs.fs_cross_attention(s["q"], s["k"], s["v"], out=out, **how)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    dst = {"d" + x: layouts(torch.zeros_like(c[x]), kind) for x in c}
    gb = fs.fs_cross_attention_grad(s["q"], s["k"], s["v"], *b, layouts(dout, kind), **dst, **how)
    for x, y in zip(ga, gb):
        assert torch.equal(x, y)


def test_broadcast_inputs():
    """One encoder output for the whole batch, one mask row, one query for all heads."""
    c, how, dout = make(3, 130, 200, 4, 2, 64, BF, seed=14)
    c["k"], c["v"] = (c[x][:1].expand(3, -1, -1, -1) for x in ("k", "v"))
    c["q"] = c["q"][:, :, :1].expand(-1, -1, 4, -1)
    how["key_mask"] = (torch.arange(200, device="cuda") % 3 != 0)[None].expand(3, -1)
    check(c, how, dout)


@pytest.mark.parametrize("n", [1, 140])
def test_offsets_beyond_32_bits(n):
    """Keys and values whose element offsets pass 2^31 (and 2^32), by tokens and by batch."""
    c, how, dout = make(2, n, 40, 2, 2, 64, BF, seed=15)
    store = torch.zeros(2 ** 32 + 2 ** 30, dtype=BF, device="cuda")
    far = {}
    for i, x in enumerate(("k", "v")):
        far[x] = store[i * 256:].as_strided((2, 40, 2, 64), (2 ** 26 + 8192, 2 ** 26 + 2 ** 25, 64, 1))
        far[x].copy_(c[x])
    check(dict(c, **far), how, dout)
    for i, x in enumerate(("k", "v")):
        far[x] = store[i * 8192:].as_strided((2, 40, 2, 64), (2 ** 32 + 64, 128, 64, 1))
        far[x].copy_(c[x])
    check(dict(c, **far), how, dout)


@pytest.mark.parametrize("B,n,H,G,d", [(1, 1, 8, 8, 64), (2, 1, 8, 1, 128), (1, 4, 8, 2, 80),
                                       (5, 2, 3, 3, 64), (1, 6, 16, 1, 64)])
def test_few_queries_long_cache(B, n, H, G, d):
    lens = [20011 - 3001 * b for b in range(B)]
    c, how, _ = make(B, n, 20011, H, G, d, BF, lens=lens, nb=32, far=128,
                     pos=[19000 - 10 * b for b in range(B)], seed=16)
    check(c, how)


def test_single_tokens_agree_with_the_whole_sequence():
    """A decoder's steps, one token each at its position, against one call of all."""
    c, how, _ = make(2, 24, 300, 4, 2, 64, HF, lens=[300, 120], nb=32, far=60, seed=17)
    ref = reference(c, how)
    for i in range(0, 24, 7):
        step = dict(how, q_pos=torch.full((2,), i, dtype=torch.int32, device="cuda"))
        out, lse = fs.fs_cross_attention(c["q"][:, i:i + 1], c["k"], c["v"], **step)
        part = {"out": ref["out"][:, i:i + 1], "lse": ref["lse"][:, :, i:i + 1],
                "tol": {"out": ref["tol"]["out"][:, i:i + 1], "lse": ref["tol"]["lse"][:, :, i:i + 1]}}
        within(out, part, "out")
        within(lse, part, "lse")


@pytest.mark.parametrize("n,m", [(1, 9000), (300, 700)])
def test_results_are_bitwise_repeatable(n, m):
    c, how, dout = make(2, n, m, 4, 2, 64, BF, lens=[m, m - 100], nb=16, far=50, seed=18)
    first = None
    for _ in range(3):
        a = fs.fs_cross_attention(c["q"], c["k"], c["v"], **how)
        r = [*a, *fs.fs_cross_attention_grad(c["q"], c["k"], c["v"], *a, dout, **how)]
        if first is None:
            first = r
        for x, y in zip(first, r):
            assert torch.equal(x, y)


@pytest.mark.parametrize("n,m,d", [(1, 5000, 64), (200, 300, 72), (3, 60, 33)])
def test_graph_replay_and_other_streams(n, m, d):
    c, how, dout = make(2, n, m, 4, 2, d, BF, lens=[m, m // 2], drop=0.1, nb=16, far=50, seed=19)
    a = fs.fs_cross_attention(c["q"], c["k"], c["v"], **how)
    ga = fs.fs_cross_attention_grad(c["q"], c["k"], c["v"], *a, dout, **how)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    b = fs.fs_cross_attention(c["q"], c["k"], c["v"], stream=side, **how)
    gb = fs.fs_cross_attention_grad(c["q"], c["k"], c["v"], *b, dout, stream=side, **how)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = fs.fs_cross_attention(c["q"], c["k"], c["v"], **how)
        gr = fs.fs_cross_attention_grad(c["q"], c["k"], c["v"], *r, dout, **how)
    for x in (*r, *gr):
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for x, y, z in zip((*a, *ga), (*b, *gb), (*r, *gr)):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_gradients_against_differences():
    """The directional derivative of <out, dout> along each input, from two calls with
    that input moved by +-h.  float16 results of rms 0.3, rounded with u = 2^-11, make the
    difference of the two sums of N values uncertain by about 2 u 0.3 sqrt(N) |dout|; h
    moves the inputs by 2^-5 of their size, exactly representable directions."""
    c, how, dout = make(1, 64, 96, 2, 1, 32, HF, nb=8, far=20, seed=20, gain=1.0)
    out, lse = fs.fs_cross_attention(c["q"], c["k"], c["v"], **how)
    grads = dict(zip(("q", "k", "v", "bias"),
                     fs.fs_cross_attention_grad(c["q"], c["k"], c["v"], out, lse, dout, **how)))
    g = torch.Generator(device="cuda").manual_seed(21)
    for name, grad in grads.items():
        x = how["bias"] if name == "bias" else c[name]
        h = 2.0 ** -5
        sign = torch.where(torch.rand(x.shape, generator=g, device="cuda") < 0.5, -1.0, 1.0)
        # moves that the type can hold, the same size up and down
        up, down = (x.float() + h * sign).to(HF), (x.float() - h * sign).to(HF)
        sums = []
        for y in (up, down):
            cc, hh = dict(c), dict(how)
            (hh if name == "bias" else cc)[name] = y
            o, _ = fs.fs_cross_attention(cc["q"], cc["k"], cc["v"], **hh)
            sums.append(float((o.double() * dout.double()).sum()))
        want = float((grad.double() * (up.double() - down.double())).sum())
        got = sums[0] - sums[1]
        N = out.numel()
        noise = 6 * 2 * 2.0 ** -11 * 0.3 * math.sqrt(N)
        # third-order term: moves of 2^-5 in each of d = 32 coordinates change z by up to
        # scale |h| sum |k| ~ 0.14, so (0.14)^2 / 6 of the value itself
        assert abs(got - want) <= noise + 0.01 * abs(want), name


def test_binding_refusals():
    c, how, dout = make(2, 3, 5, 4, 2, 64, BF, nb=8, far=9)
    q, k, v = c["q"], c["k"], c["v"]

    def refused(error, *args, **kw):
        with pytest.raises(error):
            fs.fs_cross_attention(*args, **kw)

    refused(TypeError, q, k.half(), v)
    refused(TypeError, q.float(), k.float(), v.float())
    refused(TypeError, q, k.cpu(), v)
    refused(TypeError, q, k.transpose(2, 3).contiguous().transpose(2, 3), v)
    refused(ValueError, q, k, v[:, :4])
    refused(ValueError, q[0], k, v)
    refused(TypeError, q, k, v, kv_len=torch.ones(2, dtype=torch.int64, device="cuda"))
    refused(ValueError, q, k, v, key_mask=torch.ones(2, 4, dtype=torch.bool, device="cuda"))
    refused(TypeError, q, k, v, key_mask=torch.ones(2, 5, device="cuda"))
    refused(TypeError, q, k, v, bias=how["bias"])
    refused(ValueError, q, k, v, bias=how["bias"][:2], bias_buckets=how["bias_buckets"])
    refused(ValueError, q, k, v, bias=how["bias"], bias_buckets=how["bias_buckets"][1:])
    refused(TypeError, q, k, v, out=torch.empty(2, 3, 4, 64, device="cuda"))
    for scale in (0.0, -1.0, math.nan):
        refused(fs.FlashSinkhornError, q, k, v, scale=scale)
    wide = torch.zeros(1, 2, 2, 136, dtype=BF, device="cuda")
    refused(fs.FlashSinkhornError, wide, wide, wide)
    refused(fs.FlashSinkhornError, q, k, v, out=q[:, :, :1].expand(-1, -1, 4, -1))   # rows overlap
    out, lse = fs.fs_cross_attention(q, k, v, **how)
    with pytest.raises(ValueError):
        fs.fs_cross_attention_grad(q, k, v, out, lse[:1], dout, **how)
    with pytest.raises(TypeError):
        fs.fs_cross_attention_grad(q, k, v, out, lse, dout, dbias=how["bias"].float(), **how)


@pytest.mark.parametrize("n,m,nb,far", [(900, 60, 8, 300), (300, 1500, 16, 64)])
def test_bias_gradient_where_one_bucket_holds_most_of_the_weight(n, m, nb, far):
    """The sum of ds over a row is 0, so such a bucket's gradient is a small remainder; in the
    2-norm it is as exact as its rounding to 8 bits allows (2^-9), and as much again for
    the scores' and the sums' rounding."""
    c, how, dout = make(2, n, m, 4, 2, 64, BF, nb=nb, far=far, seed=31)
    out, lse = fs.fs_cross_attention(c["q"], c["k"], c["v"], **how)
    dbias = fs.fs_cross_attention_grad(c["q"], c["k"], c["v"], out, lse, dout, **how)[3]
    want = reference(c, how, dout)["dbias"]
    assert float((dbias.cpu().double() - want).norm()) <= 2.0 ** -8 * float(want.norm())


@pytest.mark.parametrize("n,m,H,G,d,nb", [(40, 3100, 4, 2, 80, 16), (40, 3100, 2, 2, 64, 0),
                                          (2600, 100, 4, 1, 128, 0), (2600, 140, 2, 1, 64, 16)])
def test_gradients_of_few_blocks_with_many_tiles(n, m, H, G, d, nb):
    """Shares of the tiles in blocks of their own, with a share that no key counts in."""
    check(*make(2, n, m, H, G, d, BF, lens=[m, m // 3], drop=0.2, nb=nb, far=90, seed=32))
