"""Tree attention and rotary positions at the ends of their ranges: keys that no row or not every row
sees, scales and queries of very different sizes, far angles; short
last blocks, padded rows.  Bounds as in kv_ref."""
import math
from fractions import Fraction

import pytest
import torch

from streaming_sinkhorn_solver_gb300 import binding as fs
from tests.kv_ref import quantise, rotary64, tree64
from tests.test_gpu_cache import BF, E4M3, HALF, I8, NAN, check, gen, random_parents, setting, within

pytestmark = pytest.mark.gpu
EIGHT = [E4M3, I8]


def values_of(x, held):
    """What rows x stand for in a cache, float64."""
    if held in (BF, HALF):
        return x.double()
    code, scale = quantise(x, held)
    return code.double() * scale.double()[..., None]


def attend(q, cache, table, ctx, parents):
    got = fs.fs_tree_attention(q.cuda(), cache, table.cuda(), torch.tensor(ctx, dtype=torch.int32).cuda(),
                               None if parents is None else parents.cuda())
    fs.fs_check()
    return got


# --- keys that a row does not see ----------------------------------------------

@pytest.mark.parametrize("held", [BF, *EIGHT])
@pytest.mark.parametrize("n,d", [(1, 64), (2, 128), (3, 72), (9, 128), (20, 64), (40, 128)])
@pytest.mark.parametrize("which", ["k", "v"])
def test_absent_tokens_beside_rows_that_are_not_numbers(held, n, d, which):
    """A NaN row of the context: the tokens that are there see it, padding does not."""
    ctx = [300, 77]
    q, cache, table, k, v = setting(n + d, 2, n, ctx, 8, 2, d, BF, held, 16)
    rows = torch.ones(2, 1, 2, d, dtype=BF)
    rows[0] = NAN
    at = torch.tensor([[40], [-1]], dtype=torch.int32)
    one = torch.ones_like(rows)
    fs.fs_cache_write(cache, table.cuda(), at.cuda(), *((rows.cuda(), one.cuda()) if which == "k"
                                                        else (one.cuda(), rows.cuda())))
    parents = random_parents(gen(n), 2, n)
    parents[:, -1] = -2
    out, lse = attend(q, cache, table, ctx, parents)
    assert not out[:, -1].any() and bool((lse[:, :, -1] == -math.inf).all())
    assert bool(torch.isnan(out[0, :-1]).all())
    want = tree64(q[1:], k[1:], v[1:], torch.ones(k.shape[:2], dtype=torch.bool)[1:], ctx[1:], parents[1:],
                  weights=HALF if held in EIGHT else None)
    within(out[1:], want["out"], want["tol"]["out"], "out")
    within(lse[1:], want["lse"], want["tol"]["lse"], "lse")


@pytest.mark.parametrize("held", EIGHT)
@pytest.mark.parametrize("n,H,G,d", [(2, 4, 2, 64), (3, 4, 4, 128), (5, 8, 2, 72), (12, 8, 2, 128), (40, 4, 2, 64),
                                     (50, 8, 2, 128)])
@pytest.mark.parametrize("fill", [0.0, 1e-40, -1.0, -1e-40, 3e38, math.inf, NAN])
def test_scales_of_slots_that_were_never_written(held, n, H, G, d, fill):
    """Padding's tokens are left out of the write: their slots' scales may be anything."""
    ctx = [100, 61]
    gone = max(1, n // 4)
    g = gen(n + d)
    page, per = 16, -(-(max(ctx) + n) // 16)
    cache = fs.KVCache(*(torch.zeros(2 * per, G, page, d, dtype=torch.int8, device="cuda").view(held)
                         for _ in range(2)),
                       *(torch.full((2 * per, G, page), fill, device="cuda") for _ in range(2)))
    table = torch.randperm(2 * per, generator=g).int().view(2, per)
    x, y = (torch.randn(2, per * page, G, d, generator=g).bfloat16() for _ in range(2))
    at = torch.arange(per * page, dtype=torch.int32).expand(2, -1).clone()
    for b in range(2):
        at[b, ctx[b] + n - gone:] = -1
    fs.fs_cache_write(cache, table.cuda(), at.cuda(), x.cuda(), y.cuda())
    q = (2 * torch.randn(2, n, H, d, generator=g)).bfloat16()
    parents = random_parents(g, 2, n, absent=gone)
    check(q, cache, table, values_of(x, held), values_of(y, held), ctx, parents)


@pytest.mark.parametrize("held", EIGHT)
@pytest.mark.parametrize("n,H", [(4, 2), (40, 8)])
@pytest.mark.parametrize("scale", [0.0, 1e-40, -1.0, 3e38, math.inf])
def test_value_scales_that_are_none(held, n, H, scale):
    """A value scale that no row can have: NaN for the tokens that see it, nothing for others."""
    ctx = [100, 61]
    q, cache, table, k, v = setting(8, 2, n, ctx, H, 2, 64, BF, held, 16)
    bad = n // 2
    for b in range(2):
        p = ctx[b] + bad
        cache.v_scale[int(table[b, p // 16]), :, p % 16] = scale
    parents = torch.full((2, n), -1, dtype=torch.int32)
    parents[:, -1] = bad
    out, lse = attend(q, cache, table, ctx, parents)
    others = [t for t in range(n - 1) if t != bad]
    want = tree64(q, k, v, torch.ones(k.shape[:2], dtype=torch.bool), ctx, parents, weights=HALF)
    within(out[:, others], want["out"][:, others], want["tol"]["out"][:, others], "out")
    within(lse[:, :, others], want["lse"][:, :, others], want["tol"]["lse"][:, :, others], "lse")
    assert bool(torch.isnan(out[:, [bad, n - 1]]).all())


# --- scales and queries of very different sizes -----------------------------------

@pytest.mark.parametrize("held", EIGHT)
@pytest.mark.parametrize("n,H,G,d", [(1, 4, 2, 64), (2, 8, 2, 128), (20, 4, 2, 64), (20, 4, 2, 128), (40, 4, 2, 128),
                                     (90, 4, 2, 64)])
@pytest.mark.parametrize("ctx", [37, 700])
@pytest.mark.parametrize("size", [2.0 ** 60, 2.0 ** 119])
@pytest.mark.parametrize("order", ["first", "last", "between", "mixed"])
def test_rows_of_zeros_beside_large_ones(held, n, H, G, d, ctx, size, order):
    """Every key counts in the sum by its score alone, whatever its value: rows of zeros (held at
    2^-80) beside values of 2^60 and of 2^119, all of one weight."""
    q, cache, table, k, v = setting(n, 1, n, [ctx], H, G, d, BF, held, 16)
    m = ctx + n
    g = gen(m)
    rows = torch.randn(1, m, G, d, generator=g).clamp(-4, 4) * size
    small = {"first": torch.arange(m) >= 3, "last": torch.arange(m) < ctx - 2,
             "between": torch.arange(m) % 7 != 3, "mixed": torch.rand(m, generator=g) < 0.5}[order]
    rows[:, small] = 0
    vv, kk = rows.bfloat16(), torch.zeros(1, m, G, d, dtype=BF)
    fs.fs_cache_write(cache, table.cuda(), torch.arange(m, dtype=torch.int32)[None].cuda(), kk.cuda(), vv.cuda())
    k[:, :m], v[:, :m] = values_of(kk, held), values_of(vv, held)
    check(q, cache, table, k, v, [ctx])


@pytest.mark.parametrize("held", EIGHT)
@pytest.mark.parametrize("n", [1, 20, 40, 100])
def test_weights_of_rows_that_end_small(held, n):
    """The large values come with scores that leave them next to no weight: rows of zeros and of
    small values have it all."""
    ctx = 200
    q, cache, table, k, v = setting(n, 1, n, [ctx], 4, 2, 64, BF, held, 16)
    m = ctx + n
    g = gen(m)
    q = torch.ones_like(q)
    kk = torch.randn(1, m, 2, 64, generator=g).bfloat16()
    vv = torch.randn(1, m, 2, 64, generator=g).bfloat16()
    vv[:, ::3] = 0
    vv[:, 5] *= 2.0 ** 118
    kk[:, 5] = -12.0                 # 96 below the others: 2^-138 of their weight
    fs.fs_cache_write(cache, table.cuda(), torch.arange(m, dtype=torch.int32)[None].cuda(), kk.cuda(), vv.cuda())
    k[:, :m], v[:, :m] = values_of(kk, held), values_of(vv, held)
    check(q, cache, table, k, v, [ctx])


@pytest.mark.parametrize("held", EIGHT)
@pytest.mark.parametrize("n,H,d", [(2, 8, 64), (20, 8, 64), (20, 8, 128), (30, 8, 128), (70, 8, 64), (70, 8, 128)])
@pytest.mark.parametrize("size", [45, 100, -45, -120])
def test_one_large_query_leaves_its_neighbours(held, n, H, d, size):
    """Queries of one token, or of one head, times 2^size: no other row notices."""
    ctx = [150]
    q, cache, table, k, v = setting(n, 1, n, ctx, H, 2, d, BF, held, 16)
    q[0, n // 2] *= 2.0 ** size
    check(q, cache, table, k, v, ctx)
    # one head of a token; what others get is as without it
    q, *_ = setting(n, 1, n, ctx, H, 2, d, BF, held, 16)
    a, la = attend(q, cache, table, ctx, None)
    q[0, n // 2, 1] *= 2.0 ** size
    b, lb = attend(q, cache, table, ctx, None)
    a[0, n // 2, 1] = b[0, n // 2, 1] = 0
    la[0, 1, n // 2] = lb[0, 1, n // 2] = 0
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("held", EIGHT)
@pytest.mark.parametrize("dtype", [BF, HALF])
@pytest.mark.parametrize("n,H,G,d", [(1, 8, 2, 128), (20, 8, 2, 64), (20, 8, 2, 128), (30, 8, 2, 64), (30, 8, 2, 128),
                                     (70, 8, 2, 64), (70, 8, 2, 128)])
@pytest.mark.parametrize("first", [0, 500])
def test_large_queries_and_scales_apart_over_many_tiles(held, dtype, n, H, G, d, first):
    """Both at once, from some tile on, with a tree and padding: every loop of a block, one after the other."""
    ctx = [900, 333]
    q, cache, table, k, v = setting(n, 2, n, ctx, H, G, d, dtype, held, 32)
    g = gen(n + first)
    m = max(ctx) + n
    if dtype == BF:
        q[0, n // 3, 1] *= 2.0 ** 50
    kk, vv = (torch.randn(2, m, G, d, generator=g).to(dtype) for _ in range(2))
    vv[:, first::5] = 0
    if dtype == BF:
        vv[:, first + 3::7] *= 2.0 ** 40
    at = torch.arange(m, dtype=torch.int32).expand(2, m).clone()
    for b in range(2):
        at[b, ctx[b] + n:] = -1
    fs.fs_cache_write(cache, table.cuda(), at.cuda(), kk.cuda(), vv.cuda())
    k[:, :m], v[:, :m] = values_of(kk, held), values_of(vv, held)
    check(q, cache, table, k, v, ctx, random_parents(g, 2, n, absent=n // 8))


@pytest.mark.parametrize("held", EIGHT)
@pytest.mark.parametrize("n", [1, 20])
def test_small_elements_of_a_query(held, n):
    """Elements 2^-26 of a row's largest that meet the only large elements of the keys."""
    ctx = [150]
    q, cache, table, k, v = setting(n, 1, n, ctx, 4, 2, 64, BF, held, 16)
    m = ctx[0] + n
    g = gen(m)
    q[..., 1:] *= 2.0 ** -26
    q[..., 0] = 1.0
    kk = (torch.randn(1, m, 2, 64, generator=g) * 2.0 ** 24).bfloat16()
    kk[..., 0] = 0
    vv = torch.randn(1, m, 2, 64, generator=g).bfloat16()
    fs.fs_cache_write(cache, table.cuda(), torch.arange(m, dtype=torch.int32)[None].cuda(), kk.cuda(), vv.cuda())
    k[:, :m], v[:, :m] = values_of(kk, held), values_of(vv, held)
    check(q, cache, table, k, v, ctx)


# --- angles -------------------------------------------------------------------

TURN = Fraction("0.159154943091895335768883763372514362034459645740456448747667344058896797634226535")    # 1 / 2 pi


def exact_rotary(x, freqs, pos, interleaved, back):
    """(result, bound) of rotary64, its angles from whole numbers.  Beside a float32 angle's bound
    the 2^-32 turns that a position's angle is cut at: 2 pi 2^-32, within its margin."""
    half = freqs.numel()
    turns = torch.tensor([[[float((int(p) * Fraction(float(w)) * TURN) % 1) for w in freqs] for p in row]
                          for row in pos], dtype=torch.float64)
    near = turns * (2 * math.pi)
    want, tol = rotary64(x, torch.ones(half, dtype=torch.float64), torch.zeros_like(pos), interleaved, 1.0, back)
    c, s = torch.cos(near)[:, :, None], torch.sin(near)[:, :, None] * (-1.0 if back else 1.0)
    at = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    a, b = x.double()[..., at[0]], x.double()[..., at[1]]
    want[..., at[0]], want[..., at[1]] = a * c - b * s, a * s + b * c
    u = torch.finfo(x.dtype).eps / 2
    tol[..., at[0]] = tol[..., at[1]] = 2.0 ** -21 * (a.abs() + b.abs())
    tol[..., :2 * half] += u * want[..., :2 * half].abs() + 2.0 ** -25
    return want, tol


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d", [16, 17])
def test_rotary_of_frequencies_of_any_size(interleaved, d):
    g = gen(d)
    w = torch.tensor([1e6 + 0.3, 1e9, -3.7e5, 2.0 ** 40 - 1.5, 1e-9, -1e-12, 6.283185307179586, 0.0],
                     dtype=torch.float64)
    pos = torch.tensor([[0, 1, -1, 10 ** 6, 2 ** 31 - 1, -(2 ** 31), 123456789]], dtype=torch.int32)
    q = torch.randn(1, 7, 3, d, generator=g).half()
    for fn, back in ((fs.fs_rotary, False), (fs.fs_rotary_grad, True)):
        got, _ = fn(q.cuda(), None, w.cuda(), pos.cuda(), interleaved=interleaved)
        within(got, *exact_rotary(q, w, pos, interleaved, back), "rotary")


@pytest.mark.parametrize("d", [16, 21])
@pytest.mark.parametrize("bad", [NAN, math.inf, -math.inf])
def test_rotary_of_frequencies_that_are_not_numbers(d, bad):
    g = gen(d)
    w = torch.tensor([1.0, bad, 0.01, 0.001], dtype=torch.float64)
    pos = torch.tensor([[0, 1, 2, 3]], dtype=torch.int32)
    q = torch.randn(1, 4, 2, d, generator=g).bfloat16()
    got = fs.fs_rotary(q.cuda(), None, w.cuda(), pos.cuda())[0].cpu()
    assert bool(torch.isnan(got[..., [1, 5]]).all())
    w[1] = 0.1
    fine = fs.fs_rotary(q.cuda(), None, w.cuda(), pos.cuda())[0].cpu()
    rest = [c for c in range(d) if c not in (1, 5)]
    assert torch.equal(got[..., rest], fine[..., rest])


# --- ends of blocks, rows that are padded ----------------------------------------

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,n,H,G,d,rotary,skew", [
    (1, 8197, 2, 1, 32, 32, False), (3, 2777, 3, 1, 40, 16, False), (1, 2051, 2, 2, 24, 16, False),
    (1, 3001, 2, 1, 17, 8, False), (2, 4103, 2, 1, 16, 16, True), (1, 6149, 1, 0, 9, 2, False)])
def test_rotary_of_blocks_that_end_short(interleaved, B, n, H, G, d, rotary, skew):
    """Several tokens to a block, the last block with fewer; rows that take 16-byte accesses and others."""
    g = gen(n)
    q, k = (torch.randn(B, n, h, d, generator=g).bfloat16() for h in (H, G))
    pos = torch.randint(0, 100000, (B, n), generator=g, dtype=torch.int32)
    w = torch.from_numpy(fs.fs_rotary_frequencies(rotary))

    def there(x):
        if not skew:
            return x.cuda()
        y = torch.zeros(*x.shape[:3], d + 3, dtype=BF, device="cuda")[..., 1:d + 1]
        y.copy_(x)
        return y

    for fn, back in ((fs.fs_rotary, False), (fs.fs_rotary_grad, True)):
        got = fn(there(q), there(k) if G else None, w.cuda(), pos.cuda(), interleaved=interleaved)
        for x, y in zip((q, k), got):
            if y is not None:
                within(y, *rotary64(x, w, pos, interleaved, 1.0, back), "rotary")


@pytest.mark.parametrize("held", EIGHT)
@pytest.mark.parametrize("dtype", [BF, HALF])
@pytest.mark.parametrize("B,n,ctx,H,G,d,page", [
    (2, 9, [70, 33], 8, 2, 8, 16), (1, 40, [200], 4, 1, 24, 8), (2, 27, [333, 90], 10, 2, 72, 16),
    (1, 100, [190], 4, 2, 72, 64), (1, 60, [1000], 8, 1, 104, 32), (2, 2, [300, 9], 4, 2, 72, 16)])
def test_rows_that_are_padded_to_whole_pieces(held, dtype, B, n, ctx, H, G, d, page):
    """Heads of no multiple of 16, as fs_cache_new lays them out: the padding of the rows may hold anything."""
    g = gen(n + d)
    per = -(-(max(ctx) + n) // page)
    cache = fs.fs_cache_new(B * per + 1, G, page, d, held)
    wide = cache.k.stride(2)
    for x in (cache.k, cache.v):
        x.as_strided((B * per + 1, G, page, wide), x.stride()).view(torch.int8).fill_(0x7f)
    for x in (cache.k_scale, cache.v_scale):
        x.fill_(NAN)
    table = torch.randperm(B * per + 1, generator=g)[:B * per].int().view(B, per)
    k, v = (torch.randn(B, per * page, G, d, generator=g).to(dtype) for _ in range(2))
    at = torch.arange(per * page, dtype=torch.int32).expand(B, -1).clone()
    for b in range(B):
        at[b, ctx[b] + n:] = -1
    fs.fs_cache_write(cache, table.cuda(), at.cuda(), k.cuda(), v.cuda())
    q = (2 * torch.randn(B, n, H, d, generator=g)).to(dtype)
    parents = random_parents(gen(n), B, n, absent=n // 5)
    check(q, cache, table, values_of(k, held), values_of(v, held), ctx, parents)
