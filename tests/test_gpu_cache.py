"""Rotary positions, the cache in pages and the attention of drafted trees on the GPU,
against their definitions in 64 bits (kv_ref)."""
import math

import pytest
import torch

from streaming_sinkhorn_solver_gb300 import binding as fs
from tests.kv_ref import quantise, rotary64, sees, tree64

pytestmark = pytest.mark.gpu
BF, HALF, E4M3, I8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.int8
NAN = math.nan


def gen(seed):
    return torch.Generator().manual_seed(seed)


def within(got, want, tol, name):
    got = got.detach().cpu().double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine) and torch.equal(got[~fine & ~torch.isnan(want)],
                                                                  want[~fine & ~torch.isnan(want)]), name
    off = ((got - want).abs() - tol)[fine]
    assert off.numel() == 0 or float(off.max()) <= 0, f"{name}: {float(off.max())} beyond the bound"


# --- rotary positions ---------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, HALF])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,n,H,G,d,rotary", [
    (1, 1, 4, 2, 64, 64), (2, 37, 8, 1, 128, 128), (3, 5, 6, 3, 80, 40), (1, 9, 5, 5, 72, 18),
    (2, 3, 1, 1, 7, 2), (1, 4200, 2, 1, 32, 16), (2, 2, 2, 0, 24, 24)])
def test_rotary(dtype, interleaved, B, n, H, G, d, rotary):
    g = gen(n)
    q, k = (torch.randn(B, n, h, d, generator=g).to(dtype) for h in (H, G))
    pos = torch.randint(0, 100000, (B, n), generator=g, dtype=torch.int32)
    w = torch.from_numpy(fs.fs_rotary_frequencies(rotary))
    amp = 1.0 if n % 2 else 0.8
    how = dict(interleaved=interleaved, amplitude=amp)
    for fn, back in ((fs.fs_rotary, False), (fs.fs_rotary_grad, True)):
        got = fn(q.cuda(), k.cuda() if G else None, w.cuda(), pos.cuda(), **how)
        for x, y in zip((q, k), got):
            if y is not None:
                within(y, *rotary64(x, w, pos, interleaved, amp, back), "rotary")
        assert (got[1] is None) == (G == 0)


def test_rotary_of_far_and_negative_positions():
    g = gen(1)
    q = torch.randn(1, 8, 2, 64, generator=g).half()
    pos = torch.tensor([[0, -1, 2 ** 20 + 1, 2 ** 24 + 1, 2 ** 30 + 7, -(2 ** 30) - 3, 2 ** 31 - 1, 77777777]],
                       dtype=torch.int32)
    w = torch.from_numpy(fs.fs_rotary_frequencies(64))
    got, _ = fs.fs_rotary(q.cuda(), None, w.cuda(), pos.cuda())
    within(got, *rotary64(q, w, pos), "far")


def test_rotary_in_place_strides_and_shared_positions():
    g = gen(2)
    qkv = torch.randn(2, 11, 6, 64, generator=g).bfloat16().cuda()
    w = torch.from_numpy(fs.fs_rotary_frequencies(32)).cuda()
    pos = torch.arange(11, dtype=torch.int32, device="cuda") + 5
    q, k = qkv[:, :, :3], qkv[:, :, 3:5]
    want_q, want_k = fs.fs_rotary(q.contiguous(), k.contiguous(), w, pos)
    # other strides, results too; one row of positions for all
    heads_first = torch.empty(2, 3, 11, 64, dtype=BF, device="cuda").transpose(1, 2)
    odd = torch.empty(2, 11, 2, 67, dtype=BF, device="cuda")[..., 1:65]
    a, b = fs.fs_rotary(q, k, w, pos.expand(2, 11), q_out=heads_first, k_out=odd)
    assert a is heads_first and b is odd
    assert torch.equal(a, want_q) and torch.equal(b, want_k)
    # the same from rows that are not aligned
    skew = torch.empty(2, 11, 6, 65, dtype=BF, device="cuda")[..., :64]
    skew.copy_(qkv)
    a, _ = fs.fs_rotary(skew[:, :, :3], None, w, pos)
    assert torch.equal(a, want_q)
    # in place, and nothing beside the queries and keys is touched
    rest = qkv[:, :, 5:].clone()
    fs.fs_rotary(q, k, w, pos, q_out=q, k_out=k)
    assert torch.equal(q, want_q) and torch.equal(k, want_k) and torch.equal(qkv[:, :, 5:], rest)


def test_rotary_gradient_is_the_transpose():
    g = gen(3)
    q, dy = (torch.randn(2, 6, 4, 48, generator=g).half().cuda() for _ in range(2))
    w = torch.from_numpy(fs.fs_rotary_frequencies(24)).cuda()
    pos = torch.randint(0, 5000, (2, 6), generator=g, dtype=torch.int32).cuda()
    y, _ = fs.fs_rotary(q, None, w, pos, interleaved=True, amplitude=1.25)
    dq, _ = fs.fs_rotary_grad(dy, None, w, pos, interleaved=True, amplitude=1.25)
    a, b = (y.double() * dy.double()).sum(), (q.double() * dq.double()).sum()
    # each element rounded once: u |y| |dy| summed, twice over for both sides
    u = 2.0 ** -11
    assert abs(float(a - b)) <= 1.1 * u * float((y.double() * dy.double()).abs().sum() +
                                                (q.double() * dq.double()).abs().sum())
    # differences along one direction: a linear map, so whole steps
    e = torch.randn(q.shape, generator=gen(4)).half().cuda()
    up, _ = fs.fs_rotary(q + e, None, w, pos, interleaved=True, amplitude=1.25)
    step = ((up.double() - y.double()) * dy.double()).sum()
    want = ((q + e - q.double()) * dq.double()).sum()
    mass = ((up.double().abs() + y.double().abs()) * dy.double().abs()).sum()
    mass += ((q + e).double().abs() * dq.double().abs()).sum() * 2
    assert abs(float(step - want)) <= 1.1 * u * float(mass)


def test_rotary_of_nothing():
    q = torch.zeros(0, 3, 2, 8, dtype=BF, device="cuda")
    w = torch.zeros(4, dtype=torch.float64, device="cuda")
    y, _ = fs.fs_rotary(q, None, w, torch.zeros(0, 3, dtype=torch.int32, device="cuda"))
    assert y.shape == q.shape


# --- the cache ----------------------------------------------------------------

def pool(held, pages, G, page, d, fill=NAN, order="head"):
    """A cache whose rows are all `fill` (codes: a NaN's, or -128), of two layouts."""
    def rows():
        shape = (pages, G, page, d) if order == "head" else (pages, page, G, d)
        if held == I8:
            x = torch.full(shape, -128, dtype=I8, device="cuda")
        elif held == E4M3:
            x = torch.full(shape, 0x7f, dtype=torch.uint8, device="cuda").view(E4M3)
        else:
            x = torch.full(shape, fill, dtype=held, device="cuda")
        return x if order == "head" else x.transpose(1, 2)
    if held in (E4M3, I8):
        return fs.KVCache(rows(), rows(), *(torch.full((pages, G, page), fill, device="cuda")
                                            for _ in range(2)))
    return fs.KVCache(rows(), rows())


def bits(x):
    return x.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()]).cpu()


@pytest.mark.parametrize("held", [None, E4M3, I8])
@pytest.mark.parametrize("dtype", [BF, HALF])
@pytest.mark.parametrize("order", ["head", "token"])
@pytest.mark.parametrize("B,n,G,d,page", [(1, 1, 1, 64, 16), (3, 37, 2, 128, 16), (2, 70, 3, 72, 8),
                                          (2, 9, 4, 32, 64)])
def test_write_and_read(held, dtype, order, B, n, G, d, page):
    g = gen(B * n + d)
    held = held or dtype
    per = 3 + n // page
    pages = B * per + 2
    cache = pool(held, pages, G, page, d, order=order)
    before = [bits(x) for x in cache if x is not None]
    table = torch.randperm(pages, generator=g)[:B * per].int().view(B, per)
    table[0, 1] = -1 if n % 2 else pages          # no page there
    k, v = (torch.randn(B, n, 2 * G, d, generator=g).to(dtype)[:, :, ::2] for _ in range(2))
    k[0, 0] *= 2.0 ** -14
    v[-1, -1] = 0
    if n > 1:
        k[0, 1, 0, 3], v[0, 1, 0, 5] = NAN, math.inf
    # distinct positions in any order, some beyond the table; some tokens are left out
    at = torch.stack([torch.randperm(per * page + 9, generator=g)[:n] for _ in range(B)]).int()
    at[torch.rand(B, n, generator=g) < 0.2] = -3
    fs.fs_cache_write(cache, table.cuda(), at.cuda(), k.cuda(), v.cuda())
    want = {}
    for name, x in (("k", k), ("v", v)):
        rows = getattr(cache, name).cpu()
        code, scale = (x, None) if held == dtype else quantise(x, held)
        want[name] = torch.zeros(B, per * page, G, d, dtype=dtype)
        touched = torch.zeros(pages, page, dtype=torch.bool)
        for b in range(B):
            for t in range(n):
                p = int(at[b, t])
                where = int(table[b, p // page]) if 0 <= p < per * page else -1
                if not 0 <= where < pages:
                    continue
                touched[where, p % page] = True
                assert torch.equal(bits(rows[where, :, p % page]), bits(code[b, t])), (name, b, t)
                if scale is None:
                    want[name][b, p] = x[b, t]
                else:
                    s = getattr(cache, name + "_scale").cpu()[where, :, p % page]
                    assert torch.equal(bits(s), bits(scale[b, t])), (name, b, t)
                    want[name][b, p] = (code[b, t].float() * scale[b, t][:, None]).to(dtype)
        # every other row is as it was
        now = bits(getattr(cache, name)).view(pages, G, page, d)
        old = before[0 if name == "k" else 1].view(pages, G, page, d)
        assert torch.equal(now.transpose(1, 2)[~touched], old.transpose(1, 2)[~touched])
    # what no token was written to holds NaN: set aside in the comparison
    lens = torch.tensor([per * page - 5 * b for b in range(B)], dtype=torch.int32)
    got = fs.fs_cache_read(cache, table.cuda(), lens.cuda(), dtype=dtype)
    for name, y in zip("kv", got):
        y = y.cpu()
        for b in range(B):
            written = {int(p) for p in at[b] if p >= 0}
            for p in range(per * page):
                where = int(table[b, p // page])
                if p >= int(lens[b]) or not 0 <= where < pages:
                    assert not bits(y[b, p]).any(), (name, b, p)
                elif p in written:
                    a, w = y[b, p], want[name][b, p]
                    nan = torch.isnan(w)
                    assert torch.equal(torch.isnan(a), nan) and torch.equal(a[~nan], w[~nan]), (name, b, p)


def test_reading_other_types_and_given_tensors():
    g = gen(5)
    cache = fs.fs_cache_new(4, 2, 16, 64, E4M3)
    table = torch.tensor([[2, 0], [3, 1]], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(2, 20, 2, 64, generator=g).bfloat16().cuda() for _ in range(2))
    at = torch.arange(20, dtype=torch.int32, device="cuda").expand(2, 20)
    fs.fs_cache_write(cache, table, at, k, v)
    a, b = fs.fs_cache_read(cache, table, n=20)
    assert a.dtype == BF and a.shape == k.shape
    # e4m3 has 4 bits: half a step of 2^-4 relative, or of the smallest step 2^-9 scale
    scale = k.float().abs().amax(-1, keepdim=True) / 448
    assert bool(((a.float() - k.float()).abs() <= (2.0 ** -4 + 2.0 ** -8) * k.float().abs() +
                 2.0 ** -10 * scale).all())
    mine = [torch.empty(2, 2, 20, 67, dtype=HALF, device="cuda")[..., :64].transpose(1, 2) for _ in range(2)]
    got = fs.fs_cache_read(cache, table, n=20, dtype=HALF, k=mine[0], v=mine[1])
    assert got[0] is mine[0]
    whole, _ = fs.fs_cache_read(cache, table, n=20, dtype=HALF)
    assert torch.equal(mine[0], whole)
    # past the table: zeros
    far, _ = fs.fs_cache_read(cache, table, n=50)
    assert torch.equal(far[:, :20], a) and not far[:, 32:].any()


def test_expanded_positions_are_refused_where_rows_overlap():
    cache = pool(BF, 2, 1, 16, 64)
    wide = fs.KVCache(cache.k[:, :, :1].expand(2, 1, 16, 64), cache.v)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    k = torch.zeros(1, 1, 1, 64, dtype=BF, device="cuda")
    at = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    with pytest.raises(fs.FlashSinkhornError):
        fs.fs_cache_write(wide, table, at, k, k)
    skew = torch.zeros(2, 1, 16, 67, dtype=BF, device="cuda")[..., 1:65]
    with pytest.raises(fs.FlashSinkhornError):
        fs.fs_cache_write(fs.KVCache(skew, cache.v), table, at, k, k)


# --- tree attention -----------------------------------------------------------

def setting(seed, B, n, ctx, H, G, d, dtype, held, page, spare=2, order="head", tail=NAN):
    """A cache filled through the library from random rows, everything else in it NaN."""
    g = gen(seed)
    m = max(max(ctx), 0) + n
    per = -(-m // page)
    pages = B * per + spare
    cache = pool(held, pages, G, page, d, fill=tail, order=order)
    table = torch.randperm(pages, generator=g)[:B * per].int().view(B, per)
    k, v = (torch.randn(B, per * page, G, d, generator=g).to(dtype) for _ in range(2))
    at = torch.arange(per * page, dtype=torch.int32).expand(B, -1).clone()
    for b in range(B):
        at[b, max(ctx[b], 0) + n:] = -1
    fs.fs_cache_write(cache, table.cuda(), at.cuda(), k.cuda(), v.cuda())
    if held != dtype:
        k, v = ((c.float() * s[..., None]).double() for c, s in (quantise(x, held) for x in (k, v)))
    q = (2 * torch.randn(B, n, H, d, generator=g)).to(dtype)
    return q, cache, table, k, v


def random_parents(g, B, n, absent=0):
    p = torch.tensor([[int(torch.randint(-1, t, (1,), generator=g)) if t else -1 for t in range(n)]
                      for _ in range(B)], dtype=torch.int32)
    if absent:
        p[:, -absent:] = -2
    return p


def check(q, cache, table, k, v, ctx, parents=None, there=None, **how):
    held = cache.k.dtype
    got, lse = fs.fs_tree_attention(
        q.cuda() if not q.is_cuda else q, cache, table.cuda(), torch.tensor(ctx, dtype=torch.int32).cuda(),
        None if parents is None else parents.cuda(), **how)
    fs.fs_check()
    if there is None:
        there = torch.ones(k.shape[:2], dtype=torch.bool)
    want = tree64(q, k, v, there, ctx, parents, how.get("scale"),
                  weights=HALF if held in (E4M3, I8) else None)
    within(got, want["out"], want["tol"]["out"], "out")
    within(lse, want["lse"], want["tol"]["lse"], "lse")
    return got, lse


SIZES = [   # B, n, ctx, H, G, d, page
    (1, 1, [0], 1, 1, 64, 16),
    (1, 1, [1], 4, 1, 128, 16),
    (3, 1, [300, 17, 0], 8, 2, 64, 16),
    (2, 5, [129, 640], 4, 2, 128, 32),
    (2, 3, [1000, 15], 15, 5, 80, 8),
    (1, 13, [77], 8, 4, 96, 64),
    (2, 27, [333, 90], 10, 2, 72, 16),
    (1, 64, [200], 16, 2, 64, 16),
    (2, 40, [130, 64], 8, 1, 128, 128),
    (1, 100, [63], 6, 2, 32, 16),
    (1, 256, [70], 4, 2, 48, 64),
    (2, 9, [70, 33], 8, 2, 8, 16),
    (1, 5, [100], 16, 1, 24, 8),
    (1, 3, [1500], 8, 1, 64, 1024),
]


@pytest.mark.parametrize("held", [None, E4M3, I8])
@pytest.mark.parametrize("dtype", [BF, HALF])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "-".join(map(str, s)).replace(" ", ""))
def test_tree_attention(held, dtype, size):
    B, n, ctx, H, G, d, page = size
    s = setting(n + d, B, n, ctx, H, G, d, dtype, held or dtype, page)
    parents = None if n == 1 else random_parents(gen(n), B, n, absent=n // 5)
    check(*s, ctx, parents)


@pytest.mark.parametrize("held", [BF, E4M3])
@pytest.mark.parametrize("n", [1, 9, 70])
def test_chain_is_causal(held, n):
    ctx = [50, 0, 131]
    s = setting(n, 3, n, ctx, 6, 3, 64, BF, held, 16)
    a, la = check(*s, ctx)
    b, lb = check(*s, ctx, torch.arange(-1, n - 1, dtype=torch.int32))      # one tree for all
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("held", [HALF, E4M3, I8])
@pytest.mark.parametrize("n", [2, 24])
def test_strides_layouts_and_given_results(held, n):
    ctx = [90, 33]
    q, *s = setting(3, 2, n, ctx, 8, 2, 80, HALF, held, 16, order="token")
    parents = random_parents(gen(1), 2, n)
    wide = torch.zeros(2, n, 12, 80, dtype=HALF)
    wide[:, :, 2:10] = q
    out = torch.full((2, 8, n, 83), 7.0, dtype=HALF, device="cuda")[..., :80].transpose(1, 2)
    a, _ = check(q, *s, ctx, parents)
    b, _ = check(wide.cuda()[:, :, 2:10], *s, ctx, parents, out=out)
    assert b is out and torch.equal(a, b)
    # rows of queries that are not aligned
    skew = torch.zeros(2, n, 8, 83, dtype=HALF, device="cuda")[..., 1:81]
    skew.copy_(q)
    lse = torch.empty(2, 8, n, device="cuda")
    c, got = check(skew, *s, ctx, parents, lse=lse)
    assert torch.equal(a, c) and got is lse


@pytest.mark.parametrize("held", [BF, E4M3, I8])
@pytest.mark.parametrize("n", [1, 30])
def test_missing_pages_and_short_tables(held, n):
    ctx = [200, 100, 999, -4]
    q, cache, table, k, v = setting(6, 4, n, [200, 100, 220, 0], 8, 2, 64, BF, held, 16)
    m = table.shape[1] * 16
    there = torch.ones(4, m, dtype=torch.bool)
    for b, i, x in ((0, 1, -1), (0, 5, 10 ** 9), (1, 0, cache.k.shape[0]), (0, (200 + n) // 16, -7)):
        table[b, i] = x
        there[b, 16 * i:16 * i + 16] = False
    # sequence 2 is said to be longer than its table, whose end it reaches: its unwritten
    # rows are taken off the table
    written = 220 + n
    table[2, written // 16:] = -1
    there[2, written // 16 * 16:] = False
    check(q, cache, table, k, v, ctx, there=there)
    none = torch.full_like(table, -1)
    out, lse = check(q, cache, none, k, v, ctx, there=torch.zeros_like(there))
    assert not out.any() and bool((lse == -math.inf).all())
    empty = table[:, :0]
    out, lse = check(q, cache, empty, k[:, :0], v[:, :0], ctx, there=there[:, :0])
    assert not out.any()


@pytest.mark.parametrize("held", [BF, HALF, E4M3, I8])
@pytest.mark.parametrize("n,H", [(4, 2), (40, 8)])
def test_values_of_others_never_reach_a_row(held, n, H):
    """NaN and infinities in keys and values that a token does not see, in padding and behind
    the end; those that it sees make its row NaN."""
    dtype = held if held in (BF, HALF) else BF
    ctx = [100, 61]
    q, cache, table, k, v = setting(8, 2, n, ctx, H, 2, 64, dtype, held, 16)
    parents = torch.full((2, n), -1, dtype=torch.int32)     # children of the context alone
    parents[:, n - 1] = 0
    bad = n // 2
    rows = torch.full((2, 1, 2, 64), 1.0, dtype=dtype)
    rows[0, 0, :, 7], rows[1, 0, :, 9] = NAN, math.inf
    at = torch.tensor([[c + bad] for c in ctx], dtype=torch.int32)
    for which in ("k", "v"):
        fine = torch.ones_like(rows)
        fs.fs_cache_write(cache, table.cuda(), at.cuda(), *((rows.cuda(), fine.cuda()) if which == "k"
                                                            else (fine.cuda(), rows.cuda())))
        for b in range(2):
            k[b, ctx[b] + bad] = v[b, ctx[b] + bad] = 1.0
        out, lse = fs.fs_tree_attention(q.cuda(), cache, table.cuda(),
                                        torch.tensor(ctx, dtype=torch.int32).cuda(), parents.cuda())
        others = [t for t in range(n) if t != bad]
        there = torch.ones(k.shape[:2], dtype=torch.bool)
        if held in (E4M3, I8):      # the row of ones as it is held
            code, scale = quantise(fine.cpu(), held)
            one = float(code[0, 0, 0, 0].float() * scale[0, 0, 0])
            for b in range(2):
                k[b, ctx[b] + bad] = v[b, ctx[b] + bad] = one
        want = tree64(q, k, v, there, ctx, parents, weights=HALF if held in (E4M3, I8) else None)
        within(out[:, others], want["out"][:, others], want["tol"]["out"][:, others], which)
        within(lse[:, :, others], want["lse"][:, :, others], want["tol"]["lse"][:, :, others], which)
        if which == "v":
            assert bool(torch.isnan(out[:, bad]).all())
        else:
            assert bool((~torch.isfinite(out[:, bad])).any(-1).any())


@pytest.mark.parametrize("held", [BF, E4M3])
@pytest.mark.parametrize("n", [3, 33])
def test_tokens_that_are_not_there(held, n):
    ctx = [40, 40]
    q, *s = setting(9, 2, n, ctx, 8, 2, 128, BF, held, 16)
    q[:, 1] = NAN
    parents = random_parents(gen(2), 2, n)
    parents[0, 1], parents[1, 1] = -2, 1
    parents[0, 2] = 1                               # a child of one that is not there
    parents[1, 2] = n + 5
    out, lse = check(q, *s, ctx, parents)
    assert not out[:, 1:3].any() and bool((lse[:, :, 1:3] == -math.inf).all())
    all_gone = torch.full((2, n), -2, dtype=torch.int32)
    out, lse = check(q, *s, ctx, all_gone)
    assert not out.any()


@pytest.mark.parametrize("held", [BF, E4M3, I8])
@pytest.mark.parametrize("n", [1, 20, 64])
def test_long_contexts_are_split_and_joined(held, n):
    ctx = [9000, 4100]
    s = setting(11, 2, n, ctx, 4, 1, 64, BF, held, 64)
    parents = random_parents(gen(3), 2, n)
    a, la = check(*s, ctx, parents)
    b, lb = check(*s, ctx, parents)
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("held", [BF, HALF, E4M3, I8])
@pytest.mark.parametrize("n,R,d", [(9, 4, 128), (9, 4, 64), (20, 8, 128), (20, 8, 64), (1, 2, 128)])
def test_blocks_of_many_tiles(held, n, R, d):
    """As many sequences and key heads as the GPU has SMs: every ring of a block goes round
    several times, with contexts that end anywhere."""
    G = 4
    B = torch.cuda.get_device_properties(0).multi_processor_count // G
    dtype = held if held in (BF, HALF) else BF
    ctx = [1300 - 19 * b for b in range(B)]
    s = setting(16, B, n, ctx, R * G, G, d, dtype, held, 32)
    parents = random_parents(gen(5), 1, n)[0]
    check(*s, ctx, parents)


@pytest.mark.parametrize("n", [1, 32])
def test_scales_that_differ_widely(n):
    """Values of a key may be 2^30 times those of another: each weighs in by its own."""
    ctx = [300]
    q, cache, table, k, v = setting(12, 1, n, ctx, 4, 2, 64, BF, E4M3, 16)
    g = gen(4)
    e = torch.randint(-40, 40, (300 + n, 2), generator=g)
    rows = torch.randn(1, 300 + n, 2, 64, generator=g)
    vv = (rows * torch.exp2(e.float())[None, :, :, None]).bfloat16()
    kk = torch.randn(1, 300 + n, 2, 64, generator=g).bfloat16()
    at = torch.arange(300 + n, dtype=torch.int32)[None]
    fs.fs_cache_write(cache, table.cuda(), at.cuda(), kk.cuda(), vv.cuda())
    for x, y in ((k, kk), (v, vv)):
        code, scale = quantise(y, E4M3)
        x[:, :300 + n] = code.double() * scale.double()[..., None]
    check(q, cache, table, k, v, ctx)
    # one value of 2^40 that hardly weighs beside many small ones that do
    kk[:, :, :, :] = 0
    vv = rows.bfloat16()
    vv[0, 5] *= 2.0 ** 40
    kk[0, 5] = -q[0, 0, 0].sign()[None]
    q[0] = (q[0, :1, :1].sign() * 4).expand_as(q[0]).contiguous()
    fs.fs_cache_write(cache, table.cuda(), at.cuda(), kk.cuda(), vv.cuda())
    for x, y in ((k, kk), (v, vv)):
        code, scale = quantise(y, E4M3)
        x[:, :300 + n] = code.double() * scale.double()[..., None]
    check(q, cache, table, k, v, ctx)


@pytest.mark.parametrize("held", [BF, E4M3])
@pytest.mark.parametrize("n", [2, 48])
def test_queries_of_any_size(held, n):
    ctx = [150]
    q, cache, table, k, v = setting(13, 1, n, ctx, 4, 2, 64, BF, held, 16)
    q[0, 0] *= 2.0 ** -100
    q[0, 1, 0] *= 2.0 ** 3
    q[0, 1, 1] = 0
    check(q, cache, table, k, v, ctx)
    check(q, cache, table, k, v, ctx, scale=1e-3)


@pytest.mark.parametrize("n", [1, 50])
def test_streams_and_graphs(n):
    ctx = [700, 300]
    q, cache, table, k, v = setting(14, 2, n, ctx, 8, 2, 64, BF, E4M3, 16)
    w = torch.from_numpy(fs.fs_rotary_frequencies(64)).cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    tree = torch.arange(-1, n - 1, dtype=torch.int32, device="cuda")
    lens = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    q, table = q.cuda(), table.cuda()
    kk, vv = (torch.randn(2, n, 2, 64, generator=gen(6)).bfloat16().cuda() for _ in range(2))

    def step(stream=None):
        a, b = fs.fs_rotary(q, kk, w, pos, stream=stream)
        fs.fs_cache_write(cache, table, (lens[:, None] + pos).int(), b, vv, stream=stream)
        return fs.fs_tree_attention(a, cache, table, lens, tree, stream=stream)

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for x in got:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    # new inputs in the same places
    q.mul_(0.5)
    lens.sub_(7)
    graph.replay()
    torch.cuda.synchronize()
    again = step()
    assert all(torch.equal(x, y) for x, y in zip(got, again))


def test_a_run_of_them_together():
    """A prompt goes into an 8-bit cache, trees of drafts are attended to and their accepted
    chains written behind it, as a server does; against the plain computation."""
    B, H, G, d, page = 2, 4, 2, 64, 16
    g = gen(20)
    cache = fs.fs_cache_new(24, G, page, d, E4M3)
    table = torch.randperm(24, generator=g).int().view(B, 12).cuda()
    w = torch.from_numpy(fs.fs_rotary_frequencies(d))
    lens = [40, 23]
    k, v = (torch.randn(B, 40, G, d, generator=g).bfloat16() for _ in range(2))
    at = torch.arange(40).expand(B, 40).int().clone()
    at[1, 23:] = -1
    turned = fs.fs_rotary(k.cuda(), None, w.cuda(), torch.arange(40, dtype=torch.int32).cuda())[0]
    fs.fs_cache_write(cache, table, at.cuda(), turned, v.cuda())
    known = [(turned[b, :lens[b]].cpu(), v[b, :lens[b]]) for b in range(B)]
    parents = torch.tensor([-1, 0, 0, 2, -1], dtype=torch.int32)
    depth = torch.tensor([0, 1, 1, 2, 0], dtype=torch.int32)
    accepted = [0, 2, 3]
    for _ in range(3):
        n = parents.numel()
        q, dk, dv = (torch.randn(B, n, h, d, generator=g).bfloat16() for h in (H, G, G))
        ctx = torch.tensor(lens, dtype=torch.int32)
        pos = ctx[:, None] + depth
        tq, tk = fs.fs_rotary(q.cuda(), dk.cuda(), w.cuda(), pos.cuda())
        within(tq, *rotary64(q, w, pos), "rotary")
        fs.fs_cache_write(cache, table, (ctx[:, None] + torch.arange(n)).int().cuda(), tk, dv.cuda())
        out, lse = fs.fs_tree_attention(tq, cache, table, ctx.cuda(), parents.cuda())
        m = max(lens) + n
        rows = torch.zeros(2, B, m, G, d, dtype=torch.float64)
        for b in range(B):
            for i, x in enumerate((torch.cat([known[b][0], tk[b].cpu()]), torch.cat([known[b][1], dv[b]]))):
                code, scale = quantise(x, E4M3)
                rows[i, b, :lens[b] + n] = code.double() * scale.double()[..., None]
        want = tree64(tq, rows[0], rows[1], torch.ones(B, m, dtype=torch.bool), lens, parents, weights=HALF)
        within(out, want["out"], want["tol"]["out"], "out")
        within(lse, want["lse"], want["tol"]["lse"], "lse")
        # the accepted chain moves up behind the context
        slots = torch.full((B, n), -1, dtype=torch.int32)
        for i, t in enumerate(accepted):
            slots[:, t] = ctx + i
        fs.fs_cache_write(cache, table, slots.cuda(), tk, dv.cuda())
        known = [(torch.cat([known[b][0], tk[b, accepted].cpu()]), torch.cat([known[b][1], dv[b, accepted]]))
                 for b in range(B)]
        lens = [x + len(accepted) for x in lens]
    # read back, it serves the cross attention of all the queries so far
    back = fs.fs_cache_read(cache, table, torch.tensor(lens, dtype=torch.int32).cuda(), max(lens))
    for b in range(B):
        for x, y in zip(known[b], back):
            code, scale = quantise(x, E4M3)
            assert torch.equal(y[b, :lens[b]].cpu(), (code.float() * scale[..., None]).bfloat16())
    out, _ = fs.fs_cross_attention(tq, *back, kv_len=torch.tensor(lens, dtype=torch.int32).cuda())
    assert bool(torch.isfinite(out).all())


def test_the_first_call_of_a_process_is_like_the_others():
    """Results do not depend on what ran before: the first call splits its keys as later ones do."""
    import os
    import subprocess
    import sys
    code = """
import torch
from tests.test_gpu_cache import *
for held, d in ((E4M3, 64), (I8, 128), (BF, 64)):
    q, cache, table, k, v = setting(14, 2, 1, [700, 300], 8, 2, d, BF, held, 16)
    ctx = torch.tensor([700, 300], dtype=torch.int32).cuda()
    a, b = (fs.fs_tree_attention(q.cuda(), cache, table.cuda(), ctx) for _ in range(2))
    assert all(torch.equal(x, y) for x, y in zip(a, b)), (held, d)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


@pytest.mark.parametrize("held", [BF, E4M3])
def test_nothing_to_do(held):
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    table = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    cache = fs.fs_cache_new(4, 2, 16, 64, held)
    q = torch.ones(2, 3, 4, 64, dtype=BF, device="cuda")
    k = q[:, :, :2]
    fs.fs_cache_write(cache, table, torch.zeros(2, 0, dtype=torch.int32, device="cuda"), k[:, :0], k[:, :0])
    assert not cache.k.float().any()
    a, _ = fs.fs_cache_read(cache, table, n=0)
    assert a.shape == (2, 0, 2, 64)
    out, lse = fs.fs_tree_attention(q[:, :0], cache, table, lens)
    assert out.shape == (2, 0, 4, 64) and lse.shape == (2, 4, 0)
    out, _ = fs.fs_tree_attention(q[:0], cache, table[:0], lens[:0])
    assert out.shape == (0, 3, 4, 64)
    # a pool without pages
    none = fs.fs_cache_new(0, 2, 16, 64, held)
    fs.fs_cache_write(none, table, torch.zeros(2, 3, dtype=torch.int32, device="cuda"), k, k)
    a, _ = fs.fs_cache_read(none, table)
    assert a.shape == (2, 48, 2, 64) and not a.any()
    for n in (1, 3):
        out, lse = fs.fs_tree_attention(q.repeat(1, 1, 4, 1)[:, :n], none, table, lens + 20)
        assert not out.any() and bool((lse == -math.inf).all())


def test_the_example_holds_its_keys_in_8_bits():
    import examples.distill_plan as example
    k, v = (torch.randn(3, 50, example.KEY_HEADS, example.D, generator=gen(30)).bfloat16().cuda()
            for _ in range(2))
    lens = torch.tensor([50, 17, 33], dtype=torch.int32, device="cuda")
    for x, y in zip((k, v), example.held(k, v, lens)):
        code, scale = quantise(x, E4M3)
        want = (code.float() * scale[..., None]).bfloat16()
        for b in range(3):
            assert torch.equal(y[b, :lens[b]].cpu(), want[b, :lens[b]]) and not y[b, lens[b]:].any()


def test_refusals():
    q, cache, table, k, v = setting(15, 2, 3, [20, 30], 4, 2, 64, BF, E4M3, 16)
    q, table = q.cuda(), table.cuda()
    lens = torch.tensor([20, 30], dtype=torch.int32, device="cuda")
    par = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    for bad in (dict(q=q.float()), dict(q=q[..., :32]), dict(q=q[:, :, :3]), dict(q=q.cpu()), dict(q=q[:1]),
                dict(table=table.long()), dict(table=table[:1]), dict(table=table.t()), dict(ctx_len=lens.long()),
                dict(ctx_len=lens[:1]), dict(ctx_len=lens.cpu()), dict(parents=par.long()),
                dict(parents=par[:, :2]), dict(parents=par.cpu()),
                dict(cache=cache._replace(k_scale=None)), dict(cache=cache._replace(v=cache.v[:1])),
                dict(cache=cache._replace(v=cache.v.view(torch.int8))), dict(scale=0.0), dict(scale=math.nan),
                dict(cache=fs.KVCache(cache.k.to(HALF), cache.v.to(HALF))), dict(out=q.float()),
                dict(cache=fs.KVCache(q.new_zeros(2, 2, 16, 64), q.new_zeros(2, 2, 16, 64), *cache[2:])),
                dict(q=torch.zeros(2, 257, 4, 64, dtype=BF, device="cuda"), parents=None),
                dict(out=q[:, :1].expand_as(q)), dict(lse=lens)):
        how = dict(q=q, cache=cache, table=table, ctx_len=lens, parents=par)
        how.update(bad)
        with pytest.raises((TypeError, ValueError, fs.FlashSinkhornError)):
            fs.fs_tree_attention(**how)
    at = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    kk = torch.zeros(2, 3, 2, 64, dtype=BF, device="cuda")
    for bad in (dict(k=kk.float()), dict(k=kk[:, :2]), dict(v=kk.half()), dict(v=kk[:, :, :1]),
                dict(positions=at.long()), dict(positions=at[:, :2]), dict(positions=at.cpu()),
                dict(table=table.cpu())):
        how = dict(cache=cache, table=table, positions=at, k=kk, v=kk)
        how.update(bad)
        with pytest.raises((TypeError, ValueError, fs.FlashSinkhornError)):
            fs.fs_cache_write(**how)
    for bad in (dict(dtype=torch.float32), dict(lens=lens.long()), dict(lens=lens[:1]), dict(n=-1),
                dict(k=kk), dict(table=table.float())):
        how = dict(cache=cache, table=table, lens=lens, n=4)
        how.update(bad)
        with pytest.raises((TypeError, ValueError, fs.FlashSinkhornError)):
            fs.fs_cache_read(**how)
    w = torch.zeros(16, dtype=torch.float64, device="cuda")
    pos = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    for bad in (dict(freqs=w.float()), dict(freqs=w.cpu()), dict(freqs=w[::2]), dict(pos=pos.long()),
                dict(pos=pos[:, :2]), dict(k=kk.half()), dict(k=kk[:1]), dict(amplitude=math.nan),
                dict(freqs=torch.zeros(33, dtype=torch.float64, device="cuda")), dict(freqs=w[:0]),
                dict(q_out=kk), dict(k=None, k_out=kk), dict(q_out=q[:, :1].expand_as(q))):
        how = dict(q=q, k=kk, freqs=w, pos=pos)
        how.update(bad)
        with pytest.raises((TypeError, ValueError, fs.FlashSinkhornError)):
            fs.fs_rotary(**how)
