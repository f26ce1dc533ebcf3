"""Cross attention in float16 over the range of the type: small weights, and gradients of the
sizes that scaled and unscaled losses send back, against 64 bits on the GPU.

float16 holds relative 2^-11 only from 2^-14 up, below that multiples of 2^-24, and nothing
from 65520 on.  The operands of the second products are scaled for that, so the bounds here
grant a weight an absolute error of 2^-32 of its row's largest, and a result its own rounding
(2^-25 where it is subnormal)."""
import math

import pytest
import torch

from streaming_sinkhorn_solver_gb300 import binding as fs
from tests.test_gpu_attention import HF, make

pytestmark = pytest.mark.gpu
F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available()
    fs.load_library()


@pytest.fixture(autouse=True)
def _no_wait_gave_up():
    yield
    fs.fs_check()


def exact(c, how, dout=None):
    """out, the sums of p |v| and |v|, and the gradients by differentiation, in 64 bits."""
    q, k, v = (c[x].to(F64).requires_grad_(dout is not None) for x in ("q", "k", "v"))
    (B, n, H, _), (m, G) = q.shape, k.shape[1:3]
    R = H // G
    z = how["scale"] * torch.einsum("bigrc,bjgc->bgrij", q.unflatten(2, (G, R)), k)
    leaves = [q, k, v]
    if "bias" in how:
        table = how["bias"].to(F64).requires_grad_(dout is not None)
        leaves.append(table)
        D = how["bias_buckets"].numel() // 2
        rel = torch.arange(m, device="cuda")[None] - torch.arange(n, device="cuda")[:, None]
        z = z + table[:, how["bias_buckets"].long()[rel.clamp(-D, D) + D]].unflatten(0, (G, R))
    counts = torch.ones(B, m, dtype=torch.bool, device="cuda")
    if "kv_len" in how:
        counts &= torch.arange(m, device="cuda")[None] < how["kv_len"][:, None]
    if "key_mask" in how:
        counts &= how["key_mask"]
    p = z.masked_fill(~counts[:, None, None, None], -math.inf).softmax(-1)
    out = torch.einsum("bgrij,bjgc->bigrc", p, v).flatten(2, 3)
    with torch.no_grad():
        r = {"out": out.detach(), "lse": torch.logsumexp(
            z.masked_fill(~counts[:, None, None, None], -math.inf), -1).flatten(1, 2),
            "pv": torch.einsum("bgrij,bjgc->bigrc", p, v.abs()).flatten(2, 3),
            "v": v.abs().sum(1).repeat_interleave(R, 1)[:, None]}
    if dout is not None:
        r.update(zip(("dq", "dk", "dv", "dbias"), torch.autograd.grad(out, leaves, dout.to(F64))))
    return r


def check_out(c, how, one=None):
    """`one`: the same call with the entries that c repeats once."""
    out, lse = fs.fs_cross_attention(c["q"], c["k"], c["v"], **how)
    want = exact(one or c, how)
    u = 2.0 ** -11
    # relative error of p from scores of up to 32, summed in float32 over d <= 128 terms
    e = 2 * (128 + 8) * 2.0 ** -24 * 32 + 2.0 ** -16
    tol = u * want["out"].abs() + (u + e) * want["pv"] + 2.0 ** -32 * want["v"] + 2.0 ** -24
    over = (out.to(F64) - want["out"]).abs() - tol
    assert float(over.max()) <= 0, f"{float(over.max()):.3g} over the bound, out about {float(want['out'].mean()):.3g}"
    assert float((lse.to(F64) - want["lse"]).abs().max()) <= e


@pytest.mark.parametrize("B,n,H", [(1, 1, 1), (4097, 1, 1), (1, 300, 1), (1, 300, 80)])
@pytest.mark.parametrize("d", [64, 128])
def test_many_small_weights_reach_the_output(B, n, H, d):
    """One heavy key with value 0 at the start, 200000 keys 18 below it: they bring all that
    `out` holds, 0.3 % of the weight.  (2^-32 each is 1.6 % of that.)  With 4097 sequences
    or 80 heads the keys are not split, and all are weighted against the heavy one."""
    m = 200001
    g = torch.Generator(device="cuda").manual_seed(51)
    c = {x: torch.zeros(1, t, 1, d, dtype=HF, device="cuda") for x, t in (("q", n), ("k", m), ("v", m))}
    c["q"][..., 0], c["k"][:, 0, :, 0] = 6.0, 3.0
    c["v"][:, 1:] = (0.5 + torch.rand(1, m - 1, 1, d, generator=g, device="cuda")).to(HF)
    many = {x: y.expand(B, -1, H if x == "q" else 1, -1) for x, y in c.items()}
    check_out(many, dict(scale=1.0), c)


@pytest.mark.parametrize("n,H,G", [(2, 4, 2), (200, 4, 2)])
def test_spread_scores(n, H, G):
    c, how, _ = make(2, n, 3000, H, G, 64, HF, lens=[3000, 2900], drop=0.1, seed=52, gain=6.0)
    check_out(c, how)


# (n, m): delta from the scores, from out, few blocks with many tiles, sums that many tiles share
SHAPES = [(200, 300, 4, 2, 64, 0), (200, 300, 4, 2, 64, 16), (130, 1500, 4, 2, 128, 0),
          (130, 1500, 4, 2, 80, 16), (40, 3100, 4, 2, 80, 16), (40, 3100, 2, 2, 64, 0),
          (2600, 100, 4, 1, 128, 0), (1, 700, 2, 2, 64, 0)]


@pytest.mark.parametrize("n,m,H,G,d,nb", SHAPES)
@pytest.mark.parametrize("size", [1e-4, 1e-2, 1.0, 1e3])
def test_gradients_of_every_size(n, m, H, G, d, nb, size):
    """Scores of about two standard deviations.  In the 2-norm, 2^-11 at most for the rounding
    of p or ds, as much for the result's own, and 2^-25 for each result that is subnormal."""
    c, how, dout = make(2, n, m, H, G, d, HF, lens=[m, m - m // 3], drop=0.1, nb=nb, far=90, seed=53)
    dout = (size * dout.float()).to(HF)
    check_gradients(c, how, dout, 2.0 ** -10)


@pytest.mark.parametrize("spread", [2.0 ** -10, 2.0 ** 10])
def test_gradients_of_rows_of_unequal_sizes(spread):
    """Every other query's gradient is 2^10 smaller or larger than its neighbour's; each kind by itself."""
    c, how, dout = make(2, 140, 500, 4, 2, 64, HF, seed=54)
    dout = dout.float()
    dout[:, 1::2] *= spread
    got = check_gradients(c, how, dout.to(HF), 2.0 ** -10)
    want = exact(c, how, dout.to(HF))["dq"]
    for part in (slice(0, None, 2), slice(1, None, 2)):
        x, y = got["dq"].to(F64)[:, part], want[:, part]
        assert float((x - y).norm()) <= 2.0 ** -10 * float(y.norm()) + 2.0 ** -25 * math.sqrt(y.numel())


@pytest.mark.parametrize("m,nb", [(400, 0), (400, 16), (1500, 0)])
def test_large_gradients_do_not_overflow(m, nb):
    """ds passes 65504 although no gradient does.  Results near the type's end are left out;
    delta of more than 1024 keys is formed from the rounded out, which peaked rows feel
    most (2^-11 of dP against ds of some of the rows alone)."""
    c, how, dout = make(1, 200, m, 4, 2, 64, HF, nb=nb, far=60, seed=56, gain=2.8)
    c["k"], c["v"] = (2.8 * c["k"].float()).to(HF), (6.0 * c["v"].float()).to(HF)
    check_gradients(c, how, (2e3 * dout.float()).to(HF), 2.0 ** -8)


def test_value_gradients_of_long_sequences():
    """Weights of 2^-17, subnormal as they are."""
    c, how, dout = make(1, 130, 150000, 1, 1, 64, HF, seed=57, gain=0.5)
    check_gradients(c, how, dout, 2.0 ** -10)


def test_not_a_number_stays_in_its_rows():
    """A NaN in one query's gradient reaches that dq, and all dk and dv; the other rows of
    dq keep their values."""
    c, how, dout = make(1, 140, 300, 2, 2, 64, HF, seed=58)
    a = fs.fs_cross_attention(c["q"], c["k"], c["v"], **how)
    bad = dout.clone()
    bad[0, 7, 1, 3] = math.nan
    clean = fs.fs_cross_attention_grad(c["q"], c["k"], c["v"], *a, dout, **how)
    dq, dk, dv, _ = fs.fs_cross_attention_grad(c["q"], c["k"], c["v"], *a, bad, **how)
    assert bool(torch.isnan(dq[0, 7, 1]).all()) and bool(torch.isnan(dk[:, :, 1]).all())
    assert bool(torch.isnan(dv[:, :, 1, 3]).all())
    rest = torch.arange(140, device="cuda") != 7
    x, y = dq[0, rest, 1].double(), clean[0][0, rest, 1].double()
    assert float((x - y).norm()) <= 2.0 ** -10 * float(y.norm())
    assert torch.equal(dq[:, :, 0], clean[0][:, :, 0]) and torch.equal(dk[:, :, 0], clean[1][:, :, 0])


def check_gradients(c, how, dout, share):
    a = fs.fs_cross_attention(c["q"], c["k"], c["v"], **how)
    got = dict(zip(("dq", "dk", "dv", "dbias"),
                   fs.fs_cross_attention_grad(c["q"], c["k"], c["v"], *a, dout, **how)))
    want = exact(c, how, dout)
    missed = []
    for name, x in got.items():
        if x is None:
            continue
        y, x = want[name], x.to(F64)
        y, x = y[y.abs() < 6e4], x[y.abs() < 6e4]
        bound = share * float(y.norm()) + 2.0 ** -25 * math.sqrt(y.numel())
        off = float((x - y).norm())
        if not off <= bound:
            missed.append(f"{name}: {off / float(y.norm()):.3g} of its norm, bound {bound / float(y.norm()):.3g}")
    assert not missed, "; ".join(missed)
    return got
