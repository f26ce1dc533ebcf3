"""Cases that time the library's operators for serving from a cache of keys and values:
rotary positions (with their gradient), the cache as it is written and read back, and the
attention of a tree of drafted tokens over it.

Rotary positions: the first `rotary` elements of a head are pairs (i, i + rotary / 2), or
(2 i, 2 i + 1) where interleaved; pair i of a token at position p is turned by the angle
p * freqs[i] and multiplied by `amplitude`, the rest of the head is left as it is.

Cache: (pages, kv_heads, page_size, d) for keys and values each, in the type of the tokens
or in 8 bits with a float32 scale for every token and head; position p of sequence b lies at
place p % page_size of page table[b, p // page_size].  In 8 bits a row x is held as
x * (top / amax), quotient and product in float32, rounded to the type, with the scale
amax / top; amax is its largest magnitude, 2^-80 at least, and top the type's largest number
that is used: 448 (e4m3) or 127 (whole numbers).

Tree attention: token t of a sequence is at position ctx_len + t of its cache.  It sees the
ctx_len positions before the tree, itself, its parent parents[t], that one's parent and so
on up to a parent of -1; a token whose chain does not end so is not there (output 0,
log-sum-exp -inf).
"""
import math

import torch

own = False

TOP = {"float8_e4m3fn": 448.0, "int8": 127.0}
FLOOR = 2.0 ** -80

# kind: "rotate" turns queries and keys, "rotate-train" their gradients too, "store" writes
# a chunk of tokens and reads the sequences back, "tree" attends.
# short: how much shorter than `ctx` the shortest sequence of a batch is (lengths fall
# evenly from ctx); absent: the share of the tree's tokens that are padding.


def _rotate(name, kind, batch, n, heads, kv_heads, d, dtype, rotary=0, interleaved=False,
            far=0, factor=1.0, amplitude=1.0):
    return {"name": name, "kind": kind, "batch": batch, "n": n, "heads": heads,
            "kv_heads": kv_heads, "d": d, "dtype": dtype, "rotary": rotary or d,
            "interleaved": interleaved, "far": far, "factor": factor, "amplitude": amplitude}


def _store(name, batch, n, ctx, kv_heads, d, dtype, held, page, short=0.0):
    return {"name": name, "kind": "store", "batch": batch, "n": n, "ctx": ctx,
            "kv_heads": kv_heads, "d": d, "dtype": dtype, "held": held, "page": page,
            "short": short}


def _tree(name, batch, n, ctx, heads, kv_heads, d, dtype, held, page, short=0.0, chain=False,
          absent=0.0):
    return {"name": name, "kind": "tree", "batch": batch, "n": n, "ctx": ctx, "heads": heads,
            "kv_heads": kv_heads, "d": d, "dtype": dtype, "held": held, "page": page,
            "short": short, "chain": chain, "absent": absent}


def listed():
    return [
        # the next token of a few sequences: latency alone
        _rotate("rotate-step", "rotate", 4, 1, 32, 8, 128, "bfloat16", far=30000),
        # prompts as they are read in
        _rotate("rotate-prompt", "rotate", 2, 8192, 32, 8, 128, "bfloat16"),
        # a training step at far positions: neighbours as pairs, part of the head, stretched
        # frequencies
        _rotate("rotate-train-part", "rotate-train", 3, 2777, 24, 4, 80, "float16", rotary=40,
                interleaved=True, far=1000000, factor=8.0, amplitude=1.2),
        # a short prompt of one sequence
        _store("store-short", 1, 33, 33, 8, 64, "bfloat16", "float8_e4m3fn", 16),
        # a batch of prompts goes into the cache and is read back for a whole attention
        _store("store-prompts", 8, 4096, 4096, 8, 128, "bfloat16", "float8_e4m3fn", 64),
        # a chunk joins longer sequences, whole numbers, a head size between the powers of two
        _store("store-chunk", 5, 777, 9001, 4, 80, "float16", "int8", 32, short=0.6),
        # one sequence's next token: latency
        _tree("token-one", 1, 1, 1500, 16, 4, 64, "bfloat16", "bfloat16", 16, chain=True),
        # a serving batch, one token each, against caches of unequal lengths
        _tree("token-batch", 64, 1, 8192, 32, 8, 128, "bfloat16", "float8_e4m3fn", 64,
              short=0.5, chain=True),
        # one long document, a small tree
        _tree("tree-long", 1, 12, 200001, 16, 4, 64, "float16", "int8", 32),
        # a serving batch with trees of a few tokens
        _tree("tree-batch", 32, 16, 8192, 32, 8, 128, "bfloat16", "float8_e4m3fn", 64,
              short=0.5),
        # large trees, a cache in the type of the queries
        _tree("tree-wide", 16, 64, 16384, 32, 8, 128, "bfloat16", "bfloat16", 128, short=0.2),
        # sizes that divide nothing, padded trees of unequal sequences
        _tree("tree-odd", 7, 27, 3001, 20, 4, 80, "float16", "float16", 16, short=0.9,
              absent=0.2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        kind = rng.choice(["rotate", "rotate-train", "store", "store", "tree", "tree", "tree"])
        kv_heads = rng.choice([1, 2, 4, 8, 12, 16])
        group = rng.choice([1, 2, 3, 4, 5, 8])
        d = rng.choice([64, 64, 128, 128, 128, 32, 48, 72, 80, 96, 112])
        dtype = rng.choice(["bfloat16", "bfloat16", "float16"])
        held = rng.choice([dtype, "float8_e4m3fn", "float8_e4m3fn", "int8"])
        page = rng.choice([16, 16, 32, 64, 128])
        short = rng.choice([0.0, round(rng.uniform(0.1, 0.95), 2)])
        if kind.startswith("rotate"):
            c = _rotate("", kind, _log(rng, 1, 32), _log(rng, 1, 16384), kv_heads * group,
                        kv_heads, d, dtype, rng.choice([d, d, d // 2, d // 4]),
                        rng.random() < 0.5, _log(rng, 1, 2000000),
                        rng.choice([1.0, 4.0, round(rng.uniform(1.5, 32.0), 2)]),
                        rng.choice([1.0, round(rng.uniform(0.8, 1.5), 2)]))
        elif kind == "store":
            ctx = _log(rng, 1, 32768)
            c = _store("", _log(rng, 1, 64), min(ctx, _log(rng, 1, 32768)), ctx, kv_heads, d,
                       dtype, held, page, short)
        else:
            n = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 8, 128)])
            c = _tree("", _log(rng, 1, 64), n, _log(rng, 1, 200000), kv_heads * group,
                      kv_heads, d, dtype, held, page, short, rng.random() < 0.3,
                      rng.choice([0.0, 0.0, round(rng.uniform(0.05, 0.5), 2)]))
            if c["batch"] * c["heads"] * n * (c["ctx"] + n) > 4.0e8:
                continue
        del c["name"]
        w = work(c)
        if w["flops"] <= 5.0e11 and w["bytes"] <= (7.0e8 if kind == "tree" else 3.0e8):
            return c


def _lengths(c):
    return [c["ctx"] - int(c["ctx"] * c["short"] * b / c["batch"]) for b in range(c["batch"])]


def _frequencies(c, dev):
    """Angles a position, falling from 1; where the context is stretched by `factor`, those
    that turn less than once over 8192 positions are divided by it, those that turn more than
    four times are kept, and the ones between go over evenly."""
    half = c["rotary"] // 2
    f = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
    keep = ((8192 * f / (2 * math.pi) - 1.0) / 3.0).clamp(0.0, 1.0)
    return f * keep + f / c["factor"] * (1.0 - keep)


def _quantised(x, held):
    """(codes, scales) of rows x (..., d)."""
    amax = x.float().abs().amax(-1, keepdim=True).clamp_min(FLOOR)
    top = torch.full_like(amax, TOP[held])      # (a division by a plain number is not rounded once)
    y = x.float() * (top / amax)
    if held == "int8":
        code = torch.round(y).to(torch.int8)
    else:
        code = y.to(torch.float8_e4m3fn)
    return code, (amax / top).squeeze(-1)


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = getattr(torch, c["dtype"])

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=gen, device=dev, dtype=torch.int32)

    B, n, G, d = c["batch"], c["n"], c["kv_heads"], c["d"]
    s = {"case": c, "kind": c["kind"]}
    if c["kind"].startswith("rotate"):
        H = c["heads"]
        # one projection's output holds queries, keys and values
        qkv = rnd(B, n, H + 2 * G, d).to(dt)
        s["q"], s["k"] = qkv[:, :, :H], qkv[:, :, H:H + G]
        s["freqs"] = _frequencies(c, dev)
        first = whole(0, c["far"], B, 1) if c["far"] else whole(0, 1, B, 1)
        s["pos"] = first + torch.arange(n, dtype=torch.int32, device=dev)
        if c["kind"] == "rotate-train":
            s["dq"], s["dk"] = rnd(B, n, H, d).to(dt), rnd(B, n, G, d).to(dt)
        return s
    page, held = c["page"], c["held"]
    lens = torch.tensor(_lengths(c), dtype=torch.int32, device=dev)
    lens = lens[torch.randperm(B, generator=gen, device=dev)]
    tree = c["kind"] == "tree"
    span = c["ctx"] + (n if tree else 0)
    per = -(-span // page)
    # the pages that a sequence needs lie anywhere in the pool
    table = torch.randperm(B * per, generator=gen, device=dev).to(torch.int32).view(B, per)
    need = (lens + (n if tree else 0) + page - 1) // page
    unused = torch.arange(per, device=dev)[None, :] >= need[:, None]
    s["table"] = torch.where(unused, torch.full_like(table, -1), table)
    s["k_scale"] = s["v_scale"] = None
    for x in ("k", "v"):
        rows = torch.randn(B * per, G, page, d, generator=gen, device=dev, dtype=dt)
        if held == c["dtype"]:
            s[x + "_pages"] = rows
        else:
            s[x + "_pages"], s[x + "_scale"] = _quantised(rows, held)
    if not tree:
        # the last n positions of a sequence (or all of a shorter one) are written
        kv = rnd(B, n, 2, G, d).to(dt)
        s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
        at = lens[:, None] - n + torch.arange(n, dtype=torch.int32, device=dev)
        s["slots"] = torch.where(at >= 0, at, torch.full_like(at, -1))
        s["lens"] = lens
        return s
    s["q"] = (2.0 * rnd(B, n, c["heads"], d)).to(dt)
    s["ctx_len"] = lens
    s["parents"] = None
    if not c["chain"]:
        t = torch.arange(n, device=dev)
        back = (torch.rand(B, n, generator=gen, device=dev) ** 2 * (t + 1)).long()
        parents = (t - 1 - back).clamp_min(-1).to(torch.int32)
        if c["absent"]:     # padding at the end of the tree
            there = n - (torch.rand(B, 1, generator=gen, device=dev) * 2 * c["absent"] * n).long()
            parents = torch.where(t < there.clamp_min(0), parents, torch.full_like(parents, -2))
        s["parents"] = parents
    return s


# ---------------------------------------------------------------------------
# plain forms

def _turn(x, c, cos, sin):
    """Rows x (batch, n, heads, d) turned by angles of (batch, n, 1, rotary / 2)."""
    half = c["rotary"] // 2
    y = x.float().clone()
    if c["interleaved"]:
        a, b = x[..., 0:2 * half:2].float(), x[..., 1:2 * half:2].float()
        y[..., 0:2 * half:2] = a * cos - b * sin
        y[..., 1:2 * half:2] = a * sin + b * cos
    else:
        a, b = x[..., :half].float(), x[..., half:2 * half].float()
        y[..., :half] = a * cos - b * sin
        y[..., half:2 * half] = a * sin + b * cos
    return y.to(x.dtype)


def _plain_rotate(s):
    c = s["case"]
    angle = s["pos"].double()[:, :, None, None] * s["freqs"]
    cos, sin = ((f(angle) * c["amplitude"]).float() for f in (torch.cos, torch.sin))
    r = {"q": _turn(s["q"], c, cos, sin), "k": _turn(s["k"], c, cos, sin)}
    if c["kind"] == "rotate-train":
        r["dq"], r["dk"] = _turn(s["dq"], c, cos, -sin), _turn(s["dk"], c, cos, -sin)
    return r


def _bytes_of(x):
    """The same memory as whole numbers, which indexing knows for every type."""
    return x.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()])


def _rows_at(s, x, positions):
    """Rows x_pages of (batch, n) positions in float32, (batch, n, kv_heads, d), and where
    there is a page for them."""
    c = s["case"]
    pages = s[x + "_pages"]
    within = (positions >= 0) & (positions < s["table"].shape[1] * c["page"])
    p = torch.where(within, positions, torch.zeros_like(positions)).long()
    at = torch.gather(s["table"].long(), 1, p // c["page"])
    there = within & (at >= 0) & (at < pages.shape[0])
    at = torch.where(there, at, torch.zeros_like(at))
    rows = _bytes_of(pages)[at, :, p % c["page"]].view(pages.dtype).float()
    if s[x + "_scale"] is not None:
        rows = rows * s[x + "_scale"][at, :, p % c["page"]].unsqueeze(-1)
    return rows, there


def _plain_store(s):
    c = s["case"]
    dt = s["k"].dtype
    page = c["page"]
    keep = s["slots"] >= 0
    b = torch.arange(c["batch"], device=s["k"].device)[:, None].expand_as(keep)[keep]
    slot = s["slots"][keep].long()
    at = s["table"][b, slot // page].long()
    for x in ("k", "v"):
        rows = s[x][keep]
        if c["held"] == c["dtype"]:
            s[x + "_pages"][at, :, slot % page] = rows
        else:
            code, scale = _quantised(rows, c["held"])
            _bytes_of(s[x + "_pages"])[at, :, slot % page] = _bytes_of(code)
            s[x + "_scale"][at, :, slot % page] = scale
    j = torch.arange(c["ctx"], dtype=torch.int32, device=s["k"].device).expand(c["batch"], -1)
    j = torch.where(j < s["lens"][:, None], j, torch.full_like(j, -1))
    r = {}
    for x in ("k", "v"):
        rows, there = _rows_at(s, x, j)
        r[x] = torch.where(there[:, :, None, None], rows, torch.zeros_like(rows)).to(dt)
        if s[x + "_scale"] is not None:
            r[x + "_scale"] = s[x + "_scale"]
    return r


def _sees(s):
    """(batch, n, n): whether token t of the tree sees token u of it, and (batch, n): whether
    token t is there."""
    c = s["case"]
    n = c["n"]
    dev = s["q"].device
    eye = torch.eye(n, dtype=torch.bool, device=dev)
    if s["parents"] is None:
        low = torch.ones(n, n, dtype=torch.bool, device=dev).tril()
        return low.expand(c["batch"], n, n), torch.ones(c["batch"], n, dtype=torch.bool,
                                                        device=dev)
    t = torch.arange(n, device=dev)
    parents = s["parents"]
    step = (parents[:, :, None] == t) & (t[:, None] > t[None, :])
    root = parents == -1
    # chains of up to n steps, counted
    sees = torch.matrix_power((eye | step).double(), n).gt(0)
    there = (sees & root[:, None, :]).any(-1)
    return sees, there


def _plain_tree(s):
    c = s["case"]
    B, n, H, G, d = c["batch"], c["n"], c["heads"], c["kv_heads"], c["d"]
    dev = s["q"].device
    dt = s["q"].dtype
    m = c["ctx"] + n
    j = torch.arange(m, dtype=torch.int32, device=dev).expand(B, m)
    k, there = _rows_at(s, "k", j)
    v, _ = _rows_at(s, "v", j)
    sees, live = _sees(s)
    u = j - s["ctx_len"][:, None]                       # place within the tree
    inside = (u >= 0) & (u < n)
    drafted = torch.gather(sees, 2, u.clamp(0, n - 1).long()[:, None, :].expand(B, n, m))
    ok = ((u < 0)[:, None, :] | (inside[:, None, :] & drafted)) & there[:, None, :] & live[:, :, None]
    q = s["q"].float().view(B, n, G, H // G, d).permute(0, 2, 3, 1, 4).reshape(B, G, -1, d)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * d ** -0.5
    score = score.view(B, G, H // G, n, m)
    ok = ok[:, None, None]
    score = torch.where(ok, score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(-1).reshape(B, H, n)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    v = torch.where(there[:, :, None, None], v, torch.zeros_like(v))
    out = torch.matmul(p.view(B, G, -1, m), v.permute(0, 2, 1, 3))
    out = out.view(B, G, H // G, n, d).permute(0, 3, 1, 2, 4).reshape(B, n, H, d)
    return {"out": out.to(dt), "lse": lse}


def run(state):
    s = state
    c = s["case"]
    if not own:
        if c["kind"] == "tree":
            return _plain_tree(s)
        return _plain_store(s) if c["kind"] == "store" else _plain_rotate(s)
    from streaming_sinkhorn_solver_gb300 import binding as fs
    if c["kind"].startswith("rotate"):
        how = dict(interleaved=c["interleaved"], amplitude=c["amplitude"])
        q, k = fs.fs_rotary(s["q"], s["k"], s["freqs"], s["pos"], **how)
        r = {"q": q, "k": k}
        if c["kind"] == "rotate-train":
            r["dq"], r["dk"] = fs.fs_rotary_grad(s["dq"], s["dk"], s["freqs"], s["pos"], **how)
        return r
    cache = fs.KVCache(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
    if c["kind"] == "store":
        fs.fs_cache_write(cache, s["table"], s["slots"], s["k"], s["v"])
        k, v = fs.fs_cache_read(cache, s["table"], s["lens"], c["ctx"], dtype=s["k"].dtype)
        r = {"k": k, "v": v}
        if cache.k_scale is not None:
            r.update(k_scale=cache.k_scale, v_scale=cache.v_scale)
        return r
    out, lse = fs.fs_tree_attention(s["q"], cache, s["table"], s["ctx_len"], s["parents"])
    return {"out": out, "lse": lse}


def work(case):
    c = case
    B, n, G, d = c["batch"], c["n"], c["kv_heads"], c["d"]
    if c["kind"].startswith("rotate"):
        rows = B * n * (c["heads"] + G)
        times = 2 if c["kind"] == "rotate-train" else 1
        return {"bytes": float(times * (4 * rows * d + 4 * B * n) + 4 * c["rotary"]),
                "flops": float(times * 3 * rows * c["rotary"])}
    lens = _lengths(c)
    row = 2 * d if c["held"] == c["dtype"] else d + 4       # bytes of a key, or a value
    if c["kind"] == "store":
        written = sum(min(x, n) for x in lens)
        # read the tokens, write them; read the sequences, give them out (the rest as zeros)
        moved = 2 * G * (written * (2 * d + row) + sum(lens) * row + B * c["ctx"] * 2 * d)
        return {"bytes": float(moved), "flops": float(2 * G * d * (4 * written + sum(lens)))}
    H = c["heads"]
    keys = sum(lens)
    moved = 2 * G * row * (keys + B * n) + 4 * B * n * H * d + 4 * B * n * H
    pairs = n * keys + B * n * (n + 1) / 2 if c["chain"] else n * keys + B * n
    return {"bytes": float(moved), "flops": float(4 * d * H * pairs)}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits

def _turn64(x, case, pos, freqs, back):
    """Pairs as complex numbers, multiplied by amplitude * exp(i * angle)."""
    half = case["rotary"] // 2
    angle = pos.double()[..., None] * freqs.double()
    z = torch.polar(torch.full_like(angle, case["amplitude"]), -angle if back else angle)
    x = x.double()
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    if case["interleaved"]:
        w = torch.complex(*turned.unflatten(-1, (half, 2)).unbind(-1)) * z[:, :, None]
        turned = torch.view_as_real(w).flatten(-2)
    else:
        w = torch.complex(*turned.unflatten(-1, (2, half)).unbind(-2)) * z[:, :, None]
        turned = torch.cat([w.real, w.imag], -1)
    return torch.cat([turned, rest], -1)


def _held64(x, held):
    """Values that rows x (..., d) are held as, and the scales."""
    x = x.double()
    amax = x.abs().amax(-1, keepdim=True).clamp_min(FLOOR)
    scale = (amax / TOP[held]).float().double()
    # the quotient and the product are float32 by definition: halfway values depend on them
    y = (x * (TOP[held] / amax).float().double()).float().double()
    if held == "int8":
        return torch.round(y) * scale, scale.squeeze(-1)
    # three bits after the leading one, the smallest step 2^-9
    _, e = torch.frexp(y)
    step = torch.exp2((e - 4).clamp_min(-9).double())
    return torch.round(y / step) * step * scale, scale.squeeze(-1)


def _values64(s, x, b, count):
    """Positions 0 .. count - 1 of sequence b in 64 bits, (count, kv_heads, d), from pages
    that are there."""
    c = s["case"]
    pages = s["table"][b, :-(-count // c["page"])].long()
    rows = _bytes_of(s[x + "_pages"])[pages].view(s[x + "_pages"].dtype).double()
    if s[x + "_scale"] is not None:
        rows = rows * s[x + "_scale"][pages].double()[..., None]
    return rows.transpose(1, 2).flatten(0, 1)[:count]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["kind"].startswith("rotate"):
        names = ("q", "k", "dq", "dk") if c["kind"] == "rotate-train" else ("q", "k")
        return {x: _turn64(s[x], c, s["pos"], s["freqs"], x[0] == "d") for x in names}
    B, n, G, d = c["batch"], c["n"], c["kv_heads"], c["d"]
    dev = s["table"].device
    if c["kind"] == "store":
        r = {}
        for x in ("k", "v"):
            r[x] = torch.zeros(B, c["ctx"], G, d, dtype=torch.float64, device=dev)
            if s[x + "_scale"] is not None:
                r[x + "_scale"] = s[x + "_scale"].double()
            for b in range(B):
                count = int(s["lens"][b])
                fresh = min(count, n)
                r[x][b, :count] = _values64(s, x, b, count)
                rows = s[x][b, n - fresh:].double()
                if s[x + "_scale"] is not None:
                    rows, scale = _held64(rows, c["held"])
                    at = torch.arange(count - fresh, count, device=dev)
                    r[x + "_scale"][s["table"][b].long()[at // c["page"]], :, at % c["page"]] = scale
                r[x][b, count - fresh:count] = rows
        return r
    H = c["heads"]
    R = H // G
    out = torch.zeros(B, n, H, d, dtype=torch.float64, device=dev)
    lse = torch.full((B, H, n), -math.inf, dtype=torch.float64, device=dev)
    for b in range(B):
        ctx = int(s["ctx_len"][b])
        parents = list(range(-1, n - 1)) if s["parents"] is None else s["parents"][b].tolist()
        allowed = torch.zeros(n, ctx + n, dtype=torch.bool)
        for t in range(n):
            u, chain = t, []
            while u >= 0:
                chain.append(u)
                u = parents[u] if parents[u] < u else -2
            if u == -1:
                allowed[t, :ctx] = True
                allowed[t, [ctx + x for x in chain]] = True
        live = [t for t in range(n) if allowed[t].any()]
        if not live:
            continue
        allowed = allowed[live].to(dev)
        k, v = (_values64(s, x, b, ctx + n) for x in ("k", "v"))
        for g in range(G):
            heads = slice(g * R, g * R + R)
            q = s["q"][b, live, heads].double()
            z = torch.einsum("nrd,md->rnm", q, k[:, g]) / math.sqrt(d)
            z = z.masked_fill(~allowed, -math.inf)
            out[b, live, heads] = torch.einsum("rnm,md->nrd", torch.softmax(z, -1), v[:, g])
            lse[b, heads][:, live] = torch.logsumexp(z, -1)
    return {"out": out, "lse": lse}
