"""Cases that time the cross attention of the library, with and without a learned
relative position bias: forward, forward with its gradients, and single tokens
against a long cache of keys and values.

Queries are (batch, n, heads, d), keys and values (batch, m, kv_heads, d), with
heads / kv_heads query heads on each key head.  Key j of batch b counts where
j < kv_len[b] and key_mask[b, j]; a query that no key counts for has output 0
and log-sum-exp -inf.  The bias of head h between query i and key j is
table[h, buckets[clamp(j - (q_pos[b] + i), -D, D) + D]].
"""
import math

import torch

own = False

# kind: "infer" is the forward pass, "train" the forward pass and every gradient,
# "decode" the forward pass of a few tokens against a cache.
# short: how much shorter than m the shortest sequence of a batch is (lengths fall
# evenly from m); drop: the share of the keys that a mask takes out, the front of a
# sequence (padding on the left) and single keys; buckets = 0: no position bias.


def _case(name, kind, batch, n, m, heads, kv_heads, d, dtype, short=0.0, drop=0.0, buckets=0,
          distance=0):
    return {"name": name, "kind": kind, "batch": batch, "n": n, "m": m, "heads": heads,
            "kv_heads": kv_heads, "d": d, "dtype": dtype, "short": short, "drop": drop,
            "buckets": buckets, "distance": distance}


def listed():
    return [
        # a short prompt's encoding attended to by a few latents: latency alone
        _case("infer-short", "infer", 1, 21, 77, 8, 8, 64, "float16"),
        # an encoder-decoder batch of sentences of unequal lengths, with a position bias
        _case("infer-ragged-bias", "infer", 8, 500, 1500, 16, 16, 64, "bfloat16", short=0.6,
              buckets=32, distance=128),
        # a long document read against another one: the matrix units' rate
        _case("infer-long", "infer", 4, 4096, 8192, 16, 16, 128, "bfloat16"),
        # shared key heads, a head size between the powers of two, padding on the left
        _case("infer-grouped-mask", "infer", 3, 777, 2050, 24, 8, 80, "float16", drop=0.3),
        # one sequence's next token against its encoder's states
        _case("decode-one", "decode", 1, 1, 1500, 16, 16, 64, "bfloat16"),
        # a serving batch, one token each, against caches of unequal lengths
        _case("decode-batch", "decode", 64, 1, 4096, 32, 8, 128, "bfloat16", short=0.5),
        # few sequences with a very long cache, two tokens each, with a position bias
        _case("decode-long-bias", "decode", 2, 2, 200001, 16, 4, 64, "float16", short=0.3,
              buckets=32, distance=128),
        # a small training step: short sequences, position bias
        _case("train-short-bias", "train", 2, 40, 120, 8, 8, 64, "bfloat16", buckets=32,
              distance=128),
        # an ordinary training step of an encoder-decoder layer
        _case("train-ragged-bias", "train", 8, 512, 1024, 16, 16, 64, "bfloat16", short=0.5,
              buckets=32, distance=128),
        # long sequences of both sides, the largest training step
        _case("train-long", "train", 2, 4096, 4096, 16, 16, 128, "bfloat16"),
        # shared key heads, masks and bias together, sizes that divide nothing
        _case("train-grouped-mask", "train", 3, 777, 1290, 16, 4, 96, "float16", drop=0.25,
              buckets=48, distance=300),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        kind = rng.choice(["infer", "decode", "train"])
        kv_heads = rng.choice([1, 2, 4, 8, 12, 16])
        group = rng.choice([1, 1, 2, 3, 4, 8])
        if kind == "decode":
            batch, n, m = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 4]), _log(rng, 60, 200000)
        else:
            batch, n, m = _log(rng, 1, 8), _log(rng, 16, 4096), _log(rng, 60, 8192)
        c = _case("", kind, batch, n, m, kv_heads * group, kv_heads,
                  rng.choice([64, 64, 128, 128, 72, 80, 96, 112, 48, 32]),
                  rng.choice(["bfloat16", "bfloat16", "float16"]))
        del c["name"]
        mask = rng.choice(["none", "short", "drop", "both"])
        if mask in ("short", "both"):
            c["short"] = round(rng.uniform(0.1, 0.9), 2)
        if mask in ("drop", "both"):
            c["drop"] = round(rng.uniform(0.05, 0.5), 2)
        if rng.random() < 0.5:
            c["buckets"] = 2 * rng.randint(4, 32)
            c["distance"] = _log(rng, 2 * c["buckets"], 1000)
        pairs = c["batch"] * c["heads"] * n * m
        top = {"infer": 2.0e9, "train": 5.0e8, "decode": 1.0e8}[kind]
        w = work(c)
        if pairs <= top and w["flops"] <= 9.0e11 and w["bytes"] <= 1.0e9:
            return c


def _lengths(c):
    return [c["m"] - int(c["m"] * c["short"] * b / c["batch"]) for b in range(c["batch"])]


def relative_buckets(buckets, distance):
    """Bucket of each relative position -distance..distance: half of the buckets for each
    side, of which the nearer half hold one position each and the rest widen
    geometrically up to `distance`; the boundaries are those of exact arithmetic."""
    half = buckets // 2
    near = half // 2
    out = []
    for rel in range(-distance, distance + 1):
        a = abs(rel)
        b = a
        if a >= near:
            # the largest step with near * (distance / near) ** (step / (half - near)) <= a
            step = 0
            while step + 1 < half - near and \
                    near ** (half - near) * distance ** (step + 1) <= \
                    a ** (half - near) * near ** (step + 1):
                step += 1
            b = near + step
        out.append(b + (half if rel > 0 else 0))
    return out


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = getattr(torch, c["dtype"])

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    B, n, m, H, G, d = c["batch"], c["n"], c["m"], c["heads"], c["kv_heads"], c["d"]
    s = {"case": c, "kind": c["kind"], "scale": 1.0 / math.sqrt(d)}
    s["q"] = (2.0 * rnd(B, n, H, d)).to(dt)
    if c["kind"] == "decode":   # a cache: each head's keys lie together
        s["k"], s["v"] = (rnd(B, G, m, d).to(dt).transpose(1, 2) for _ in range(2))
    else:                       # one projection's output holds both
        kv = rnd(B, m, 2, G, d).to(dt)
        s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
    s["kv_len"] = s["key_mask"] = s["table"] = s["buckets"] = s["q_pos"] = None
    if c["short"]:
        order = torch.randperm(B, generator=gen, device=dev)
        s["kv_len"] = torch.tensor(_lengths(c), dtype=torch.int32, device=dev)[order]
    if c["drop"]:
        front = torch.rand(B, 1, generator=gen, device=dev) * (2 * 0.9 * c["drop"] * m)
        keep = torch.rand(B, m, generator=gen, device=dev) >= 0.1 * c["drop"]
        s["key_mask"] = keep & (torch.arange(m, device=dev) >= front)
    if c["buckets"]:
        s["table"] = rnd(H, c["buckets"]).to(dt)
        s["buckets"] = torch.tensor(relative_buckets(c["buckets"], c["distance"]),
                                    dtype=torch.int32, device=dev)
        if c["kind"] == "decode":
            s["q_pos"] = torch.randint(0, m, (B,), generator=gen, device=dev, dtype=torch.int32)
    if c["kind"] == "train":
        s["dout"] = rnd(B, n, H, d).to(dt)
    return s


def _valid(s):
    c = s["case"]
    j = torch.arange(c["m"], device=s["q"].device)
    valid = torch.ones(c["batch"], c["m"], dtype=torch.bool, device=s["q"].device)
    if s["kv_len"] is not None:
        valid = j[None, :] < s["kv_len"][:, None]
    if s["key_mask"] is not None:
        valid = valid & s["key_mask"]
    return valid


def _bucket_index(s):
    """(batch or 1, n, m) bucket of every pair."""
    c = s["case"]
    dev = s["q"].device
    pos = torch.zeros(1, dtype=torch.int64, device=dev) if s["q_pos"] is None else s["q_pos"].long()
    at = pos[:, None] + torch.arange(c["n"], device=dev)
    rel = torch.arange(c["m"], device=dev) - at[:, :, None]
    return s["buckets"].long()[rel.clamp(-c["distance"], c["distance"]) + c["distance"]]


def _plain(s):
    c = s["case"]
    B, n, m, H, G, d = c["batch"], c["n"], c["m"], c["heads"], c["kv_heads"], c["d"]
    R = H // G
    dt = s["q"].dtype

    def rows(x):        # (B, n, H, d) -> (B, G, R n, d)
        return x.float().permute(0, 2, 1, 3).reshape(B, G, R * n, d)

    def unrows(x):
        return x.reshape(B, H, n, d).permute(0, 2, 1, 3).to(dt)

    q = rows(s["q"])
    k, v = (s[x].float().permute(0, 2, 1, 3) for x in ("k", "v"))
    score = (torch.matmul(q, k.transpose(2, 3)) * s["scale"]).view(B, H, n, m)
    index = None
    if s["table"] is not None:
        index = _bucket_index(s)
        score = score + s["table"].float()[:, index].transpose(0, 1)
    valid = _valid(s)[:, None, None, :]
    score = torch.where(valid, score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(-1)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    flat = p.view(B, G, R * n, m)
    out = {"out": unrows(torch.matmul(flat, v)), "lse": lse}
    if s["kind"] != "train":
        return out
    do = rows(s["dout"])
    out["dv"] = torch.matmul(flat.transpose(2, 3), do).permute(0, 2, 1, 3).to(dt)
    dp = torch.matmul(do, v.transpose(2, 3))
    ds = flat * (dp - (flat * dp).sum(-1, keepdim=True))
    out["dq"] = unrows(torch.matmul(ds, k) * s["scale"])
    out["dk"] = (torch.matmul(ds.transpose(2, 3), q) * s["scale"]).permute(0, 2, 1, 3).to(dt)
    if index is not None:
        per_pair = ds.view(B, H, n * m).sum(0)
        hot = (index.view(n * m, 1) == torch.arange(c["buckets"], device=q.device)).float()
        out["dbias"] = torch.matmul(per_pair, hot).to(dt)
    return out


def run(state):
    if not own:
        return _plain(state)
    from streaming_sinkhorn_solver_gb300 import binding as fs
    s = state
    how = dict(scale=s["scale"], kv_len=s["kv_len"], key_mask=s["key_mask"],
               bias=s["table"], bias_buckets=s["buckets"], q_pos=s["q_pos"])
    out, lse = fs.fs_cross_attention(s["q"], s["k"], s["v"], **how)
    if s["kind"] != "train":
        return {"out": out, "lse": lse}
    dq, dk, dv, dbias = fs.fs_cross_attention_grad(s["q"], s["k"], s["v"], out, lse, s["dout"],
                                                   **how)
    r = {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    if dbias is not None:
        r["dbias"] = dbias
    return r


def work(case):
    """Counted keys only: a masked key need not be read or multiplied."""
    c = case
    B, n, H, G, d = c["batch"], c["n"], c["heads"], c["kv_heads"], c["d"]
    keys = sum(_lengths(c)) * (1.0 - c["drop"])
    train = c["kind"] == "train"
    one = 2 * d * B * n * H            # bytes of q; of out, dout and dq too
    kv = 2 * d * keys * G              # bytes of the counted keys; of the values too
    table = 2 * H * c["buckets"]
    # forward: q, k, v -> out, lse; gradients: dout too -> dq, dk, dv, dbias
    moved = 2 * one + 2 * kv + 4 * B * H * n + table
    if c["drop"]:
        moved += B * c["m"]
    if train:
        moved += 2 * one + 2 * 2 * d * B * c["m"] * G + table
    # two products a pair forward; dV, dP, dQ, dK besides
    return {"bytes": float(moved), "flops": float((12 if train else 4) * d * H * n * keys)}


def exact(case, seed):
    """One batch entry and key head at a time, over its counted keys alone, in 64 bits; the
    gradients by automatic differentiation of that."""
    s = prepare(case, seed)
    c = s["case"]
    B, n, m, H, G, d = c["batch"], c["n"], c["m"], c["heads"], c["kv_heads"], c["d"]
    R = H // G
    dev = s["q"].device
    train = s["kind"] == "train"

    def zeros(*shape):
        return torch.zeros(*shape, dtype=torch.float64, device=dev)

    out = {"out": zeros(B, n, H, d), "lse": torch.full_like(zeros(B, H, n), -math.inf)}
    if train:
        out.update(dq=zeros(B, n, H, d), dk=zeros(B, m, G, d), dv=zeros(B, m, G, d))
        if s["table"] is not None:
            out["dbias"] = zeros(H, c["buckets"])
    for b in range(B):
        keep = torch.ones(m, dtype=torch.bool, device=dev)
        if s["kv_len"] is not None:
            keep[int(s["kv_len"][b]):] = False
        if s["key_mask"] is not None:
            keep &= s["key_mask"][b]
        at = keep.nonzero()[:, 0]
        if not len(at):
            continue
        bucket = None
        if s["table"] is not None:
            first = 0 if s["q_pos"] is None else int(s["q_pos"][b])
            rel = at[None, :] - (first + torch.arange(n, device=dev))[:, None]
            bucket = s["buckets"].long()[torch.clamp(rel, -c["distance"], c["distance"])
                                         + c["distance"]]
        for g in range(G):
            heads = slice(g * R, g * R + R)
            q = s["q"][b, :, heads].double().requires_grad_(train)
            k, v = (s[x][b, at, g].double().requires_grad_(train) for x in ("k", "v"))
            leaves = [q, k, v]
            z = torch.einsum("nrd,md->rnm", q, k) * s["scale"]
            if bucket is not None:
                t = s["table"][heads].double().requires_grad_(train)
                leaves.append(t)
                z = z + t[:, bucket.reshape(-1)].view(R, n, -1)
            y = torch.einsum("rnm,md->nrd", torch.softmax(z, -1), v)
            out["out"][b, :, heads] = y.detach()
            out["lse"][b, heads] = torch.logsumexp(z.detach(), -1)
            if train:
                got = torch.autograd.grad(y, leaves, s["dout"][b, :, heads].double())
                out["dq"][b, :, heads] = got[0]
                out["dk"][b, at, g] = got[1]
                out["dv"][b, at, g] = got[2]
                if bucket is not None:
                    out["dbias"][heads] += got[3]
    return out
