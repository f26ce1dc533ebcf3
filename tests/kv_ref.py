"""Rotary positions, a cache in pages and the attention of drafted trees from their
definitions on the CPU, with bounds on the error that results may have.

Rows of a cache are held exactly (a quotient, a product and a rounding, each of them
defined), so codes, scales and what is read back are compared bit by bit.

Bounds.  u: unit roundoff of the results' type (2^-8 bfloat16, 2^-11 float16).
Rotary: the float32 angle is off by pi 2^-25 at most (a fraction of half a turn rounded
to float32), sine and cosine by two units in the last place more (2^-23), and a turned
element takes a product with the amplitude, two products and a sum (4 2^-24): together
below 2^-21 (|x| + |y|) amplitude; frequencies are rounded to float64 twice, here and there
once more in the product with the position, 2^-51 |p w| in all; then u once.
Tree attention: as a computation with float32 sums of 16-bit operands:
  z    (d + 12) 2^-24 Z_ij, Z_ij = scale sum_c |q_ic k_jc|, and so p relatively
       e_p = 2 (d + 12) 2^-24 max Z + 2^-16 (float32 exponentials, logarithms, sums)
  out  u |o| + (u_p + e_p) sum_j p_ij |v_j|, u_p the roundoff of the weights' 16-bit type
       (float16 for a cache in 8 bits)
  lse  the bound of z + 2^-20 (1 + |lse|)
plus 2^-24 of each |v_j| where weights are held in float16, whose small numbers lie
2^-25 apart at the largest weight of 2^7 or more.
"""
import math

import torch

F64 = torch.float64
TOP = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


def roundoff(dtype):
    return torch.finfo(dtype).eps / 2


def rotary64(x, freqs, pos, interleaved=False, amplitude=1.0, back=False):
    """(result, bound) for x (B, n, H, d) and pos (B, n)."""
    dtype = x.dtype
    x = x.detach().cpu().to(F64)
    half = freqs.numel()
    w = freqs.cpu().to(F64)
    angle = pos.cpu().to(F64)[..., None, None] * w
    c, s = amplitude * torch.cos(angle), amplitude * torch.sin(angle)
    if back:
        s = -s
    at = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else \
        (slice(0, half), slice(half, 2 * half))
    a, b = x[..., at[0]], x[..., at[1]]
    out, tol = x.clone(), torch.zeros_like(x)
    out[..., at[0]], out[..., at[1]] = a * c - b * s, a * s + b * c
    off = (2.0 ** -21 + 2.0 ** -51 * (pos.cpu().to(F64)[..., None, None] * w).abs()) * abs(amplitude)
    tol[..., at[0]] = tol[..., at[1]] = off * (a.abs() + b.abs())
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -134
    tol[..., :2 * half] += roundoff(dtype) * out[..., :2 * half].abs() + tiny
    return out, tol


def quantise(x, held):
    """(codes, scales) of rows x (..., d), 16-bit, on the CPU."""
    x = x.detach().cpu().float()
    amax = x.abs().amax(-1)
    fine = torch.isfinite(x).all(-1)
    amax = torch.where(fine, amax, torch.ones_like(amax)).clamp_min(2.0 ** -80)
    top = torch.full_like(amax, TOP[held])
    y = torch.where(fine[..., None], x * (top / amax)[..., None], torch.zeros_like(x))
    code = torch.round(y).to(torch.int8) if held == torch.int8 else y.to(held)
    return code, torch.where(fine, amax / top, torch.full_like(amax, math.nan))


def sees(n, parents):
    """(n, n) bool: row t of what token t of a tree sees, from a list of parents or None."""
    r = torch.zeros(n, n, dtype=torch.bool)
    for t in range(n):
        chain, u = [], t
        while u >= 0:
            chain.append(u)
            up = u - 1 if parents is None else int(parents[u])
            u = up if -1 <= up < u else -2
        if u == -1:
            r[t, chain] = True
    return r


def tree64(q, k, v, there, ctx, parents=None, scale=None, reach=None, weights=None):
    """out, lse and their bounds (under "tol") for q (B, n, H, d) and the values k, v
    (B, m, G, d) that the cache stands for at positions 0 .. m - 1; there (B, m): whether a
    position has a page; parents (B, n) or (n,)."""
    dtype = q.dtype
    u, u_p = roundoff(dtype), roundoff(weights or dtype)
    tiny = 2.0 ** -24 if (weights or dtype) == torch.float16 else 2.0 ** -126
    q, k, v = (x.detach().cpu().to(F64) for x in (q, k, v))
    B, n, H, d = q.shape
    m, G = k.shape[1], k.shape[2]
    R = H // G
    scale = d ** -0.5 if scale is None else scale
    out = torch.zeros(B, n, H, d, dtype=F64)
    lse = torch.full((B, H, n), -math.inf, dtype=F64)
    tol = {"out": torch.zeros_like(out), "lse": torch.zeros_like(lse)}
    for b in range(B):
        c = min(max(int(ctx[b]), 0), m)
        rows = None if parents is None else (parents[b] if parents.dim() == 2 else parents).cpu()
        tree = sees(n, rows)
        for t in range(n):
            if not tree[t, t]:
                continue
            keys = [j for j in range(c) if there[b, j]] + \
                [c + x for x in range(t + 1) if tree[t, x] and c + x < m and there[b, c + x]]
            if not keys:
                continue
            kk = k[b, keys].repeat_interleave(R, 1)
            vv = v[b, keys].repeat_interleave(R, 1)
            z = scale * torch.einsum("hc,jhc->hj", q[b, t], kk)
            zmax = float((scale * torch.einsum("hc,jhc->hj", q[b, t].abs(), kk.abs())).max())
            lse[b, :, t] = torch.logsumexp(z, -1)
            p = torch.softmax(z, -1)
            e_z = (d + 12) * 2.0 ** -24 * zmax
            e_p = 2 * e_z + 2.0 ** -16
            out[b, t] = torch.einsum("hj,jhc->hc", p, vv)
            tol["out"][b, t] = u * out[b, t].abs() + \
                (u_p + e_p) * torch.einsum("hj,jhc->hc", p, vv.abs()) + \
                tiny * vv.abs().sum(0) + (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -126)
            tol["lse"][b, :, t] = e_z + 2.0 ** -20 * (1 + lse[b, :, t].abs())
    return {"out": out, "lse": lse, "tol": tol}
