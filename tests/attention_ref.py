"""Cross attention from its definition in 64 bits on the CPU, its gradients
from their formulas, and bounds on the error that 16-bit results may have.

The bounds follow a computation that multiplies 16-bit operands with float32
sums, keeps the softmax in float32, rounds the probabilities p and the score
gradients ds once to 16 bits (unit roundoff u) as operands of the next
product, and rounds each result once:
  z     (d + 8) 2^-24 Z_ij, Z_ij = scale sum_c |q_ic k_jc|, and so p relatively
        e_p = 2 (d + 8) 2^-24 max Z + 2^-16 (float32 exponentials, sums, lse)
  out   u |o| + (u + e_p) sum_j p_ij |v_j|
  D     sum_c |dout_ic| times the bound of out (D is formed from the rounded out)
  ds    (u + e_p) |ds| + p (bound of D + 2^-16 sum_c |dout_ic| (|v_jc| + |o_ic|))
  dq, dk, dv, dbias   u |result| + the bounds of their terms, summed
plus, in float16, 2^-24 for each term whose 16-bit operand may be subnormal, and
2^-126 in every p, below which float32 and bfloat16 hold no normal numbers.
"""
import torch

F64 = torch.float64


def valid_keys(B, m, kv_len=None, key_mask=None):
    valid = torch.ones(B, m, dtype=torch.bool)
    if kv_len is not None:
        valid &= torch.arange(m)[None, :] < kv_len.cpu()[:, None]
    if key_mask is not None:
        valid &= key_mask.cpu() != 0
    return valid


def pair_buckets(B, n, m, buckets, q_pos=None):
    D = buckets.numel() // 2
    pos = torch.zeros(B, dtype=torch.int64) if q_pos is None else q_pos.cpu().long()
    rel = torch.arange(m)[None, None, :] - pos[:, None, None] - torch.arange(n)[None, :, None]
    return buckets.cpu().long()[rel.clamp(-D, D) + D]


def attention64(q, k, v, scale, kv_len=None, key_mask=None, bias=None, buckets=None, q_pos=None,
                dout=None):
    """{"out", "lse", ...} and, under "tol", the error bound of each entry."""
    half = q.dtype == torch.float16
    u = 2.0 ** -11 if half else 2.0 ** -8
    flush = 2.0 ** -126
    tiny = 2.0 ** -24 if half else flush
    q, k, v = (x.detach().cpu().to(F64) for x in (q, k, v))
    B, n, H, d = q.shape
    m, G = k.shape[1], k.shape[2]
    R = H // G
    valid = valid_keys(B, m, kv_len, key_mask)
    k = torch.where(valid[:, :, None, None], k, torch.zeros_like(k))
    v = torch.where(valid[:, :, None, None], v, torch.zeros_like(v))
    kh, vh = (x.repeat_interleave(R, dim=2) for x in (k, v))
    z = scale * torch.einsum("bihc,bjhc->bhij", q, kh)
    zabs = scale * torch.einsum("bihc,bjhc->bhij", q.abs(), kh.abs())
    if bias is not None:
        idx = pair_buckets(B, n, m, buckets, q_pos)
        t = bias.detach().cpu().to(F64).expand(H, -1)
        t = torch.where(t < -1e30, torch.full_like(t, -torch.inf), t)
        z = z + t[:, idx].transpose(0, 1)
    z = torch.where(valid[:, None, None, :], z, torch.full_like(z, -torch.inf))
    lse = torch.logsumexp(z, -1) if m else torch.full((B, H, n), -torch.inf, dtype=F64)
    p = torch.where(torch.isinf(lse)[..., None], torch.zeros_like(z), torch.exp(z - lse[..., None]))
    p = torch.nan_to_num(p, nan=0.0) if m else p
    zmax = float(zabs.max()) if zabs.numel() else 0.0
    e_z = (d + 8) * 2.0 ** -24 * zmax
    e_p = 2 * e_z + 2.0 ** -16
    pv = torch.einsum("bhij,bjhc->bihc", p, vh.abs())
    vsum = vh.abs().sum(1, keepdim=True) * tiny
    r = {"out": torch.einsum("bhij,bjhc->bihc", p, vh), "lse": lse}
    tol = {"out": u * r["out"].abs() + (u + e_p) * pv + vsum + tiny,
           "lse": e_z + 2.0 ** -20 * (1 + torch.nan_to_num(lse, neginf=0.0).abs())}
    r["tol"] = tol
    if dout is None:
        return r
    do = dout.detach().cpu().to(F64)
    D = (do * r["out"]).sum(-1).permute(0, 2, 1)
    dp = torch.einsum("bihc,bjhc->bhij", do, vh)
    ds = p * (dp - D[..., None])
    tol_D = (do.abs() * tol["out"]).sum(-1).permute(0, 2, 1)
    dpabs = torch.einsum("bihc,bjhc->bhij", do.abs(), vh.abs()) + \
        (do * r["out"]).abs().sum(-1).permute(0, 2, 1)[..., None]
    tol_ds = (u + e_p) * ds.abs() + p * (tol_D[..., None] + 2.0 ** -16 * dpabs) + tiny + \
        flush * dpabs

    def heads(x):       # sum over the query heads of each key head
        return x.reshape(x.shape[0], x.shape[1], G, R, x.shape[3]).sum(3)

    r["dq"] = scale * torch.einsum("bhij,bjhc->bihc", ds, kh)
    r["dk"] = scale * heads(torch.einsum("bhij,bihc->bjhc", ds, q))
    r["dv"] = heads(torch.einsum("bhij,bihc->bjhc", p, do))
    tol["dq"] = u * r["dq"].abs() + scale * torch.einsum("bhij,bjhc->bihc", tol_ds, kh.abs()) + tiny
    tol["dk"] = u * r["dk"].abs() + scale * heads(torch.einsum("bhij,bihc->bjhc", tol_ds, q.abs())) \
        + tiny
    tol["dv"] = u * r["dv"].abs() + tiny + heads(
        torch.einsum("bhij,bihc->bjhc", (u + e_p) * p + tiny, do.abs()))
    if bias is not None:
        nb, rows = bias.shape[1], bias.shape[0]
        for name, x in (("dbias", ds), ("tol", tol_ds)):
            acc = torch.zeros(H, nb, dtype=F64)
            for b in range(B):
                acc.index_add_(1, idx[b].reshape(-1), x[b].reshape(H, -1))
            acc = acc.sum(0, keepdim=True) if rows == 1 else acc
            if name == "dbias":
                r["dbias"] = acc
            else:
                tol["dbias"] = u * r["dbias"].abs() + acc + tiny
    return r
