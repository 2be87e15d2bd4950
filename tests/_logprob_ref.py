"""The log-probability operators from their definitions in 64 bits, and bounds
on how far an fp32 evaluation may be from them.

Bounds.  A logit is s times a sum of D products (exact in fp32 for 16- and
4-bit operands) accumulated in fp32: every accumulation is off by at most one
ulp (2^-23) of a partial sum, which is at most S = max (|x| |W|^T) + |b|, and
there are at most D of them, so |dz| <= |s| (D + 8) 2^-23 S.
  lse:      moves by at most max |dz|, plus the exponentials' and the sum's
            relative error (2^-20 covers 2^-22 for ex2 and the summation) and
            its own rounding 2^-24 |lse|.
  logprob:  z_y (recomputed in fp64) minus lse.
  entropy:  d entropy = -sum p (log p + H) dz, at most |dz| (E|log p| + H) <= 2 H |dz|
            with H <= ln V, plus the relative error of l and w, 2^-20 (1 + ln V).
Gradients.  G = s (p (-(a + e H) - e log p) + a [v = y]) has the parts
A = |s| (p (|a| + |e| (H + |log p|)) + |a| [v = y]); an error of dq in log p
changes a part by at most its size times (dq + ...) and |e| p dq; 16-bit G is
rounded once (2^-8), 16-bit results once more.
"""
import math

import torch


def bound_z(x, w, b, s):
    S = (x.double().abs() @ w.double().abs().T).max().item() if x.numel() else 0.0
    if b is not None:
        f = b.double()[torch.isfinite(b)]
        f = f[f.abs() < 1e30]
        S += f.abs().max().item() if f.numel() else 0.0
    return abs(s) * (x.shape[1] + 8) * 2.0 ** -23 * S


def bounds(x, w, b, s):
    lnv = math.log(max(w.shape[0], 2))
    dz = bound_z(x, w, b, s)
    lse = dz + 2.0 ** -20
    return {"z": dz, "lse": lse, "logprob": lse, "entropy": 2 * lnv * dz + 2.0 ** -20 * (1 + lnv)}


def forward(x, token, w, b=None, s=1.0, k=0, ignore=-100):
    """(z, logprob, entropy, lse, ids, top) in fp64; x, w as the operator gets them."""
    z = x.double() @ w.double().T
    if b is not None:
        z = z + b.double()
    z = s * z
    V = z.shape[1]
    lse = torch.logsumexp(z, 1)
    none = torch.isneginf(lse)
    logp = torch.where(none[:, None], torch.full_like(z, -math.inf), z - lse[:, None])
    p = logp.exp()
    ent = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(1)
    lp = None
    if token is not None:
        ok = (token != ignore) & (token >= 0) & (token < V)
        y = torch.where(ok, token, torch.zeros_like(token))
        lp = torch.where(ok, logp.gather(1, y[:, None])[:, 0], torch.zeros_like(lse))
    ids = top = None
    if k:
        srt = z.sort(dim=1, descending=True, stable=True)
        ids = srt.indices[:, :k].int()
        top = srt.values[:, :k] - lse[:, None]
        gone = torch.isneginf(srt.values[:, :k])
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
        top = torch.where(gone, torch.full_like(top, -math.inf), top)
    return z, lp, ent, lse, ids, top


def grads(x, token, w, b, s, a, e, ignore=-100):
    """(dH, dW, db) in fp64, and the parts A of G."""
    V = w.shape[0]
    z, lp, ent, lse, _, _ = forward(x, token, w, b, s)
    none = torch.isneginf(lse)[:, None]
    logp = z - lse[:, None]
    p = torch.where(none, 0.0, logp.exp())
    plogp = torch.where(p > 0, p * logp, torch.zeros_like(p))
    ok = (token != ignore) & (token >= 0) & (token < V)
    a = torch.where(ok, a.double(), torch.zeros_like(lse))[:, None] if a is not None else 0 * lse[:, None]
    e = e.double()[:, None] if e is not None else 0 * lse[:, None]
    a = torch.where(none, 0.0, a)
    e = torch.where(none, 0.0, e)
    d = torch.zeros_like(z)
    rows = torch.arange(len(token), device=z.device)
    d[rows[ok], token[ok]] = 1.0
    H = ent[:, None]
    G = s * (-p * (a + e * H) - e * plogp + a * d)
    A = abs(s) * (p * (a.abs() + e.abs() * H) + e.abs() * plogp.abs() + a.abs() * d + e.abs() * p)
    x, w = x.double(), w.double()
    return G @ w, G.T @ x, G.sum(0), A


def grad_bounds(x, w, A, dH, dW, db, dz, dtype, rows):
    """Elementwise bounds on dH, dW, db computed with G in `dtype`."""
    u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    x, w = x.double().abs(), w.double().abs()
    g = (1.0 + u) * u + 4 * dz + 2.0 ** -18             # G's rounding, and p's relative error
    aw, ax, ab = A @ w, A.T @ x, A.sum(0)
    acc_h, acc_w = w.shape[0] * 2.0 ** -23, rows * 2.0 ** -23
    tiny = 1e-30
    return ((g + acc_h) * aw + u * dH.abs() + tiny, (g + acc_w) * ax + u * dW.abs() + tiny,
            (g + acc_w) * ab + u * db.abs() + tiny)


def unpack(packed, scales, group, dtype=torch.float64):
    V, D = packed.shape[0], 2 * packed.shape[1]
    q = torch.stack((packed & 15, packed >> 4), 2).view(V, D).to(torch.int16)
    q = ((q ^ 8) - 8).to(dtype)
    return q * scales.to(dtype).repeat_interleave(group, 1)[:, :D]
