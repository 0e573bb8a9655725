"""Plain 64-bit forms of the gated delta rule's single tokens, the vocabulary's
loss and the embedding, and the bounds their tests use.

U is half a step of fp32 (2^-24).  A bound counts roundings times U (or what a
comment says) times the magnitudes they apply to; a result's own rounding is added
by ssm_ref.assert_within.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24


def dbl(t):
    """In 64 bits, where it is."""
    return None if t is None else t.detach().double()


# ---- the rule, one token of each request ---------------------------------------

def gates(a, b, A_log, dt_bias):
    x = a + dt_bias
    return -torch.exp(A_log) * torch.where(x > 20, x, torch.log1p(torch.exp(x.clamp(max=20)))), torch.sigmoid(b)


def rule_step(q, k, v, g, beta, S, scale, l2norm, z=None, norm_w=None, eps=1e-6):
    """q, k [B, Hk, dk], v [B, Hv, dv], g, beta [B, Hv], S [B, Hv, dk, dv], all 64 bits.
    Returns o (or the normed output), its bound, the states and theirs."""
    r, dk, dv = v.shape[1] // q.shape[1], q.shape[2], v.shape[2]
    nq = torch.rsqrt(q.square().sum(2, keepdim=True) + 1e-6) if l2norm else 1.0
    nk = torch.rsqrt(k.square().sum(2, keepdim=True) + 1e-6) if l2norm else 1.0
    q, k = (q * nq * scale).repeat_interleave(r, 1), (k * nk).repeat_interleave(r, 1)
    a = torch.exp(g)[:, :, None, None]
    P = a * S
    u = v - (P * k[..., None]).sum(2)
    new = P + (beta[..., None] * k)[..., None] * u[:, :, None, :]
    o = (new * q[..., None]).sum(2)
    # magnitudes.  Norms and gates: 16 roundings of sums, root, exponentials and products, dk / 16 + 5 of a norm's
    # sum over lanes, and the exponent's own error, 8 roundings of g.  Sums over dk: eight terms a thread, then
    # 5 + dk / 8 joined
    n = (64 + dk + 8 * g.abs())[:, :, None] * U
    mu = v.abs() + (P.abs() * k.abs()[..., None]).sum(2)
    bS = n[..., None] * (P.abs() + (beta[..., None] * k).abs()[..., None] * mu[:, :, None, :])
    # o is formed from the sums over the old state and (k.q) u: their magnitudes, not the new state's
    kq = (k.abs() * q.abs()).sum(2, keepdim=True)
    bo = 2 * n * ((P.abs() * q.abs()[..., None]).sum(2) + kq * beta[..., None] * mu)
    if z is None:
        return o, bo, new, bS
    rms = torch.sqrt(o.square().mean(2, keepdim=True) + eps)
    f = norm_w * z * torch.sigmoid(z)
    y = o / rms * f
    by = f.abs() * bo / rms + y.abs() * (torch.sqrt(bo.square().mean(2, keepdim=True)) / rms + (32 + dv) * U)
    return y, by, new, bS


# ---- embedding -------------------------------------------------------------------

def embed_bwd(dy, tokens, vocab, scale):
    """The table's gradient and the bound on its fp32 sums: a rounding for every row, one for the scale."""
    d = torch.zeros(vocab, dy.shape[1], dtype=torch.float64, device=dy.device)
    mag = torch.zeros_like(d)
    count = torch.zeros(vocab, 1, dtype=torch.float64, device=dy.device)
    real = (tokens >= 0) & (tokens < vocab)
    t = tokens[real].long()
    d.index_put_((t,), dy[real], accumulate=True)
    mag.index_put_((t,), dy[real].abs(), accumulate=True)
    count.index_put_((t,), torch.ones(len(t), 1, dtype=torch.float64, device=dy.device), accumulate=True)
    return d * scale, (count + 1) * U * mag * abs(scale)


# ---- the vocabulary's loss --------------------------------------------------------

def vocab_loss(h, w, targets, scale, f32, dloss=None):
    """h [T, W], w [V, W] in 64 bits.  Returns a dict of loss, lse, dh, dw and their bounds (the keys + "_b")."""
    T, (V, W) = h.shape[0], w.shape
    t, real = targets.long().clamp(min=0), targets >= 0
    x = scale * h @ w.t()
    mag = abs(scale) * h.abs() @ w.abs().t()
    # a logit: K in steps of 16 terms, each cut by up to 2^-22 of the terms' magnitudes, and as many more of joining
    ex = (W / 16 + 16) * 2.0 ** -22 * mag
    if f32:
        # two parts of 11 bits each side (half a step of the second: 2^-23 of the value, or 2^-39 of the largest of
        # its scaling), without the product of the second ones (2^-22)
        ex = ex + 2.0 ** -21 * mag + 2.0 ** -38 * W * abs(scale) * h.abs().amax(1, keepdim=True) * w.abs().max()
    ex = ex + 4 * U * x.abs()
    lse = torch.logsumexp(x, 1)
    # sums of exponentials: 2^-21 for the exponential and its argument (fp32's, of what lies within 2^4 of the
    # maximum; below, terms count as much less), 16 terms a thread, then joined tile by tile
    el = ex.amax(1) + (64 + V / 256) * U + 2.0 ** -20 + 4 * U * lse.abs()
    at = x.gather(1, t[:, None])[:, 0]
    out = dict(lse=lse, lse_b=el, loss=torch.where(real, lse - at, 0.0),
               loss_b=torch.where(real, el + ex.gather(1, t[:, None])[:, 0], 0.0))
    if dloss is None:
        return out
    g = torch.where(real, dloss * scale, 0.0)[:, None]
    p = torch.exp(x - lse[:, None])
    hot = torch.zeros_like(p).scatter_(1, t[:, None], 1.0)
    P = g * (p - hot)
    # P: its exponential's error, then its rounding to bf16 (the entry at the target gets what that took back), or
    # to two parts of fp16 (2^-23 of itself, or 2^-39 of dloss)
    eP = g.abs() * p * (ex + el[:, None] + 2.0 ** -20 + 4 * U * (x - lse[:, None]).abs()) + 4 * U * P.abs()
    rounding = 2.0 ** -22 * P.abs() + 2.0 ** -38 * g.abs() if f32 else 2.0 ** -8 * P.abs()
    eh = eP + (rounding if f32 else rounding * (1 - hot))
    ew = eP + rounding
    out["dh"], out["dw"] = P @ w, P.t() @ h
    out["dh_b"] = eh @ w.abs() + (V / 16 + 64) * 2.0 ** -22 * (P.abs() @ w.abs())
    out["dw_b"] = ew.t() @ h.abs() + (T / 16 + 64) * 2.0 ** -22 * (P.abs().t() @ h.abs())
    if f32:  # the other side's parts, scaled by one for all of w, by dloss for h
        out["dh_b"] = out["dh_b"] + 2.0 ** -38 * P.abs().sum(1, keepdim=True) * w.abs().max()
        hg = (h.abs().amax(1, keepdim=True) * g.abs()).max() if T else 0.0
        per = torch.where(g.abs() > 0, P.abs() / g.abs().clamp(min=1e-300), 0.0)
        out["dw_b"] = out["dw_b"] + 2.0 ** -36 * per.sum(0)[:, None] * hg
    return out
