"""Plain 64-bit forms of the selective scan layer and the block norm, token by
token, and the bounds their tests use.

U is half a step of fp32 (2^-24).  A bound on an fp32 sum is a count of
roundings times U times the sum of its terms' magnitudes (`absolute=True` runs
the same formulas on magnitudes); a result rounded to bf16 adds 2^-8 of itself.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def d(t):
    return None if t is None else t.detach().double().cpu()


def assert_within(got, ref, bound, what):
    """|got - ref| <= half a step of got's type + bound, element by element."""
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    g = got.double().cpu()
    assert torch.equal(torch.isnan(g), torch.isnan(ref)), f"{what}: NaN in other places"
    err = (g - ref).abs()
    tol = HALF_STEP[got.dtype] * ref.abs() + bound
    bad = err > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol.clamp(min=1e-300)).max()):.2f} "
                           f"times the bound, error {float(err.max()):.3e}")


def seqs(cu):
    c = cu.tolist()
    return list(zip(c[:-1], c[1:]))


# ---- conv ---------------------------------------------------------------------

def conv_pre(x, w, b, cu, state, absolute=False):
    """Pre-activations, and every token's window rows [T, K, C]."""
    K = w.shape[1]
    pre, win = torch.zeros_like(x), torch.zeros(x.shape[0], K, x.shape[1], dtype=x.dtype)
    rows = []
    for n, (s, e) in enumerate(seqs(cu)):
        h = state[n] if state is not None else x.new_zeros(K - 1, x.shape[1])
        r = torch.cat([h, x[s:e]])
        rows.append(r)
        for t in range(e - s):
            win[s + t] = r[t:t + K]
            pre[s + t] = (r[t:t + K] * w.t()).sum(0) if not absolute else (r[t:t + K] * w.t()).abs().sum(0)
    if b is not None:
        pre = pre + (b.abs() if absolute else b)
    return pre, win, rows


def conv_fwd(x, w, b, cu, state):
    """y, state_out and the bound on y's fp32 arithmetic."""
    K = w.shape[1]
    pre, _, rows = conv_pre(x, w, b, cu, state)
    mag, _, _ = conv_pre(x, w, b, cu, state, absolute=True)
    st = torch.stack([r[len(r) - (K - 1):] for r in rows])
    # K + 1 roundings of the sum through a slope of at most 1.1; the SiLU itself: e^-a by 2^v with the
    # argument rounded (|a| U) and 2 steps of its own, two more operations, all relative to |y| <= |a|
    return pre * torch.sigmoid(pre), st, U * (1.1 * (K + 1) * mag + (8 + 2 * pre.abs()) * pre.abs())


def conv_bwd(dy, x, w, b, cu, state, dso, absolute=False):
    K = w.shape[1]
    pre, win, _ = conv_pre(x, w, b, cu, state)
    s = torch.sigmoid(pre)
    ds = dy * s * (1 + pre * (1 - s))
    if absolute:
        ds = dy.abs() * (0.5 + pre.abs())  # a magnitude of the factors' parts
        win, w = win.abs(), w.abs()
    dx, dst = torch.zeros_like(x), []
    for n, (a, e) in enumerate(seqs(cu)):
        g = x.new_zeros(K - 1 + e - a, x.shape[1])
        for t in range(e - a):
            g[t:t + K] += ds[a + t] * w.t()
        if dso is not None:
            g[len(g) - (K - 1):] += dso[n].abs() if absolute else dso[n]
        dst.append(g[:K - 1])
        dx[a:e] = g[K - 1:]
    return dict(dx=dx, dw=torch.einsum("tc,tkc->ck", ds, win), dbias=ds.sum(0), dstate=torch.stack(dst))


# ---- scan ---------------------------------------------------------------------

def softplus(v):
    return torch.where(v > 20, v, torch.log1p(torch.exp(v.clamp(max=20))))


def _wide(q, ch):
    return q.repeat_interleave(ch // q.shape[1], 1)  # [T, G, N] -> [T, Ch, N]


def scan(x, dt, A_log, B, C, cu, D=None, z=None, dt_bias=None, h0=None):
    """y, h_final, their bounds, and the states before and after every token."""
    T, ch = x.shape
    raw = dt + (dt_bias if dt_bias is not None else 0.0)
    delta, A = softplus(raw), -torch.exp(A_log)
    Bw, Cw = _wide(B, ch), _wide(C, ch)
    core, err = torch.zeros_like(x), torch.zeros_like(x)
    before, after = [None] * T, [None] * T
    hf, ehf = [], []
    N = A.shape[1]
    for n, (s, e) in enumerate(seqs(cu)):
        h = h0[n].clone() if h0 is not None else x.new_zeros(ch, N)
        mag, eh = h.abs(), torch.zeros_like(h)
        for t in range(s, e):
            a = torch.exp(delta[t][:, None] * A)
            ub = (delta[t] * x[t])[:, None] * Bw[t]
            before[t] = h
            h = a * h + ub
            after[t] = h
            # a is off by 10 U from delta's and A's own errors (times |v| e^-|v| <= 0.37) and 4 U of 2^v,
            # delta x B by 10 U, the sum by one rounding: 16 U of the terms' magnitudes cover a step
            mag = a * mag + ub.abs()
            eh = a * eh + 16 * U * mag
            core[t] = (h * Cw[t]).sum(1)
            err[t] = ((eh + (N + 2) * U * mag) * Cw[t].abs()).sum(1)
        hf.append(h)
        ehf.append(eh)
    skip = core + D * x if D is not None else core
    err = err + (2 * U * (D * x).abs() if D is not None else 0.0)
    if z is not None:
        sil = z * torch.sigmoid(z)
        err = err * sil.abs() + (8 + 2 * z.abs()) * U * (skip * sil).abs()
        skip_y = skip * sil
    else:
        skip_y = skip
    return dict(y=skip_y, h_final=torch.stack(hf), y_bound=err, h_bound=torch.stack(ehf), before=before, after=after,
                delta=delta, raw=raw, A=A, skip=skip)


def scan_grads(dy, dhf, x, dt, A_log, B, C, cu, D=None, z=None, dt_bias=None, h0=None, absolute=False):
    """Gradients by the formulas, walked backwards; absolute: every product by its magnitude."""
    T, ch = x.shape
    G = B.shape[1]
    f = scan(x, dt, A_log, B, C, cu, D, z, dt_bias, h0)
    m_ = (lambda v: v.abs()) if absolute else (lambda v: v)
    A, delta, raw = f["A"], f["delta"], f["raw"]
    before, after, skip = f["before"], f["after"], f["skip"]
    if absolute:  # states of the magnitudes
        g = scan(x.abs(), dt, A_log, B.abs(), C.abs(), cu, None if D is None else D.abs(), z, dt_bias,
                 None if h0 is None else h0.abs())
        before, after, skip = g["before"], g["after"], g["skip"]
    x, dy, Bw, Cw, Am = m_(x), m_(dy), m_(_wide(B, ch)), m_(_wide(C, ch)), m_(A)
    sg = torch.sigmoid(z) if z is not None else None
    ds = dy * m_(z * sg) if z is not None else dy
    u = delta * x
    N = A.shape[1]
    dB, dC = torch.zeros(T, G, N, dtype=x.dtype), torch.zeros(T, G, N, dtype=x.dtype)
    du, dd, dA = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(A)
    dh0 = []
    for n, (s, e) in enumerate(seqs(cu)):
        dh = m_(dhf[n]) if dhf is not None else x.new_zeros(ch, N)
        for t in range(e - 1, s - 1, -1):
            a = torch.exp(delta[t][:, None] * A)
            dC[t] = (after[t] * ds[t][:, None]).view(G, -1, N).sum(1)
            dh = dh + ds[t][:, None] * Cw[t]
            dB[t] = (dh * u[t][:, None]).view(G, -1, N).sum(1)
            du[t] = (dh * Bw[t]).sum(1)
            dh = dh * a
            m = dh * before[t]
            dd[t] = (Am * m).sum(1)
            dA += delta[t][:, None] * m
        dh0.append(dh)
    dd = dd + du * x
    slope = torch.where(raw > 20, torch.ones_like(raw), torch.sigmoid(raw))
    r = dict(dx=du * delta + (m_(D) * ds if D is not None else 0.0), ddt=dd * slope, dA_log=dA * Am, dB=dB, dC=dC,
             dD=(ds * x).sum(0) if D is not None else None, dh0=torch.stack(dh0), dz=None, ddt_bias=None)
    if dt_bias is not None:
        r["ddt_bias"] = r["ddt"].sum(0)
    if z is not None:
        r["dz"] = dy * skip * (sg * (1 + m_(z) * (1 - sg)))
    return r


def scan_step(x, dt, A_log, B, C, states, D, z, dt_bias):
    """One token of each row from states [Bt, Ch, N]: as a batch of one-token sequences."""
    cu = torch.arange(x.shape[0] + 1)
    return scan(x, dt, A_log, B, C, cu, D, z, dt_bias, states)


# ---- block norm -----------------------------------------------------------------

def norm_parts(o, w_post, gate, scale, eps):
    r1 = 1 / torch.sqrt(o.square().mean(1, keepdim=True) + eps)
    p = o * r1 * w_post if w_post is not None else o
    sg = torch.sigmoid(gate) if gate is not None else torch.ones_like(o)
    sc = scale if scale is not None else torch.ones(o.shape[1], dtype=o.dtype)
    return r1, p, sg, sc


def norm_fwd(o, res, w_pre, w_post, gate, scale, eps):
    _, p, sg, sc = norm_parts(o, w_post, gate, scale, eps)
    r = res + p * sg * sc
    return r * w_pre / torch.sqrt(r.square().mean(1, keepdim=True) + eps), r


def norm_bwd(dy, dres, o, r, w_pre, w_post, gate, scale, eps, absolute=False):
    m_ = (lambda v: v.abs()) if absolute else (lambda v: v)
    r1, p, sg, sc = norm_parts(o, w_post, gate, scale, eps)
    r2 = 1 / torch.sqrt(r.square().mean(1, keepdim=True) + eps)
    rh, wd = m_(r * r2), m_(dy * w_pre)
    back = rh * (wd * rh).mean(1, keepdim=True)
    dr = (m_(dres) if dres is not None else 0.0) + r2 * (wd + back if absolute else wd - back)
    p, sc = m_(p), m_(sc)
    dp = dr * sg * sc
    g = dict(dres=dr, dw_pre=(m_(dy) * rh).sum(0), dgate=None, dscale=None, dw_post=None)
    if gate is not None:
        g["dgate"] = dr * sc * p * sg * (1 - sg)
    if scale is not None:
        g["dscale"] = (dr * sg * p).sum(0)
    if w_post is not None:
        oh, wp = m_(o * r1), m_(dp * w_post)
        g["dw_post"] = (dp * oh).sum(0)
        back = oh * (wp * oh).mean(1, keepdim=True)
        dp = r1 * (wp + back if absolute else wp - back)
    g["do"] = dp
    return g
