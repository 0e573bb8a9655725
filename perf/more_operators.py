"""The two ends of a language model and the gated delta rule's single tokens as
measured cases: the gated delta rule and its layer for one token of each request
over a cache of states, the cross entropy over a large vocabulary straight from
hidden states and output weights (loss, and loss with both gradients; the logits
are not outputs), and the embedding lookup with its gradient.  Every case runs
either in elementary torch operations (own = False) or through the package's
entry points (own = True)."""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
IX = {"i64": torch.int64, "i32": torch.int32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of the layer: a single request, where latency counts
        dict(name="layer_step_one", kind="layer_step", B=1, Hk=16, Hv=32, dk=128, dv=128, dtype="bf16", z=True,
             fresh=False, pad=0),
        # one decode step of a serving batch, some requests new and the batch padded to its captured size
        dict(name="layer_step_batch", kind="layer_step", B=256, Hk=16, Hv=32, dk=128, dv=128, dtype="bf16", z=True,
             fresh=True, pad=5),
        # the bare rule with ready gates on a small model's heads, fp32
        dict(name="rule_step_small", kind="rule_step", B=33, Hk=4, Hv=8, dk=64, dv=32, dtype="f32", fresh=False, pad=0),
        # scoring of held-out text: the loss alone, an odd vocabulary
        dict(name="loss_score", kind="loss", T=4096, V=50021, W=2048, dtype="bf16", index="i64", ignore=0.0),
        # scoring of one document in fp32
        dict(name="loss_score_f32", kind="loss", T=513, V=32000, W=1024, dtype="f32", index="i64", ignore=0.1),
        # a training step's head over a large vocabulary
        dict(name="loss_train", kind="loss_train", T=8192, V=131072, W=2048, dtype="bf16", index="i64", ignore=0.02),
        # a short micro-batch of question and answer, where the questions have no loss
        dict(name="loss_train_short", kind="loss_train", T=130, V=32000, W=2048, dtype="bf16", index="i64", ignore=0.4),
        # a small model in fp32, odd sizes
        dict(name="loss_train_f32", kind="loss_train", T=1000, V=32003, W=1001, dtype="f32", index="i32", ignore=0.1),
        # the lookup of a training batch, scaled
        dict(name="embed_batch", kind="embed", T=65536, V=131072, W=4096, dtype="bf16", index="i64", pad=0.01),
        # the lookup of one decode step
        dict(name="embed_step", kind="embed", T=256, V=32003, W=2048, dtype="f32", index="i64", pad=0.0),
        # its gradient over a training batch: a few tokens thousands of times, most of the vocabulary not at all
        dict(name="embed_grad", kind="embed_grad", T=65536, V=131072, W=2048, dtype="bf16", index="i64", pad=0.01),
        # the gradient of a short batch in fp32, odd sizes
        dict(name="embed_grad_f32", kind="embed_grad", T=1000, V=32003, W=1001, dtype="f32", index="i32", pad=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["layer_step", "rule_step", "loss", "loss_train", "loss_train", "embed", "embed_grad"])
    c = dict(kind=kind, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if kind.endswith("step"):
        Hk = rng.choice([1, 2, 4, 8, 16, 16])
        c.update(B=_log(rng, 1, 256), Hk=Hk, Hv=Hk * rng.choice([1, 2, 2]), dk=rng.choice([32, 64, 128, 128]),
                 dv=rng.choice([32, 64, 128, 128]), fresh=rng.random() < 0.3)
        c["pad"] = rng.randrange(c["B"] // 4 + 1) if rng.random() < 0.3 else 0
        if kind == "layer_step":
            c["z"] = rng.random() < 0.8
        return c
    c["index"] = rng.choice(["i64", "i32"])
    c["W"] = _log(rng, 32, 4096) if rng.random() < 0.5 else 64 * _log(rng, 1, 64)
    c["V"] = _log(rng, 100, 131072)
    if kind.startswith("loss"):
        most = 1 << (41 if c["dtype"] == "bf16" else 37)
        c.update(T=min(_log(rng, 1, 16384), most // (c["V"] * c["W"])), ignore=rng.choice([0.0, 0.1, 0.5]))
    else:
        c.update(T=min(_log(rng, 1, 65536), (1 << 28) // c["W"]), V=min(c["V"], (1 << 28) // c["W"]),
                 pad=rng.choice([0.0, 0.1]))
    return c


def _unique(T, V):
    """Different tokens that T draws of _tokens() have on average."""
    edge = np.log(np.arange(1, V + 2)) / math.log(V + 1)
    return float(np.sum(-np.expm1(T * np.log1p(-np.diff(edge)))))


def work(case):
    k = case["kind"]
    e = 2 if case["dtype"] == "bf16" else 4
    if k.endswith("step"):
        B, Hk, Hv, dk, dv = (case[n] for n in ("B", "Hk", "Hv", "dk", "dv"))
        live = B - case["pad"]
        fresh = len(range(0, live, 8)) if case["fresh"] else 0
        row = e * (2 * Hk * dk + 2 * Hv * dv) + (4 + e) * Hv + (e * Hv * (dv - 1) if case.get("z") else 0)
        return dict(bytes=4 * (2 * live - fresh) * Hv * dk * dv + B * row, flops=7 * live * Hv * dk * dv)
    T, V, W = case["T"], case["V"], case["W"]
    ix = 8 if case["index"] == "i64" else 4
    if k == "loss":
        return dict(bytes=e * (T + V) * W + (ix + 4) * T, flops=2 * T * V * W)
    if k == "loss_train":
        return dict(bytes=2 * e * (T + V) * W + (ix + 8) * T, flops=6 * T * V * W)
    if k == "embed":
        return dict(bytes=e * W * (T + _unique(T, V)) + ix * T, flops=T * W)
    return dict(bytes=e * W * (T + V) + ix * T, flops=2 * T * W)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DT[case["dtype"]]

    def rn(*shape, std=1.0, mean=0.0, dtype=None):
        t = torch.empty(shape, dtype=torch.float32 if dtype is None else dtype, device=dev)
        return t.normal_(mean, std, generator=gen)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    def _tokens(T, V):
        """Tokens with the long tail of text: token i about as often as 1 / (i + 1)."""
        t = torch.exp(uniform(T).double() * math.log(V + 1.0)) - 1.0
        return t.long().clamp(0, V - 1)

    k = case["kind"]
    s = dict(case=case, kind=k)
    if k.endswith("step"):
        B, Hk, Hv, dk, dv = (case[n] for n in ("B", "Hk", "Hv", "dk", "dv"))
        live = B - case["pad"]
        # a cache with twice the batch's slots: each request reads one and writes another (a fork of its state);
        # a new request reads none, a padded row writes none
        slots = torch.randperm(2 * B, generator=gen, device=dev).to(torch.int32)
        src, dst = slots[:B].clone(), slots[B:].clone()
        if case["fresh"]:
            src[:live:8] = -1
        dst[live:] = -1
        s.update(live=live, src=src, dst=dst, states=rn(2 * B, Hv, dk, dv, std=0.1), o=torch.empty(B, Hv, dv, dtype=dt, device=dev))
        x = rn(B, 2 * Hk * dk + Hv * dv)
        s["qkv"] = (x * torch.sigmoid(x)).to(dt)  # the short conv's output
        if k == "layer_step":
            ab = rn(B, 2, Hv, dtype=dt)  # one projection's output
            s.update(a=ab[:, 0], b=ab[:, 1], A_log=torch.log(1.0 + 15.0 * uniform(Hv)), dt_bias=rn(Hv),
                     zgate=rn(B, Hv, dv, dtype=dt) if case["z"] else None,
                     norm_w=rn(dv, mean=1.0, std=0.1, dtype=dt) if case["z"] else None)
        else:
            q, kk, v = s["qkv"].split([Hk * dk, Hk * dk, Hv * dv], 1)
            s.update(q=q.unflatten(1, (Hk, dk)), k=kk.unflatten(1, (Hk, dk)), v=v.unflatten(1, (Hv, dv)),
                     g=-torch.log1p(torch.exp(rn(B, Hv) - 2.0)), beta=torch.sigmoid(rn(B, Hv)).to(dt))
        return s
    T, V, W = case["T"], case["V"], case["W"]
    tok = _tokens(T, V)
    if k.startswith("loss"):
        # output weights of unit norm; hidden states that know their next token more or less well
        w = rn(V, W, std=W ** -0.5, dtype=dt)
        h = rn(T, W)
        h += (14.0 * uniform(T))[:, None] * w[tok].float()
        tok[uniform(T) < case["ignore"]] = -100
        s.update(h=h.to(dt), w=w, targets=tok.to(IX[case["index"]]), scale=1.0)
        if k == "loss_train":
            # the mean over a batch whose documents are weighted
            s["dloss"] = (0.5 + uniform(T)) / T
        return s
    tok[uniform(T) < case["pad"]] = -1
    s.update(tokens=tok.to(IX[case["index"]]), scale=math.sqrt(W))
    if k == "embed":
        s["table"] = rn(V, W, std=W ** -0.5, dtype=dt)
    else:
        s["dy"] = rn(T, W, dtype=dt)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return _OWN[s["kind"]](s) if own else _PLAIN[s["kind"]](s)


def _pkg():
    import linear_attention_sequence_device_gb300 as g
    return g


def _own_rule_step(s):
    o = _pkg().gdn_chunk_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["states"], src=s["src"], dst=s["dst"],
                              l2norm=True, out=s["o"])
    return dict(o=o, states=s["states"])


def _own_layer_step(s):
    c = s["case"]
    y = _pkg().gdn_layer_step(s["qkv"], s["a"], s["b"], s["A_log"], s["dt_bias"], s["zgate"], s["norm_w"], s["states"],
                              c["Hk"], c["Hv"], c["dk"], c["dv"], src=s["src"], dst=s["dst"], eps=1e-6, out=s["o"])
    return dict(y=y, states=s["states"])


def _own_loss(s):
    loss, lse = _pkg().gdn_vocab_loss_fwd(s["h"], s["w"], s["targets"], scale=s["scale"])
    return dict(loss=loss, lse=lse)


def _own_loss_train(s):
    g = _pkg()
    loss, lse = g.gdn_vocab_loss_fwd(s["h"], s["w"], s["targets"], scale=s["scale"])
    r = g.gdn_vocab_loss_bwd(s["dloss"], s["h"], s["w"], s["targets"], lse, scale=s["scale"])
    return dict(loss=loss, lse=lse, dh=r["dh"], dw=r["dw"])


def _own_embed(s):
    return dict(y=_pkg().gdn_embed_fwd(s["tokens"], s["table"], scale=s["scale"]))


def _own_embed_grad(s):
    return dict(dtable=_pkg().gdn_embed_bwd(s["dy"], s["tokens"], s["case"]["V"], scale=s["scale"]))


# ---- plain forms ----------------------------------------------------------

def _rule(s, q, k, v, g, beta):
    """One token of the gated delta rule; q, k as they come, everything fp32."""
    c, live = s["case"], s["live"]
    unit = lambda x: x * torch.rsqrt((x * x).sum(2, keepdim=True) + 1e-6)
    per = lambda x: unit(x[:live].float()).repeat_interleave(c["Hv"] // c["Hk"], 1)
    q, k, v = per(q) * c["dk"] ** -0.5, per(k), v[:live].float()
    src = s["src"][:live].long()
    S = torch.where((src >= 0)[:, None, None, None], s["states"][src.clamp(min=0)], 0.0)
    S = torch.exp(g[:live])[:, :, None, None] * S
    u = v - (S * k[:, :, :, None]).sum(2)
    S = S + (beta[:live].float()[:, :, None] * k)[:, :, :, None] * u[:, :, None, :]
    s["states"][s["dst"][:live].long()] = S
    return (S * q[:, :, :, None]).sum(2)


def _padded(s, o):
    out = torch.zeros(s["case"]["B"], *o.shape[1:], dtype=s["qkv"].dtype, device=o.device)
    out[:s["live"]] = o.to(out.dtype)
    return out


def _softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(v.clamp(max=20.0))))


def _plain_rule_step(s):
    return dict(o=_padded(s, _rule(s, s["q"], s["k"], s["v"], s["g"], s["beta"])), states=s["states"])


def _plain_layer_step(s):
    c, n = s["case"], s["live"]
    q, k, v = s["qkv"].split([c["Hk"] * c["dk"], c["Hk"] * c["dk"], c["Hv"] * c["dv"]], 1)
    g = -torch.exp(s["A_log"]) * _softplus(s["a"].float() + s["dt_bias"])
    o = _rule(s, q.unflatten(1, (c["Hk"], c["dk"])), k.unflatten(1, (c["Hk"], c["dk"])),
              v.unflatten(1, (c["Hv"], c["dv"])), g, torch.sigmoid(s["b"].float()))
    if s["zgate"] is not None:
        z = s["zgate"][:n].float()
        o = s["norm_w"].float() * o * torch.rsqrt((o * o).mean(2, keepdim=True) + 1e-6) * (z * torch.sigmoid(z))
    return dict(y=_padded(s, o), states=s["states"])


def _logits(s):
    """Logits, their log sum of exponentials, the targets' logits and which tokens count."""
    t = s["targets"].long()
    x = s["h"].float() @ s["w"].float().t()
    if s["scale"] != 1.0:
        x *= s["scale"]
    top = x.amax(1)
    lse = top + torch.log(torch.exp(x - top[:, None]).sum(1))
    t, real = t.clamp(min=0), t >= 0
    return x, lse, x.gather(1, t[:, None])[:, 0], t, real


def _plain_loss(s):
    _, lse, at, _, real = _logits(s)
    return dict(loss=torch.where(real, lse - at, 0.0), lse=lse)


def _plain_loss_train(s):
    x, lse, at, t, real = _logits(s)
    p = torch.exp(x.sub_(lse[:, None]))
    p[torch.arange(len(t), device=t.device), t] -= 1.0
    p *= torch.where(real, s["dloss"] * s["scale"], 0.0)[:, None]
    dh, dw = p @ s["w"].float(), p.t() @ s["h"].float()
    return dict(loss=torch.where(real, lse - at, 0.0), lse=lse, dh=dh.to(s["h"].dtype), dw=dw.to(s["w"].dtype))


def _plain_embed(s):
    t = s["tokens"].long()
    y = torch.where((t >= 0)[:, None], s["table"][t.clamp(min=0)].float() * s["scale"], 0.0)
    return dict(y=y.to(s["table"].dtype))


def _plain_embed_grad(s):
    t = s["tokens"].long()
    d = torch.zeros(s["case"]["V"], s["case"]["W"], dtype=torch.float32, device=t.device)
    d.index_add_(0, t.clamp(min=0), torch.where((t >= 0)[:, None], s["dy"].float(), 0.0))
    return dict(dtable=d.mul_(s["scale"]).to(s["dy"].dtype))


_PLAIN = dict(rule_step=_plain_rule_step, layer_step=_plain_layer_step, loss=_plain_loss, loss_train=_plain_loss_train,
              embed=_plain_embed, embed_grad=_plain_embed_grad)
_OWN = dict(rule_step=_own_rule_step, layer_step=_own_layer_step, loss=_own_loss, loss_train=_own_loss_train,
            embed=_own_embed, embed_grad=_own_embed_grad)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    v = {n: (t.double() if isinstance(t, torch.Tensor) and t.is_floating_point() else t) for n, t in s.items()}
    return dict(rule_step=_exact_rule_step, layer_step=_exact_layer_step, loss=_exact_loss, loss_train=_exact_loss,
                embed=_exact_embed, embed_grad=_exact_embed_grad)[case["kind"]](v)


def _exact_rule(v, g, beta):
    """(I - beta k k^T) e^g S + beta k v^T, request by request, and its product with q."""
    c = v["case"]
    Hk, Hv, dk, dv = (c[n] for n in ("Hk", "Hv", "dk", "dv"))
    states, o = v["states"].clone(), v["states"].new_zeros(c["B"], Hv, dv)
    heads = torch.arange(Hv, device=o.device) // (Hv // Hk)
    eye = torch.eye(dk, dtype=o.dtype, device=o.device)
    src, dst = v["src"].tolist(), v["dst"].tolist()
    for i in range(c["B"]):
        if dst[i] < 0:
            continue
        row = v["qkv"][i]
        q, k = (row[j * Hk * dk:(j + 1) * Hk * dk].view(Hk, dk)[heads] for j in (0, 1))
        q, k = (t / torch.sqrt((t ** 2).sum(1, keepdim=True) + 1e-6) for t in (q, k))
        val = row[2 * Hk * dk:].view(Hv, dv)
        S = v["states"][src[i]] if src[i] >= 0 else torch.zeros_like(states[0])
        b = beta[i][:, None, None]
        S = (eye - b * torch.einsum("hi,hj->hij", k, k)) @ (S * g[i].exp()[:, None, None]) \
            + b * torch.einsum("hi,hj->hij", k, val)
        states[dst[i]] = S
        o[i] = torch.einsum("hij,hi->hj", S, q) / math.sqrt(dk)
    return o, states


def _exact_rule_step(v):
    o, states = _exact_rule(v, v["g"], v["beta"])
    return dict(o=o, states=states)


def _exact_layer_step(v):
    g = -torch.exp(v["A_log"]) * torch.logaddexp(v["a"] + v["dt_bias"], torch.zeros_like(v["a"]))
    o, states = _exact_rule(v, g, 1.0 / (1.0 + torch.exp(-v["b"])))
    if v["zgate"] is not None:
        o = o / torch.sqrt(o.square().mean(2, keepdim=True) + 1e-6) * v["norm_w"]
        o = o * v["zgate"] / (1.0 + torch.exp(-v["zgate"]))
    return dict(y=o, states=states)


def _exact_loss(v):
    """Blocks of tokens against the whole vocabulary."""
    T, V = v["case"]["T"], v["case"]["V"]
    h, w, t = v["h"], v["w"], v["targets"].long()
    loss, lse = h.new_zeros(T), h.new_empty(T)
    grads = "dloss" in v
    dh, dw = torch.zeros_like(h), torch.zeros_like(w)
    step = max(1, (1 << 28) // V)
    for a in range(0, T, step):
        x = h[a:a + step] @ w.T * v["scale"]
        z = torch.logsumexp(x, 1)
        lse[a:a + step] = z
        rows = (t[a:a + step] >= 0).nonzero()[:, 0]
        cols = t[a + rows]
        loss[a + rows] = z[rows] - x[rows, cols]
        if grads:
            p = torch.softmax(x, 1)
            p[rows, cols] -= 1.0
            f = torch.zeros_like(z)
            f[rows] = v["dloss"][a + rows] * v["scale"]
            p *= f[:, None]
            dh[a:a + step] = p @ w
            dw.addmm_(p.T, h[a:a + step])
    return dict(loss=loss, lse=lse, dh=dh, dw=dw) if grads else dict(loss=loss, lse=lse)


def _exact_embed(v):
    y = v["table"].new_zeros(v["case"]["T"], v["case"]["W"])
    at = (v["tokens"] >= 0).nonzero()[:, 0]
    y[at] = v["table"].index_select(0, v["tokens"][at].long()) * v["scale"]
    return dict(y=y)


def _exact_embed_grad(v):
    """Rows in the tokens' order, summed between the places where the token changes."""
    d = v["dy"].new_zeros(v["case"]["V"], v["case"]["W"])
    tok, order = torch.sort(v["tokens"].long(), stable=True)
    real = tok >= 0
    tok, order = tok[real], order[real]
    ids, count = torch.unique_consecutive(tok, return_counts=True)
    seg = torch.repeat_interleave(torch.arange(len(ids), device=tok.device), count)
    rows = d.new_zeros(len(ids), d.shape[1])
    rows.index_put_((seg,), v["dy"][order], accumulate=True)
    d[ids] = rows * v["scale"]
    return dict(dtable=d)
