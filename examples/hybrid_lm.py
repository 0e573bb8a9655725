"""A small hybrid language model on the library: selective scan blocks and a Gated
DeltaNet block with block norms between them, trained and served.

    python examples/hybrid_lm.py

Training runs packed sequences through the selective scan blocks with the
kernels' own gradients (three autograd functions); serving feeds a batch of
prompts of different lengths once, keeps every layer's states in a cache of
slots and continues token by token.  fp32, so that prompt and single tokens can
be compared closely.
"""
from __future__ import annotations

import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_attention_sequence_device_gb300 as g  # noqa: E402


# ---------------------------------------------------------------------------
# the kernels as autograd functions
# ---------------------------------------------------------------------------

class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b, cu):
        ctx.save_for_backward(x, w, b, cu)
        return g.gdn_ssm_conv_fwd(x, w, b, cu, output_state=False)[0]

    @staticmethod
    def backward(ctx, dy):
        x, w, b, cu = ctx.saved_tensors
        r = g.gdn_ssm_conv_bwd(dy.contiguous(), x, w, b, cu)
        return r["dx"], r["dw"].to(w.dtype), r["dbias"].to(b.dtype), None


class Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A_log, B, C, cu, D, z, dt_bias):
        y, _, ckpt = g.gdn_ssm_scan_fwd(x, dt, A_log, B, C, cu, D=D, z=z, dt_bias=dt_bias, output_final_state=False,
                                        checkpoints=True)
        ctx.save_for_backward(x, dt, A_log, B, C, cu, D, z, dt_bias, ckpt)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, dt, A_log, B, C, cu, D, z, dt_bias, ckpt = ctx.saved_tensors
        r = g.gdn_ssm_scan_bwd(dy.contiguous(), x, dt, A_log, B, C, cu, ckpt, D=D, z=z, dt_bias=dt_bias)
        return (*(r[k] for k in ("dx", "ddt", "dA_log", "dB", "dC")), None, r["dD"], r["dz"], r["ddt_bias"])


class BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, o, res, w_pre, w_post, gate, scale):
        y, res_out = g.gdn_block_norm_fwd(o, res, w_pre, w_post=w_post, gate=gate, scale=scale)
        ctx.save_for_backward(o, res_out, w_pre, w_post, gate, scale)
        return y, res_out

    @staticmethod
    def backward(ctx, dy, dres):
        o, res_out, w_pre, w_post, gate, scale = ctx.saved_tensors
        r = g.gdn_block_norm_bwd(dy, dres, o, res_out, w_pre, w_post=w_post, gate=gate, scale=scale)
        return r["do"], r["dres"], r["dw_pre"].to(w_pre.dtype), r["dw_post"].to(w_post.dtype), r["dgate"], r["dscale"]


# ---------------------------------------------------------------------------
# blocks
# ---------------------------------------------------------------------------

class SsmBlock:
    """in-projection -> conv -> projection to dt, B, C -> scan with gate -> out-projection"""

    def __init__(self, width, q, expand=2, N=16, rank=16, K=4):
        ch = expand * width
        rn = lambda *s, std: torch.randn(*s, generator=q, device="cuda") * std
        d0 = torch.exp(torch.rand(ch, generator=q, device="cuda") * 4.6 - 6.9)  # delta in [1e-3, 1e-1]
        self.p = dict(w_in=rn(2 * ch, width, std=width ** -0.5), conv_w=rn(ch, K, std=0.3), conv_b=rn(ch, std=0.0),
                      w_x=rn(rank + 2 * N, ch, std=ch ** -0.5), w_dt=rn(ch, rank, std=rank ** -0.5),
                      dt_bias=d0 + torch.log(-torch.expm1(-d0)), D=torch.ones(ch, device="cuda"),
                      A_log=torch.log(torch.arange(1, N + 1.0, device="cuda")).repeat(ch, 1),
                      w_out=rn(width, ch, std=ch ** -0.5))
        self.ch, self.N, self.rank, self.K = ch, N, rank, K

    def cache(self, slots):
        return dict(conv=torch.zeros(slots, self.K - 1, self.ch, device="cuda"),
                    h=torch.zeros(slots, self.ch, self.N, device="cuda"))

    def project(self, xc):
        """dt, B, C of the convolved channels; B and C are views of one projection."""
        p = self.p["w_x"]
        t = xc @ p.t()
        dt = t[:, :self.rank] @ self.p["w_dt"].t()
        bc = t[:, self.rank:].reshape(len(t), 2, 1, self.N)
        return dt, bc[:, 0], bc[:, 1]

    def train(self, x, cu):
        p = self.p
        xz = x @ p["w_in"].t()
        xc = Conv.apply(xz[:, :self.ch], p["conv_w"], p["conv_b"], cu)
        dt, B, C = self.project(xc)
        return Scan.apply(xc, dt, p["A_log"], B, C, cu, p["D"], xz[:, self.ch:], p["dt_bias"]) @ p["w_out"].t()

    def prompt(self, x, cu, c, slots):
        p = self.p
        xz = x @ p["w_in"].t()
        xc, conv = g.gdn_ssm_conv_fwd(xz[:, :self.ch], p["conv_w"], p["conv_b"], cu)
        dt, B, C = self.project(xc)
        y, h, _ = g.gdn_ssm_scan_fwd(xc, dt, p["A_log"], B, C, cu, D=p["D"], z=xz[:, self.ch:], dt_bias=p["dt_bias"])
        c["conv"][slots.long()], c["h"][slots.long()] = conv, h
        return y @ p["w_out"].t()

    def step(self, x, c, slots):
        p = self.p
        xz = x @ p["w_in"].t()
        xc = g.gdn_ssm_conv_step(xz[:, :self.ch], p["conv_w"], p["conv_b"], c["conv"], src=slots, dst=slots)
        dt, B, C = self.project(xc)
        y = g.gdn_ssm_scan_step(xc, dt, p["A_log"], B, C, c["h"], D=p["D"], z=xz[:, self.ch:], dt_bias=p["dt_bias"],
                                src=slots, dst=slots)
        return y @ p["w_out"].t()


class GdnBlock:
    """The Gated DeltaNet layer: its prompt is one gdn_layer_fwd; a single token is
    the conv's step and the chunk kernel on sequences of one token."""

    def __init__(self, width, q, H=4, d=32, K=4):
        rn = lambda *s, std: torch.randn(*s, generator=q, device="cuda") * std
        self.H, self.d, self.K, self.ch = H, d, K, 3 * H * d
        self.p = dict(w_in=rn(self.ch, width, std=width ** -0.5), w_ab=rn(2 * H, width, std=width ** -0.5),
                      w_z=rn(H * d, width, std=width ** -0.5), conv_w=rn(self.ch, K, std=0.3),
                      A_log=torch.log(torch.linspace(1, 8, H, device="cuda")), dt_bias=rn(H, std=0.5),
                      norm_w=torch.ones(d, device="cuda"), w_out=rn(width, H * d, std=(H * d) ** -0.5))

    def cache(self, slots):
        return dict(conv=torch.zeros(slots, self.K - 1, self.ch, device="cuda"),
                    S=torch.zeros(slots, self.H, self.d, self.d, device="cuda"))

    def prompt(self, x, cu, c, slots):
        p, H, d = self.p, self.H, self.d
        qkv, ab, z = x @ p["w_in"].t(), x @ p["w_ab"].t(), (x @ p["w_z"].t()).view(-1, H, d)
        y, S, _ = g.gdn_layer_fwd(qkv, p["conv_w"], None, ab[:, :H], ab[:, H:], p["A_log"], p["dt_bias"], z, p["norm_w"],
                                  cu, H, H, d, d, 1)
        # the conv's state: the last rows of every prompt
        _, conv = g.gdn_ssm_conv_fwd(qkv, p["conv_w"], None, cu)
        c["conv"][slots.long()], c["S"][slots.long()] = conv, S
        return y.reshape(len(x), H * d) @ p["w_out"].t()

    def step(self, x, c, slots):
        p, H, d, n = self.p, self.H, self.d, len(x)
        ab, z = x @ p["w_ab"].t(), (x @ p["w_z"].t()).view(n, H, d)
        qkv = g.gdn_ssm_conv_step(x @ p["w_in"].t(), p["conv_w"], None, c["conv"], src=slots, dst=slots)
        q, k, v = (t.view(n, H, d) for t in qkv.split(H * d, 1))
        gate = -torch.exp(p["A_log"]) * F.softplus(ab[:, :H] + p["dt_bias"])
        one = torch.arange(n + 1, dtype=torch.int32, device="cuda")
        o, S = g.gdn_chunk_fwd(q, k, v, gate, torch.sigmoid(ab[:, H:]), one, h0=c["S"][slots.long()], l2norm=True)
        c["S"][slots.long()] = S
        y = p["norm_w"] * o * torch.rsqrt(o.square().mean(-1, keepdim=True) + 1e-6) * F.silu(z)
        return y.reshape(n, H * d) @ p["w_out"].t()


class HybridLM:
    def __init__(self, vocab=97, width=128, kinds=("ssm", "gdn", "ssm"), seed=0):
        q = torch.Generator(device="cuda").manual_seed(seed)
        self.blocks = [SsmBlock(width, q) if k == "ssm" else GdnBlock(width, q) for k in kinds]
        self.embed = torch.randn(vocab, width, generator=q, device="cuda")
        one = lambda: torch.ones(width, device="cuda")
        # per block: the norm before it, the norm behind it, the gate's projection, the residual scale
        self.norms = [dict(pre=one(), post=one(), w_gate=torch.randn(width, width, generator=q, device="cuda") * width ** -0.5,
                           scale=0.5 * one()) for _ in kinds]
        self.last = one()

    def parameters(self):
        return ([self.embed, self.last] + [t for b in self.blocks for t in b.p.values()] +
                [t for n in self.norms for t in n.values()])

    def _walk(self, tokens, mix, norm):
        """Embedding, blocks and the norms between them; one block norm call per block."""
        res = self.embed[tokens]
        x = res * torch.rsqrt(res.square().mean(1, keepdim=True) + 1e-6) * self.norms[0]["pre"]
        for i, b in enumerate(self.blocks):
            n = self.norms[i]
            nxt = self.norms[i + 1]["pre"] if i + 1 < len(self.blocks) else self.last
            x, res = norm(mix(i, b, x), res, nxt, n["post"], x @ n["w_gate"].t(), n["scale"])
        return x @ self.embed.t() * self.embed.shape[1] ** -0.5

    def logits(self, tokens, cu):
        """Training logits of packed sequences (selective scan blocks only)."""
        return self._walk(tokens, lambda i, b, x: b.train(x, cu), BlockNorm.apply)

    def caches(self, slots):
        return [b.cache(slots) for b in self.blocks]

    @staticmethod
    def _norm(o, res, w_pre, w_post, gate, scale):
        return g.gdn_block_norm_fwd(o, res, w_pre, w_post=w_post, gate=gate, scale=scale, res_out=res)

    def prompt(self, tokens, cu, caches, slots):
        """Logits of every prompt token; the states after each prompt go into its slot."""
        return self._walk(tokens, lambda i, b, x: b.prompt(x, cu, caches[i], slots), self._norm)

    def step(self, tokens, caches, slots):
        """Logits of one token per request; its slots' states move on by one token."""
        return self._walk(tokens, lambda i, b, x: b.step(x, caches[i], slots), self._norm)


def offsets(lens):
    return torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)


def serve(lens=(5, 70, 1, 33), new=12, seed=0):
    """Greedy continuation of packed prompts.  Returns the tokens [requests, new],
    the logits of every step [requests, new, vocab], and the same logits from one
    prompt call over prompts and continuations together."""
    m = HybridLM(seed=seed)
    q = torch.Generator(device="cuda").manual_seed(seed + 1)
    lens = list(lens)
    prompts = [torch.randint(0, 97, (n,), generator=q, device="cuda") for n in lens]
    slots = torch.randperm(2 * len(lens), generator=q, device="cuda")[:len(lens)].to(torch.int32)
    caches = m.caches(2 * len(lens))
    cu = offsets(lens)
    at = m.prompt(torch.cat(prompts), cu, caches, slots)[cu[1:].long() - 1]
    tokens, logits = [], []
    for _ in range(new):
        logits.append(at)
        tokens.append(at.argmax(1))
        at = m.step(tokens[-1], caches, slots)
    tokens, logits = torch.stack(tokens, 1), torch.stack(logits, 1)
    whole = [torch.cat([p, tokens[i]]) for i, p in enumerate(prompts)]
    full = m.prompt(torch.cat(whole), offsets([len(w) for w in whole]), m.caches(2 * len(lens)), slots)
    full = torch.stack([f[n - 1:n - 1 + new] for f, n in zip(full.split([len(w) for w in whole]), lens)])
    return tokens, logits, full


def train(steps=30, seed=0):
    """Fits packed sequences of different lengths that count modulo the vocabulary; returns the losses."""
    m = HybridLM(kinds=("ssm", "ssm"), seed=seed)
    ps = [t.requires_grad_() for t in m.parameters()]
    opt = torch.optim.AdamW(ps, lr=3e-3)
    lens = [40, 7, 100, 1, 60]
    seqs = [(torch.arange(n + 1, device="cuda") * (i + 1) + i) % 97 for i, n in enumerate(lens)]
    x, y, cu = torch.cat([s[:-1] for s in seqs]), torch.cat([s[1:] for s in seqs]), offsets(lens)
    losses = []
    for _ in range(steps):
        loss = F.cross_entropy(m.logits(x, cu), y)
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


if __name__ == "__main__":
    losses = train()
    print("training: loss %.3f -> %.3f" % (losses[0], losses[-1]))
    tokens, logits, full = serve()
    print("serving: %d requests, %d tokens each; largest difference of logits between single tokens and one prompt %.1e"
          % (*tokens.shape, float((logits - full).abs().max())))
