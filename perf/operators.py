"""The selective scan layer's operators as measured cases: the short causal
convolution with a state per sequence (prompt, gradient, single token), the
selective state space scan (prompt, training step, single token) and the block
norm (post norm, gate, residual scale, residual add, pre norm; forward and
backward).  Every case runs either in elementary torch operations (own = False)
or through the package's entry points (own = True)."""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64  # tokens per chunk of the plain scan


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a prefill batch of mixed prompts: the packed workload's conv (8192 fused channels)
        dict(name="conv_prompt_packed", kind="conv_fwd", T=32768, C=8192, K=4, dtype="bf16", lens="uniform:512:8192",
             len_seed=1, bias=False, state=False),
        # training on many short documents with a carried history
        dict(name="conv_grad_ragged", kind="conv_bwd", T=65536, C=2048, K=4, dtype="bf16", lens="geometric:300",
             len_seed=3, bias=True, state=True),
        # one decode step of a serving batch
        dict(name="conv_step_batch", kind="conv_step", T=256, C=8192, K=4, dtype="bf16", bias=True),
        # prefill of the packed workload: 4096 channels, gate and skip
        dict(name="scan_prompt_packed", kind="scan_fwd", T=32768, D=4096, N=16, G=1, dtype="bf16",
             lens="uniform:512:8192", len_seed=1, z=True, skip=True, bias=True, h0=False),
        # one long prompt, continued from a cached state
        dict(name="scan_prompt_long", kind="scan_fwd", T=131072, D=2048, N=16, G=1, dtype="bf16", lens="one",
             len_seed=0, z=True, skip=True, bias=True, h0=True),
        # a chat-sized prompt in fp32 with an odd state size, two groups and no gate
        dict(name="scan_prompt_short", kind="scan_fwd", T=257, D=1536, N=12, G=2, dtype="f32", lens="one", len_seed=0,
             z=False, skip=True, bias=True, h0=False),
        # a training step on the packed workload
        dict(name="scan_train_packed", kind="scan_train", T=32768, D=4096, N=16, G=1, dtype="bf16",
             lens="uniform:512:8192", len_seed=1, z=True, skip=True, bias=True, h0=False),
        # a training step on short documents of odd lengths, fp32, four groups, carried states
        dict(name="scan_train_ragged", kind="scan_train", T=8191, D=1024, N=16, G=4, dtype="f32", lens="geometric:300",
             len_seed=3, z=True, skip=True, bias=True, h0=True),
        # one decode step: a single request, where latency counts
        dict(name="scan_step_one", kind="scan_step", T=1, D=4096, N=16, G=1, dtype="bf16", z=True, skip=True,
             bias=True),
        # one decode step of a serving batch
        dict(name="scan_step_batch", kind="scan_step", T=256, D=4096, N=16, G=1, dtype="bf16", z=True, skip=True,
             bias=True),
        # between two blocks, a decode batch
        dict(name="norm_decode", kind="norm_fwd", T=64, D=4096, dtype="bf16", res="f32", post=True, gate=True,
             scale=True),
        # between two blocks, the gradient over a training batch
        dict(name="norm_grad", kind="norm_bwd", T=32768, D=4096, dtype="bf16", res="bf16", post=True, gate=True,
             scale=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_fwd", "scan_train", "scan_train",
                       "scan_step", "norm_fwd", "norm_bwd"])
    c = dict(kind=kind, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if not kind.endswith("step"):
        c["lens"] = rng.choice(["one", "split:%d" % _log(rng, 2, 64), "geometric:300", "uniform:512:8192"])
        c["len_seed"] = rng.randrange(1 << 30)
    if kind.startswith("conv"):
        C = 8 * _log(rng, 4, 1024)
        T = _log(rng, 1, 512) if kind == "conv_step" else min(_log(rng, 1, 65536), (1 << 28) // C // 2)
        c.update(T=T, C=C, K=rng.choice([2, 3, 4, 4, 4]), bias=rng.random() < 0.7)
        if kind != "conv_step":
            c["state"] = rng.random() < 0.5
    elif kind.startswith("scan"):
        G = rng.choice([1, 1, 1, 2, 4])
        D = G * 8 * _log(rng, 2, 512 // G)
        N = rng.choice([4, 8, 12, 16, 16, 16, 16, 24, 32, 64])
        if kind == "scan_step":
            T = _log(rng, 1, 256)
        else:
            T = min(_log(rng, 1, 65536), (1 << 30) // (D * N))
        c.update(T=T, D=D, N=N, G=G, z=rng.random() < 0.8, skip=rng.random() < 0.8, bias=rng.random() < 0.9)
        if kind != "scan_step":
            c["h0"] = rng.random() < 0.5
    else:
        D = 8 * _log(rng, 8, 1024)
        T = min(_log(rng, 1, 65536), (1 << 27) // D)
        c.update(T=T, D=D, res=rng.choice(["f32", c["dtype"]]), post=rng.random() < 0.8, gate=rng.random() < 0.7,
                 scale=rng.random() < 0.7)
        del c["lens"], c["len_seed"]
    return c


def _lengths(case):
    """Sequence lengths of a case: whole numbers that sum to T."""
    T, spec = case["T"], case["lens"]
    rng = np.random.default_rng(case["len_seed"])
    if spec == "one":
        return [T]
    if spec.startswith("split"):  # any cuts, empty sequences among them
        cuts = np.sort(rng.integers(0, T + 1, int(spec.split(":")[1]) - 1))
        return np.diff(np.concatenate([[0], cuts, [T]])).tolist()
    out, left = [], T
    while left > 0:
        if spec.startswith("geometric"):
            n = int(np.clip(rng.geometric(1.0 / float(spec.split(":")[1])), 1, 4096))
        else:
            lo, hi = (int(v) for v in spec.split(":")[1:])
            n = int(rng.integers(lo, hi + 1))
        out.append(min(n, left))
        left -= out[-1]
    return out


def work(case):
    k, T = case["kind"], case["T"]
    e = 2 if case["dtype"] == "bf16" else 4
    if k.startswith("conv"):
        C, K = case["C"], case["K"]
        hist = (K - 1) * C
        if k == "conv_step":
            return dict(bytes=e * (2 * T * C + 2 * T * hist + C * K), flops=T * C * (2 * K + 4))
        n = len(_lengths(case))
        st = n * hist
        if k == "conv_fwd":
            return dict(bytes=e * (2 * T * C + C * K + st * (1 + case["state"])), flops=T * C * (2 * K + 4))
        return dict(bytes=e * (3 * T * C + C * K + st * case["state"]) + 4 * (2 * st + C * (K + 1)),
                    flops=T * C * (6 * K + 10))
    if k.startswith("scan"):
        D, N, G = case["D"], case["N"], case["G"]
        act = 2 + case["z"]  # x, dt, z
        if k == "scan_step":
            return dict(bytes=e * T * ((act + 1) * D + 2 * G * N) + 8 * T * D * N + 4 * D * N, flops=7 * T * D * N)
        n = len(_lengths(case))
        st = 4 * n * D * N
        if k == "scan_fwd":
            return dict(bytes=e * T * ((act + 1) * D + 2 * G * N) + st * (1 + case["h0"]) + 4 * D * N,
                        flops=7 * T * D * N)
        # in: x, dt, z, dy, B, C, h0, dh_final; out: y, dx, ddt, dz, dB, dC, h_final, dh0
        return dict(bytes=e * T * ((2 * act + 2) * D + 4 * G * N) + st * (3 + case["h0"]) + 8 * D * N,
                    flops=22 * T * D * N)
    D = case["D"]
    r = 4 if case["res"] == "f32" else 2
    if k == "norm_fwd":
        return dict(bytes=T * D * (e * (2 + case["gate"]) + 2 * r), flops=12 * T * D)
    return dict(bytes=T * D * (e * (3 + 2 * case["gate"]) + 3 * r), flops=30 * T * D)


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

    def ru(*shape, lo, hi):
        return torch.empty(shape, dtype=torch.float32, device=dev).uniform_(lo, hi, generator=gen)

    k, T = case["kind"], case["T"]
    s = dict(case=case, kind=k)
    if "lens" in case:
        lens = _lengths(case)
        cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        s.update(lens=lens, cu_host=cu, cu=torch.from_numpy(cu).to(dev))
    if k.startswith("conv"):
        C, K = case["C"], case["K"]
        s.update(x=rn(T, C, dtype=dt), w=rn(C, K, std=0.5, dtype=dt), b=rn(C, std=0.1, dtype=dt) if case["bias"] else None)
        if k == "conv_step":
            # a cache with twice the batch's slots: each request reads one and writes another (a fork of its state)
            slots = torch.randperm(2 * T, generator=gen, device=dev).to(torch.int32)
            s.update(states=rn(2 * T, K - 1, C, dtype=dt), src=slots[:T].contiguous(), dst=slots[T:].contiguous(),
                     y=torch.empty(T, C, dtype=dt, device=dev))
            return s
        n = len(s["lens"])
        s["state"] = rn(n, K - 1, C, dtype=dt) if case["state"] else None
        if k == "conv_bwd":
            s["dy"] = rn(T, C, dtype=dt)
            s["dstate_out"] = rn(n, K - 1, C)
    elif k.startswith("scan"):
        D, N, G = case["D"], case["N"], case["G"]
        x = rn(T, D)
        s["x"] = (x * torch.sigmoid(x)).to(dt)  # the conv's output
        s["dt"] = rn(T, D, std=0.5, dtype=dt)
        # B and C as slices of one projection's output
        bc = rn(T, 2, G, N, dtype=dt)
        s["B"], s["C"] = bc[:, 0], bc[:, 1]
        s["A_log"] = torch.log(torch.arange(1, N + 1, dtype=torch.float32, device=dev)).expand(D, N) \
            + rn(D, N, std=0.05)
        # the usual initialisation: softplus(dt_bias) log-uniform in [1e-3, 1e-1]
        d0 = torch.exp(ru(D, lo=math.log(1e-3), hi=math.log(1e-1)))
        s["dt_bias"] = d0 + torch.log(-torch.expm1(-d0)) if case["bias"] else None
        s["D"] = rn(D, std=0.1, mean=1.0) if case["skip"] else None
        s["z"] = rn(T, D, dtype=dt) if case["z"] else None
        if k == "scan_step":
            slots = torch.randperm(2 * T, generator=gen, device=dev).to(torch.int32)
            s.update(states=rn(2 * T, D, N, std=0.5), src=slots[:T].contiguous(), dst=slots[T:].contiguous(),
                     y=torch.empty(T, D, dtype=dt, device=dev))
            return s
        n = len(s["lens"])
        s["h0"] = rn(n, D, N, std=0.5) if case["h0"] else None
        if k == "scan_train":
            s["dy"] = rn(T, D, dtype=dt)
            s["dh_final"] = rn(n, D, N, std=0.1)
        if not own:
            s["chunks"] = _chunk_plan(s["lens"], s["cu_host"], dev)
    else:
        D, rdt = case["D"], DT[case["res"]]
        s.update(o=rn(T, D, dtype=dt), res=rn(T, D, std=2.0, dtype=rdt),
                 w_pre=rn(D, std=0.1, mean=1.0, dtype=dt),
                 w_post=rn(D, std=0.1, mean=1.0, dtype=dt) if case["post"] else None,
                 gate=rn(T, D, dtype=dt) if case["gate"] else None,
                 scale=rn(D, std=0.02, mean=0.1) if case["scale"] else None)
        if k == "norm_bwd":
            s.update(dy=rn(T, D, dtype=dt), dres=rn(T, D, dtype=rdt))
    return s


def _chunk_plan(lens, cu, dev):
    """Every sequence cut into chunks of CHUNK tokens from its own start: the
    token of every (chunk, row), which rows are real, and per chunk rank the
    chunks and sequences that have it (for the walk over chunks)."""
    seq, start, end, first = [], [], [], []
    for n, L in enumerate(lens):
        first.append(len(seq))
        for c in range(0, L, CHUNK):
            seq.append(n)
            start.append(int(cu[n]) + c)
            end.append(int(cu[n]) + min(c + CHUNK, L))
    nc = len(seq)
    tok = np.asarray(start, np.int64)[:, None] + np.arange(CHUNK) if nc else np.zeros((0, CHUNK), np.int64)
    real = tok < np.asarray(end, np.int64)[:, None] if nc else np.zeros((0, CHUNK), bool)
    tok = np.where(real, tok, tok[:, :1])
    count = [(L + CHUNK - 1) // CHUNK for L in lens]
    walk = []
    for k in range(max(count, default=0)):
        ns = [n for n in range(len(lens)) if count[n] > k]
        walk.append((torch.tensor([first[n] + k for n in ns], device=dev), torch.tensor(ns, device=dev),
                     torch.tensor([first[n] + k for n in ns if count[n] == k + 1], device=dev, dtype=torch.long),
                     torch.tensor([n for n in ns if count[n] == k + 1], device=dev, dtype=torch.long)))
    return dict(nc=nc, tok=torch.from_numpy(tok).to(dev), real=torch.from_numpy(real).to(dev), walk=walk,
                seq=torch.tensor(seq, device=dev, dtype=torch.long))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return _OWN[s["kind"]](s) if own else _PLAIN[s["kind"]](s)


def _pkg():
    import linear_attention_sequence_device_gb300 as g
    return g


def _own_conv_fwd(s):
    y, st = _pkg().gdn_ssm_conv_fwd(s["x"], s["w"], s["b"], s["cu"], state=s["state"])
    return dict(y=y, state=st)


def _own_conv_bwd(s):
    # the gradient of a bias of zeros is among the outputs where there is none
    b = s["b"] if s["b"] is not None else torch.zeros_like(s["w"][:, 0])
    r = _pkg().gdn_ssm_conv_bwd(s["dy"], s["x"], s["w"], b, s["cu"], state=s["state"], dstate_out=s["dstate_out"])
    return {k: r[k] for k in ("dx", "dw", "dbias", "dstate")}


def _own_conv_step(s):
    y = _pkg().gdn_ssm_conv_step(s["x"], s["w"], s["b"], s["states"], src=s["src"], dst=s["dst"], out=s["y"])
    return dict(y=y, states=s["states"])


def _own_scan_fwd(s):
    y, hf, _ = _pkg().gdn_ssm_scan_fwd(s["x"], s["dt"], s["A_log"], s["B"], s["C"], s["cu"], D=s["D"], z=s["z"],
                                       dt_bias=s["dt_bias"], h0=s["h0"])
    return dict(y=y, h_final=hf)


def _own_scan_train(s):
    g = _pkg()
    a = (s["x"], s["dt"], s["A_log"], s["B"], s["C"], s["cu"])
    kw = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"], h0=s["h0"])
    y, hf, ckpt = g.gdn_ssm_scan_fwd(*a, checkpoints=True, **kw)
    r = g.gdn_ssm_scan_bwd(s["dy"], *a, ckpt, dh_final=s["dh_final"], **kw)
    return dict(y=y, h_final=hf, **{k: r[k] for k in _SCAN_GRADS})


def _own_scan_step(s):
    y = _pkg().gdn_ssm_scan_step(s["x"], s["dt"], s["A_log"], s["B"], s["C"], s["states"], D=s["D"], z=s["z"],
                                 dt_bias=s["dt_bias"], src=s["src"], dst=s["dst"], out=s["y"])
    return dict(y=y, states=s["states"])


def _own_norm_fwd(s):
    y, r = _pkg().gdn_block_norm_fwd(s["o"], s["res"], s["w_pre"], w_post=s["w_post"], gate=s["gate"],
                                     scale=s["scale"], eps=1e-6)
    return dict(y=y, res=r)


def _own_norm_bwd(s):
    r = _pkg().gdn_block_norm_bwd(s["dy"], s["dres"], s["o"], s["res"], s["w_pre"], w_post=s["w_post"],
                                  gate=s["gate"], scale=s["scale"], eps=1e-6)
    return {k: r[k] for k in ("do", "dres", "dgate", "dw_pre", "dw_post", "dscale")}


_SCAN_GRADS = ("dx", "ddt", "dz", "dA_log", "dB", "dC", "dD", "ddt_bias", "dh0")


# ---- plain forms ----------------------------------------------------------

def _rows(s):
    """Sequence and position within it of every packed token."""
    cu = s["cu"].long()
    t = torch.arange(s["case"]["T"], device=cu.device)
    sid = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return t, sid, t - cu[sid]


def _taps(s, lag):
    """x `lag` tokens earlier, from the sequence's history where it starts later."""
    K = s["case"]["K"]
    t, sid, pos = _rows(s)
    v = s["x"].float()[(t - lag).clamp(min=0)]
    early = (pos < lag).nonzero()[:, 0]
    if s["state"] is None:
        v[early] = 0.0
    else:
        v[early] = s["state"].float()[sid[early], K - 1 - lag + pos[early]]
    return v


def _conv_pre(s):
    K = s["case"]["K"]
    w = s["w"].float()
    acc = 0.0 if s["b"] is None else s["b"].float()
    for j in range(K):
        acc = acc + _taps(s, K - 1 - j) * w[:, j]
    return acc


def _last_rows(s):
    """For every (sequence, row of its final state): the packed token it
    holds, or the row of the initial state where the sequence is shorter."""
    K = s["case"]["K"]
    cu = s["cu"].long()
    L = (cu[1:] - cu[:-1])[:, None]
    m = torch.arange(K - 1, device=cu.device)[None, :]
    p = L - (K - 1) + m
    return p >= 0, (cu[:-1, None] + p).clamp(min=0), (L + m).clamp(max=K - 2)


def _plain_conv_fwd(s):
    dt = s["x"].dtype
    pre = _conv_pre(s)
    y = (pre * torch.sigmoid(pre)).to(dt)
    inside, tok, hist = _last_rows(s)
    n = torch.arange(len(s["lens"]), device=tok.device)[:, None]
    old = s["state"][n, hist] if s["state"] is not None else torch.zeros((), dtype=dt, device=tok.device)
    st = torch.where(inside[:, :, None], s["x"][tok.clamp(max=s["case"]["T"] - 1)], old)
    return dict(y=y, state=st)


def _plain_conv_bwd(s):
    K, C, T = s["case"]["K"], s["case"]["C"], s["case"]["T"]
    t, sid, pos = _rows(s)
    cu = s["cu"].long()
    left = cu[sid + 1] - t  # tokens from here to the sequence's end
    pre = _conv_pre(s)
    sg = torch.sigmoid(pre)
    ds = s["dy"].float() * sg * (1.0 + pre * (1.0 - sg))
    del pre, sg
    w = s["w"].float()
    dx = torch.zeros_like(ds)
    dw = torch.empty(C, K, device=ds.device)
    dstate = torch.zeros(len(s["lens"]), K - 1, C, device=ds.device)
    for j in range(K):
        lag = K - 1 - j
        dw[:, j] = (ds * _taps(s, lag)).sum(0)
        nxt = ds[(t + lag).clamp(max=T - 1)] * w[:, j]
        nxt[left <= lag] = 0.0
        dx += nxt
        early = (pos < lag).nonzero()[:, 0]
        dstate.index_put_((sid[early], K - 1 - lag + pos[early]), ds[early] * w[:, j], accumulate=True)
    inside, tok, hist = _last_rows(s)
    n = torch.arange(len(s["lens"]), device=tok.device)[:, None].expand_as(tok)
    dx.index_put_((tok[inside],), s["dstate_out"][inside], accumulate=True)
    dstate.index_put_((n[~inside], hist[~inside]), s["dstate_out"][~inside], accumulate=True)
    return dict(dx=dx.to(s["x"].dtype), dw=dw, dbias=ds.sum(0), dstate=dstate)


def _plain_conv_step(s):
    K = s["case"]["K"]
    old = s["states"][s["src"].long()]
    rows = torch.cat([old, s["x"][:, None]], 1)
    pre = (rows.float() * s["w"].float().t()).sum(1)
    if s["b"] is not None:
        pre = pre + s["b"].float()
    s["states"][s["dst"].long()] = rows[:, 1:]
    return dict(y=(pre * torch.sigmoid(pre)).to(s["x"].dtype), states=s["states"])


def _softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(v.clamp(max=20.0))))


def _channel_blocks(s):
    D, G, N = s["case"]["D"], s["case"]["G"], s["case"]["N"]
    per = D // G
    step = max(1, min(per, (512 * 16) // N))
    for g in range(G):
        for d0 in range(0, per, step):
            yield g, slice(g * per + d0, g * per + min(per, d0 + step))


def _block_inputs(s, sl):
    """delta and x of one channel block in chunk form, zero on rows past a sequence's end."""
    p = s["chunks"]
    raw = s["dt"][:, sl].float()
    if s["dt_bias"] is not None:
        raw = raw + s["dt_bias"][sl]
    real = p["real"][:, :, None]
    raw, x = raw[p["tok"]], s["x"][:, sl].float()[p["tok"]]
    return raw, _softplus(raw) * real, x * real, real


def _chain(s, H, total, A):
    """State before every chunk from the chunks' own end states and decays;
    the final state of every sequence."""
    n = len(s["lens"])
    hf = s["h0"].clone() if s["h0"] is not None else torch.zeros((n,) + H.shape[1:], device=H.device)
    hin = torch.empty_like(H)
    for chunk, seq, _, _ in s["chunks"]["walk"]:
        cur = hf[seq]
        hin[chunk] = cur
        hf[seq] = torch.exp(total[chunk][:, :, None] * A) * cur + H[chunk]
    return hin, hf


def _plain_scan_fwd(s):
    c, p = s["case"], s["chunks"]
    T, D, N = c["T"], c["D"], c["N"]
    A = -torch.exp(s["A_log"])
    dev = A.device
    H, total = torch.empty(p["nc"], D, N, device=dev), torch.empty(p["nc"], D, device=dev)
    for g, sl in _channel_blocks(s):
        _, delta, x, _ = _block_inputs(s, sl)
        u, B = delta * x, s["B"][:, g].float()[p["tok"]]
        h = torch.zeros(p["nc"], u.shape[2], N, device=dev)
        for i in range(CHUNK):
            h = torch.exp(delta[:, i, :, None] * A[sl]) * h + u[:, i, :, None] * B[:, i, None, :]
        H[:, sl], total[:, sl] = h, delta.sum(1)
    hin, hf = _chain(s, H, total, A)
    y = torch.empty(T, D, device=dev)
    for g, sl in _channel_blocks(s):
        _, delta, x, _ = _block_inputs(s, sl)
        u, B, C = delta * x, s["B"][:, g].float()[p["tok"]], s["C"][:, g].float()[p["tok"]]
        h = hin[:, sl]
        out = torch.empty_like(u)
        for i in range(CHUNK):
            h = torch.exp(delta[:, i, :, None] * A[sl]) * h + u[:, i, :, None] * B[:, i, None, :]
            out[:, i] = (h * C[:, i, None, :]).sum(2)
        blk = torch.empty(T, u.shape[2], device=dev)
        blk[p["tok"][p["real"]]] = out[p["real"]]
        if s["D"] is not None:
            blk += s["D"][sl] * s["x"][:, sl].float()
        if s["z"] is not None:
            z = s["z"][:, sl].float()
            blk *= z * torch.sigmoid(z)
        y[:, sl] = blk
    return dict(y=y.to(s["x"].dtype), h_final=hf)


def _plain_scan_train(s):
    c, p = s["case"], s["chunks"]
    T, D, N, G = c["T"], c["D"], c["N"], c["G"]
    dtype = s["x"].dtype
    A = -torch.exp(s["A_log"])
    dev = A.device
    tokr = p["tok"][p["real"]]

    def unchunk(v):
        r = torch.empty((T,) + v.shape[2:], device=dev)
        r[tokr] = v[p["real"]]
        return r

    def gate(sl):
        z = s["z"][:, sl].float()
        sg = torch.sigmoid(z)
        return z * sg, sg * (1.0 + z * (1.0 - sg))

    # 1: the chunks' own end states and decays, and the gradient that each
    # chunk's outputs send to the state before it
    H, Gs, total = (torch.empty(p["nc"], D, N, device=dev), torch.empty(p["nc"], D, N, device=dev),
                    torch.empty(p["nc"], D, device=dev))
    for g, sl in _channel_blocks(s):
        _, delta, x, real = _block_inputs(s, sl)
        dout = s["dy"][:, sl].float()
        if s["z"] is not None:
            dout = dout * gate(sl)[0]
        dout = dout[p["tok"]] * real
        u, B, C = delta * x, s["B"][:, g].float()[p["tok"]], s["C"][:, g].float()[p["tok"]]
        h = torch.zeros(p["nc"], u.shape[2], N, device=dev)
        acc, dec = torch.zeros_like(h), torch.ones_like(h)
        for i in range(CHUNK):
            a = torch.exp(delta[:, i, :, None] * A[sl])
            h = a * h + u[:, i, :, None] * B[:, i, None, :]
            dec = dec * a
            acc += dec * (dout[:, i, :, None] * C[:, i, None, :])
        H[:, sl], Gs[:, sl], total[:, sl] = h, acc, delta.sum(1)
    hin, hf = _chain(s, H, total, A)
    # the gradient after every chunk, from the sequences' ends
    dh0 = s["dh_final"].clone()
    dend = torch.empty_like(H)
    for chunk, seq, _, _ in reversed(p["walk"]):
        cur = dh0[seq]
        dend[chunk] = cur
        dh0[seq] = torch.exp(total[chunk][:, :, None] * A) * cur + Gs[chunk]
    del H, Gs

    # 2: outputs and gradients
    r = dict(y=torch.empty(T, D, device=dev), dx=torch.empty(T, D, device=dev), ddt=torch.empty(T, D, device=dev),
             dA_log=torch.empty(D, N, device=dev), dB=torch.zeros(T, G, N, device=dev),
             dC=torch.zeros(T, G, N, device=dev), ddt_bias=torch.empty(D, device=dev))
    r["dz"] = torch.empty(T, D, device=dev) if s["z"] is not None else None
    r["dD"] = torch.empty(D, device=dev) if s["D"] is not None else None
    for g, sl in _channel_blocks(s):
        raw, delta, x, real = _block_inputs(s, sl)
        xt, dy = s["x"][:, sl].float(), s["dy"][:, sl].float()
        sil, dsil = gate(sl) if s["z"] is not None else (None, None)
        dout = dy * sil if sil is not None else dy
        dout_c = dout[p["tok"]] * real
        u, B, C = delta * x, s["B"][:, g].float()[p["tok"]], s["C"][:, g].float()[p["tok"]]
        hs, out, h = [hin[:, sl]], torch.empty_like(u), hin[:, sl]
        for i in range(CHUNK):
            h = torch.exp(delta[:, i, :, None] * A[sl]) * h + u[:, i, :, None] * B[:, i, None, :]
            hs.append(h)
            out[:, i] = (h * C[:, i, None, :]).sum(2)
        dh = dend[:, sl].clone()
        dB, dC = torch.empty_like(B), torch.empty_like(C)
        du, ddelta, dA = torch.empty_like(u), torch.empty_like(u), torch.zeros(dh.shape[1:], device=dev)
        for i in reversed(range(CHUNK)):
            a = torch.exp(delta[:, i, :, None] * A[sl])
            dC[:, i] = (hs[i + 1] * dout_c[:, i, :, None]).sum(1)
            dh = dh + dout_c[:, i, :, None] * C[:, i, None, :]
            dB[:, i] = (dh * u[:, i, :, None]).sum(1)
            du[:, i] = (dh * B[:, i, None, :]).sum(2)
            dh = dh * a
            m = dh * hs[i]
            ddelta[:, i] = (m * A[sl]).sum(2)
            dA += (m * delta[:, i, :, None]).sum(0)
        ddelta = ddelta + du * x
        draw_ = ddelta * torch.where(raw > 20.0, torch.ones_like(raw), torch.sigmoid(raw)) * real
        y, dx = unchunk(out), unchunk(du * delta)
        if s["D"] is not None:
            y = y + s["D"][sl] * xt
            dx = dx + s["D"][sl] * dout
            r["dD"][sl] = (dout * xt).sum(0)
        if s["z"] is not None:
            r["dz"][:, sl] = dy * y * dsil
            y = y * sil
        r["y"][:, sl], r["dx"][:, sl], r["ddt"][:, sl] = y, dx, unchunk(draw_)
        r["ddt_bias"][sl] = draw_.sum((0, 1))
        r["dA_log"][sl] = dA * A[sl]
        r["dB"][:, g] += unchunk(dB)
        r["dC"][:, g] += unchunk(dC)
    if s["dt_bias"] is None:
        r["ddt_bias"] = None
    for k in ("y", "dx", "ddt", "dz", "dB", "dC"):
        r[k] = None if r[k] is None else r[k].to(dtype)
    out = dict(y=r["y"], h_final=hf, dh0=dh0, **{k: r[k] for k in _SCAN_GRADS if k != "dh0"})
    return {k: out[k] for k in ("y", "h_final") + _SCAN_GRADS}


def _plain_scan_step(s):
    D, G, T = s["case"]["D"], s["case"]["G"], s["case"]["T"]
    raw, x = s["dt"].float(), s["x"].float()
    if s["dt_bias"] is not None:
        raw = raw + s["dt_bias"]
    delta = _softplus(raw)
    A = -torch.exp(s["A_log"])
    per = lambda v: v.float().repeat_interleave(D // G, 1)
    h = torch.exp(delta[:, :, None] * A) * s["states"][s["src"].long()] + (delta * x)[:, :, None] * per(s["B"])
    y = (h * per(s["C"])).sum(2)
    if s["D"] is not None:
        y = y + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    s["states"][s["dst"].long()] = h
    return dict(y=y.to(s["x"].dtype), states=s["states"])


def _branch(s):
    """The post norm's output, the gate and their product with the scale, fp32."""
    o = s["o"].float()
    r1 = torch.rsqrt((o * o).mean(1, keepdim=True) + 1e-6)
    p = o * r1 * s["w_post"].float() if s["w_post"] is not None else o
    f = torch.ones_like(p) if s["gate"] is None else torch.sigmoid(s["gate"].float())
    return o, r1, p, f


def _plain_norm_fwd(s):
    _, _, p, f = _branch(s)
    b = p * f if s["scale"] is None else p * f * s["scale"]
    r = s["res"].float() + b
    y = r * torch.rsqrt((r * r).mean(1, keepdim=True) + 1e-6) * s["w_pre"].float()
    return dict(y=y.to(s["o"].dtype), res=r.to(s["res"].dtype))


def _plain_norm_bwd(s):
    o, r1, p, f = _branch(s)
    dy, r = s["dy"].float(), s["res"].float()
    r2 = torch.rsqrt((r * r).mean(1, keepdim=True) + 1e-6)
    rh = r * r2
    g = dy * s["w_pre"].float()
    dr = s["dres"].float() + r2 * (g - rh * (g * rh).mean(1, keepdim=True))
    sc = s["scale"] if s["scale"] is not None else 1.0
    dp = dr * f * sc
    out = dict(do=None, dres=dr.to(s["res"].dtype), dgate=None, dw_pre=(dy * rh).sum(0), dw_post=None, dscale=None)
    if s["gate"] is not None:
        out["dgate"] = (dr * sc * p * f * (1.0 - f)).to(s["o"].dtype)
    if s["scale"] is not None:
        out["dscale"] = (dr * f * p).sum(0)
    if s["w_post"] is not None:
        oh = o * r1
        out["dw_post"] = (dp * oh).sum(0)
        g = dp * s["w_post"].float()
        dp = r1 * (g - oh * (g * oh).mean(1, keepdim=True))
    out["do"] = dp.to(s["o"].dtype)
    return out


_PLAIN = dict(conv_fwd=_plain_conv_fwd, conv_bwd=_plain_conv_bwd, conv_step=_plain_conv_step,
              scan_fwd=_plain_scan_fwd, scan_train=_plain_scan_train, scan_step=_plain_scan_step,
              norm_fwd=_plain_norm_fwd, norm_bwd=_plain_norm_bwd)
_OWN = dict(conv_fwd=_own_conv_fwd, conv_bwd=_own_conv_bwd, conv_step=_own_conv_step, scan_fwd=_own_scan_fwd,
            scan_train=_own_scan_train, scan_step=_own_scan_step, norm_fwd=_own_norm_fwd, norm_bwd=_own_norm_bwd)


# ---------------------------------------------------------------------------
# the definition in 64 bits, sequence by sequence and token by token
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    k = case["kind"]
    if k.startswith("scan") and k != "scan_step" and (max(_lengths(case)) > 140000
                                                      or case["T"] * case["D"] * case["N"] > (1 << 33)):
        return None
    v = {n: (t.double() if isinstance(t, torch.Tensor) and t.is_floating_point() else t) for n, t in s.items()}
    return dict(conv_fwd=_exact_conv_fwd, conv_bwd=_exact_conv_bwd, conv_step=_exact_conv_step,
                scan_fwd=_exact_scan, scan_train=_exact_scan, scan_step=_exact_scan_step, norm_fwd=_exact_norm_fwd,
                norm_bwd=_exact_norm_bwd)[k](v)


def _exact_conv_seq(v, n):
    """Rows of sequence n after its history, and every row's window."""
    K, C = v["case"]["K"], v["case"]["C"]
    a, b = int(v["cu_host"][n]), int(v["cu_host"][n + 1])
    hist = v["state"][n] if v["state"] is not None else v["x"].new_zeros(K - 1, C)
    rows = torch.cat([hist, v["x"][a:b]])
    return a, b, rows


def _exact_conv_fwd(v):
    K = v["case"]["K"]
    y, st = torch.empty_like(v["x"]), []
    for n in range(len(v["lens"])):
        a, b, rows = _exact_conv_seq(v, n)
        st.append(rows[len(rows) - (K - 1):])
        if b > a:
            pre = torch.einsum("tck,ck->tc", rows.unfold(0, K, 1), v["w"])
            pre = pre + v["b"] if v["b"] is not None else pre
            y[a:b] = pre / (1.0 + torch.exp(-pre))
    return dict(y=y, state=torch.stack(st))


def _exact_conv_bwd(v):
    K, C = v["case"]["K"], v["case"]["C"]
    dx, dst = torch.empty_like(v["x"]), []
    dw, db = v["x"].new_zeros(C, K), v["x"].new_zeros(C)
    for n in range(len(v["lens"])):
        a, b, rows = _exact_conv_seq(v, n)
        dr = torch.zeros_like(rows)
        dr[len(rows) - (K - 1):] += v["dstate_out"][n]
        if b > a:
            win = rows.unfold(0, K, 1)
            pre = torch.einsum("tck,ck->tc", win, v["w"])
            pre = pre + v["b"] if v["b"] is not None else pre
            e = torch.exp(-pre)
            ds = v["dy"][a:b] * (1.0 + e + pre * e) / (1.0 + e) ** 2
            dw += torch.einsum("tc,tck->ck", ds, win)
            db += ds.sum(0)
            for j in range(K):
                dr[j:j + b - a] += ds * v["w"][:, j]
        dst.append(dr[:K - 1])
        dx[a:b] = dr[K - 1:]
    return dict(dx=dx, dw=dw, dbias=db, dstate=torch.stack(dst))


def _exact_conv_step(v):
    y, states = torch.empty_like(v["x"]), v["states"].clone()
    rows = torch.cat([v["states"].index_select(0, v["src"]), v["x"].unsqueeze(1)], 1)
    pre = torch.einsum("bkc,ck->bc", rows, v["w"])
    pre = pre + v["b"] if v["b"] is not None else pre
    y = pre / (1.0 + torch.exp(-pre))
    states.index_copy_(0, v["dst"].long(), rows[:, 1:])
    return dict(y=y, states=states)


def _exact_scan(v):
    c = v["case"]
    T, D, N, G = c["T"], c["D"], c["N"], c["G"]
    train = v["kind"] == "scan_train"
    x = v["x"]
    raw = v["dt"] + v["dt_bias"] if v["dt_bias"] is not None else v["dt"]
    delta = torch.where(raw > 20.0, raw, torch.log1p(torch.exp(raw.clamp(max=20.0))))
    A = -torch.exp(v["A_log"])
    u = delta * x
    wide = lambda q: q if G == 1 else q.repeat_interleave(D // G, -2)  # [.., G, N] -> [.., D or 1, N]
    order = sorted(range(len(v["lens"])), key=lambda n: -v["lens"][n])  # longest first
    start = v["cu"].long()[torch.tensor(order, device=x.device)]
    lens = [v["lens"][n] for n in order]
    pick = torch.tensor(order, device=x.device)
    h = v["h0"][pick].clone() if v["h0"] is not None else x.new_zeros(len(order), D, N)
    core = torch.empty_like(x)
    keep = []
    live = len(order)
    steps = lens[0] if lens else 0
    lives = []
    for i in range(steps):
        while lens[live - 1] <= i:
            live -= 1
        lives.append(live)
        t = start[:live] + i if live > 1 else slice(int(v["cu_host"][order[0]]) + i, int(v["cu_host"][order[0]]) + i + 1)
        if train:
            keep.append(h[:live].clone())
        cur = torch.exp(delta[t].unsqueeze(2) * A) * h[:live] + u[t].unsqueeze(2) * wide(v["B"][t])
        h[:live] = cur
        core[t] = (cur * wide(v["C"][t])).sum(2)
    hf = torch.empty_like(h)
    hf[pick] = h
    skip = core + v["D"] * x if v["D"] is not None else core
    sg = torch.sigmoid(v["z"]) if v["z"] is not None else None
    y = skip * v["z"] * sg if sg is not None else skip
    if not train:
        return dict(y=y, h_final=hf)
    dout = v["dy"] * v["z"] * sg if sg is not None else v["dy"]
    dz = v["dy"] * skip * sg * (1.0 + v["z"] * (1.0 - sg)) if sg is not None else None
    dB, dC = torch.empty_like(v["B"]), torch.empty_like(v["C"])
    du, dd, dA = torch.empty_like(x), torch.empty_like(x), torch.zeros_like(A)
    dh = v["dh_final"][pick].clone()
    group = lambda q: q.unflatten(1, (G, D // G)).sum(2)
    for i in range(steps - 1, -1, -1):
        live = lives[i]
        t = start[:live] + i
        a = torch.exp(delta[t].unsqueeze(2) * A)
        prev = keep[i]
        keep[i] = None
        Bt = wide(v["B"][t])
        cur = a * prev + u[t].unsqueeze(2) * Bt
        g = dout[t].unsqueeze(2)
        dC[t] = group(cur * g)
        q = dh[:live] + g * wide(v["C"][t])
        dB[t] = group(q * u[t].unsqueeze(2))
        du[t] = (q * Bt).sum(2)
        q = q * a
        m = q * prev
        dd[t] = (m * A).sum(2)
        dA += (m * delta[t].unsqueeze(2)).sum(0)
        dh[:live] = q
    dh0 = torch.empty_like(dh)
    dh0[pick] = dh
    ddt = (dd + du * x) * torch.where(raw > 20.0, torch.ones_like(raw), torch.sigmoid(raw))
    dx = du * delta + (v["D"] * dout if v["D"] is not None else 0.0)
    return dict(y=y, h_final=hf, dx=dx, ddt=ddt, dz=dz, dA_log=dA * A, dB=dB, dC=dC,
                dD=(dout * x).sum(0) if v["D"] is not None else None,
                ddt_bias=ddt.sum(0) if v["dt_bias"] is not None else None, dh0=dh0)


def _exact_scan_step(v):
    D, G = v["case"]["D"], v["case"]["G"]
    states = v["states"].clone()
    raw = v["dt"] + v["dt_bias"] if v["dt_bias"] is not None else v["dt"]
    delta = torch.logaddexp(raw, torch.zeros_like(raw))
    a = torch.exp(-delta.unsqueeze(2) * torch.exp(v["A_log"]))
    wide = lambda q: q.unsqueeze(2).expand(-1, -1, D // G, -1).flatten(1, 2)
    h = a * v["states"].index_select(0, v["src"]) + (delta * v["x"]).unsqueeze(2) * wide(v["B"])
    y = torch.einsum("bdn,bdn->bd", h, wide(v["C"]))
    y = y + v["D"] * v["x"] if v["D"] is not None else y
    y = y * v["z"] / (1.0 + torch.exp(-v["z"])) if v["z"] is not None else y
    states.index_copy_(0, v["dst"].long(), h)
    return dict(y=y, states=states)


def _exact_norm_fwd(v):
    norm = lambda q: q / torch.sqrt(q.square().mean(1, keepdim=True) + 1e-6)
    b = norm(v["o"]) * v["w_post"] if v["w_post"] is not None else v["o"]
    b = b / (1.0 + torch.exp(-v["gate"])) if v["gate"] is not None else b
    b = b * v["scale"] if v["scale"] is not None else b
    r = v["res"] + b
    return dict(y=norm(r) * v["w_pre"], res=r)


def _exact_norm_bwd(v):
    """By automatic differentiation of the forward's definition, the pre norm
    at the given residual stream."""
    norm = lambda q: q / torch.sqrt(q.square().mean(1, keepdim=True) + 1e-6)
    leaf = lambda n: None if v[n] is None else v[n].detach().requires_grad_()
    r, w_pre = leaf("res"), leaf("w_pre")
    dr, dw_pre = torch.autograd.grad(norm(r) * w_pre, (r, w_pre), v["dy"])
    dr = dr + v["dres"]
    o, w, gate, scale = leaf("o"), leaf("w_post"), leaf("gate"), leaf("scale")
    b = norm(o) * w if w is not None else o * 1.0
    b = b * torch.sigmoid(gate) if gate is not None else b
    b = b * scale if scale is not None else b
    have = [q for q in (o, w, gate, scale) if q is not None]
    gr = iter(torch.autograd.grad(b, have, dr))
    do, dw, dg, dsc = (next(gr) if q is not None else None for q in (o, w, gate, scale))
    return dict(do=do, dres=dr, dgate=dg, dw_pre=dw_pre, dw_post=dw, dscale=dsc)
