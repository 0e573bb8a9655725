"""The selective scan layer's kernels where their loops go round: segments of
several tiles, strips of many batches of rows, requests that follow one another
in a block, against the 64-bit forms of ssm_ref.py (run on the GPU).

Few tokens are cut down to one tile or batch a block, so the sizes here are taken
from how calls are cut: wide channels, which leave few segments, many rows, and
more requests than the grid has blocks.  Each test first asserts that its case is
one of these, by the workspace's size (one piece a segment or strip) or by the
blocks that can be resident on the GPU.

Tolerances: those of test_gpu_ssm.py, counted there, and for the scan what its
decays add where a step is large (see large_steps)."""
import pytest
import torch

from tests import ssm_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def g():
    from linear_attention_sequence_device_gb300 import build
    build.build_library()
    import linear_attention_sequence_device_gb300 as pkg
    pkg.load()
    return pkg


def gen(seed):
    return torch.Generator().manual_seed(seed)


def cu_of(lens):
    return torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32)


def rnd(q, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=q) * std).to(dtype).cuda()


def wide(t):
    """In 64 bits, where it lies."""
    return None if t is None else t.double()


def within(got, ref, bound, what):
    R.assert_within(got, ref.cpu(), bound.cpu() if isinstance(bound, torch.Tensor) else bound, what)


def blocks_at_once():
    """More blocks of 128 threads than a launch of these kernels has in one wave: four an SM."""
    return 4 * torch.cuda.get_device_properties(0).multi_processor_count


# ---- scan -----------------------------------------------------------------------

LONG = [0, 200, 0, 3, 500, 1, 130, 64, 0, 325]  # ends in the middle of tiles and of segments, two spans of several


def scan_inputs(lens, ch, N, G, dtype, opts="Dzbh", seed=0):
    q = gen(seed)
    T, n = sum(lens), len(lens)
    a = dict(x=rnd(q, T, ch, dtype=dtype), dt=rnd(q, T, ch, dtype=dtype, std=0.5))
    bc = rnd(q, T, 2, G, N, dtype=dtype)
    a["B"], a["C"] = bc[:, 0], bc[:, 1]
    a["A_log"] = (torch.log(torch.arange(1, N + 1.0)).expand(ch, N) + 0.1 * torch.randn(ch, N, generator=q)).cuda()
    d0 = torch.exp(torch.rand(ch, generator=q) * 4.6 - 6.9)
    a["dt_bias"] = (d0 + torch.log(-torch.expm1(-d0))).cuda() if "b" in opts else None
    a["D"] = rnd(q, ch) if "D" in opts else None
    a["z"] = rnd(q, T, ch, dtype=dtype) if "z" in opts else None
    a["h0"] = rnd(q, n, ch, N) if "h" in opts else None
    return a, cu_of(lens).cuda()


def call(g, a, cu, **kw):
    return g.gdn_ssm_scan_fwd(a["x"], a["dt"], a["A_log"], a["B"], a["C"], cu, D=a["D"], z=a["z"], dt_bias=a["dt_bias"],
                              h0=a["h0"], **kw)


def args64(a, cu):
    v = {k: wide(t) for k, t in a.items()}
    return v["x"], v["dt"], v["A_log"], v["B"], v["C"], cu.cpu(), v["D"], v["z"], v["dt_bias"], v["h0"]


def large_steps(x, dt, A_log, B, C, cu, D, z, dt_bias, h0):
    """What the bounds of ssm_ref.scan leave out, for y and the final states.  A decay e^-v is off by 10 U v of
    itself from delta's and A's own errors; 16 U of the terms' magnitudes cover that for v of order one, but with 64
    states v reaches 40 (there fp32 functions that round correctly pass 16 U too)."""
    v = (R.softplus(dt + (dt_bias if dt_bias is not None else 0.0)))[:, :, None] * torch.exp(A_log)
    ub = (v / torch.exp(A_log) * x[:, :, None]).abs() * R._wide(B, x.shape[1]).abs()
    a, Cw = torch.exp(-v), R._wide(C, x.shape[1]).abs()
    ey, eh = torch.zeros_like(x), []
    for n, (s, e) in enumerate(R.seqs(cu)):
        mag = h0[n].abs() if h0 is not None else x.new_zeros(A_log.shape)
        er = torch.zeros_like(mag)
        for t in range(s, e):
            er = a[t] * (er + 10 * R.U * v[t] * mag)
            mag = a[t] * mag + ub[t]
            ey[t] = (er * Cw[t]).sum(1)
        eh.append(er)
    return ey * ((z * torch.sigmoid(z)).abs() if z is not None else 1.0), torch.stack(eh)


# wide: segments of several tiles of 16 tokens; the last ones two to four segments, folded without a launch of their own
SCAN = [(LONG, 4096, 16, 1, BF, "Dzbh"), (LONG, 4064, 16, 4, F32, "Dzbh"), (LONG, 4096, 8, 2, F32, "zbh"),
        (LONG, 4096, 4, 1, BF, "Dzb"), (LONG, 2048, 32, 1, F32, "Dzbh"), (LONG, 1024, 64, 2, BF, "Dbh"),
        (LONG, 1024, 64, 1, F32, "Dzbh"), (LONG, 4096, 13, 1, F32, "Dzbh"), (LONG, 2048, 24, 2, BF, "Dzbh"),
        ([50], 64, 16, 1, F32, "Dzbh"), ([30, 0, 20], 200, 8, 1, F32, "Dzbh"), ([17], 40, 32, 1, BF, "Dzbh"),
        ([64], 64, 64, 1, F32, "zbh"), ([3, 45], 96, 5, 2, BF, "Dzbh")]


@pytest.mark.parametrize("lens,ch,N,G,dtype,opts", SCAN)
def test_scan_forward(g, lens, ch, N, G, dtype, opts):
    T = sum(lens)
    segments = g.ssm_scan_workspace_size(T, ch, N, G) // (4 * ch * (N + 1))
    assert T >= 48 * segments if lens is LONG else 2 <= segments <= 4
    a, cu = scan_inputs(lens, ch, N, G, dtype, opts)
    y, hf, ck = call(g, a, cu, checkpoints=True)
    with torch.device("cuda"):
        r = R.scan(*args64(a, cu))
        ey, eh = large_steps(*args64(a, cu))
    within(hf, r["h_final"], r["h_bound"] + eh, "h_final")
    within(y, r["y"], r["y_bound"] + ey, "y")
    at = [b for b in range(ck.shape[0]) if 8 * b not in set(cu.tolist())]
    ref = torch.stack([r["before"][8 * b] for b in at])
    # 16 U a step, at most over the longest sequence
    within(ck[at], ref, max(lens) * 16 * R.U * (1 + ref.abs().amax((1, 2), keepdim=True)), "checkpoints")


@pytest.mark.parametrize("lens,ch,N,G,dtype,opts", SCAN)
def test_scan_backward(g, lens, ch, N, G, dtype, opts):
    T, n = sum(lens), len(lens)
    if lens is LONG:  # what the workspace has beside the tokens' share: a row of 2 N + 3 a segment and channel
        size = lambda t: g.ssm_scan_bwd_workspace_size(t, ch, N, G)
        assert T >= 32 * ((2 * size(T) - size(2 * T)) // (4 * ch * (2 * N + 3)))
    a, cu = scan_inputs(lens, ch, N, G, dtype, opts, seed=3)
    _, _, ck = call(g, a, cu, checkpoints=True)
    q = gen(5)
    dy = rnd(q, T, ch, dtype=dtype)
    dhf = rnd(q, n, ch, N) if "h" in opts else None
    back = lambda: g.gdn_ssm_scan_bwd(dy, a["x"], a["dt"], a["A_log"], a["B"], a["C"], cu, ck, D=a["D"], z=a["z"],
                                      dt_bias=a["dt_bias"], h0=a["h0"], dh_final=dhf)
    r = back()
    with torch.device("cuda"):
        ref = R.scan_grads(wide(dy), wide(dhf), *args64(a, cu))
        mag = R.scan_grads(wide(dy), wide(dhf), *args64(a, cu), absolute=True)
    steps = 2 * 16 * max(lens) + 32
    count = dict(dx=N, ddt=2 * N, dz=N, dA_log=T, dB=ch, dC=ch, dD=T, ddt_bias=T + 2 * N, dh0=0)
    for k, c in count.items():
        assert (r[k] is None) == (ref[k] is None), k
        if r[k] is not None:
            within(r[k], ref[k], (steps + c) * R.U * mag[k], k)
    again = back()
    assert all(torch.equal(r[k], again[k]) for k in r if r[k] is not None)


def slots(batch, q):
    """A cache of 3 batch slots: forks, updates in place, new requests, padded rows and slot numbers out of range."""
    perm = torch.randperm(3 * batch, generator=q).to(torch.int32)
    src, dst = perm[:batch].clone(), perm[batch:2 * batch].clone()
    src[::5] = dst[::5]
    src[3::11] = -1
    src[7::13] = 3 * batch + 4
    dst[2::17] = -1
    dst[5::19] = 3 * batch
    return src.cuda(), dst.cuda()


STEP = [(130, 4096, 16, 1, BF, "Dzb"), (130, 4096, 16, 2, F32, "Dzb"), (130, 4072, 16, 1, BF, "Dzb"),
        (130, 4096, 12, 1, F32, "Db"), (130, 4056, 13, 1, BF, "zb"), (900, 64, 16, 1, F32, "Dzb"), (110, 512, 11, 1, BF, "Dz"),
        (130, 4096, 8, 1, BF, "Dzb"), (130, 4072, 7, 1, F32, "Dzb"), (130, 4096, 4, 1, F32, "zb"),
        (130, 2048, 32, 1, BF, "Dzb"), (130, 2040, 24, 1, F32, "Dzb"), (130, 1024, 64, 2, F32, "Dzb"),
        (130, 1016, 50, 1, BF, "Dzb"), (2000, 8, 11, 1, F32, "Dzb"), (1200, 16, 13, 2, BF, "zb")]


@pytest.mark.parametrize("batch,ch,N,G,dtype,opts", STEP)
def test_scan_step(g, batch, ch, N, G, dtype, opts):
    # blocks side by side cover 32 to 128 channels of one request
    assert batch * G * ((ch // G + 127) // 128) > 2 * blocks_at_once() or batch * ((ch + 31) // 32) > 2 * blocks_at_once()
    a, _ = scan_inputs([1] * batch, ch, N, G, dtype, opts, seed=8)
    q = gen(9)
    pool = rnd(q, 3 * batch, ch, N)
    src, dst = slots(batch, q)
    old = pool.clone()
    y = g.gdn_ssm_scan_step(a["x"], a["dt"], a["A_log"], a["B"], a["C"], pool, D=a["D"], z=a["z"], dt_bias=a["dt_bias"],
                            src=src, dst=dst)
    have = (src >= 0) & (src < 3 * batch)
    st = wide(old)[src.clamp(0, 3 * batch - 1).long()] * have[:, None, None]
    v = {k: wide(t) for k, t in a.items()}
    with torch.device("cuda"):
        r = R.scan_step(v["x"], v["dt"], v["A_log"], v["B"], v["C"], st, v["D"], v["z"], v["dt_bias"])
        ey, eh = large_steps(v["x"], v["dt"], v["A_log"], v["B"], v["C"], torch.arange(batch + 1), v["D"], v["z"],
                             v["dt_bias"], st)
    keep = (dst >= 0) & (dst < 3 * batch)
    assert not y[~keep].any()
    within(y[keep], r["y"][keep], (r["y_bound"] + ey)[keep], "y")
    exp, bound = wide(old), torch.zeros_like(wide(old))
    exp[dst[keep].long()], bound[dst[keep].long()] = r["h_final"][keep], (r["h_bound"] + eh)[keep]
    untouched = torch.ones(3 * batch, dtype=torch.bool, device="cuda").index_fill_(0, dst[keep].long(), False)
    assert torch.equal(pool[untouched], old[untouched])
    within(pool, exp, bound, "states")


# ---- conv -----------------------------------------------------------------------

def conv_inputs(lens, C, K, dtype, state, bias, seed):
    q = gen(seed)
    T, n = sum(lens), len(lens)
    return (rnd(q, T, C, dtype=dtype), rnd(q, C, K, dtype=dtype, std=0.5), rnd(q, C, dtype=dtype, std=0.1) if bias else None,
            cu_of(lens).cuda(), rnd(q, n, K - 1, C, dtype=dtype) if state else None), q


def cuts(T, n, seed):
    """n lengths that sum to T, empty ones among them."""
    c = torch.randint(0, T + 1, (n - 1,), generator=gen(seed)).sort().values.tolist()
    return [b - a for a, b in zip([0] + c, c + [T])]


CONV = [(24500, 40, 64, 4, BF, True, True), (24501, 3, 64, 3, F32, False, True), (12300, 60, 1032, 4, F32, True, False),
        (6203, 9, 2056, 2, BF, True, True), (3100, 12, 4096, 4, BF, True, True), (3099, 7, 4096, 4, F32, True, True)]


@pytest.mark.parametrize("T,n,C,K,dtype,state,bias", CONV)
def test_conv_forward(g, T, n, C, K, dtype, state, bias):
    assert T * ((C + 1023) // 1024) > 5 * 4 * blocks_at_once()  # strips of more than five batches of four rows
    (x, w, b, cu, st), _ = conv_inputs(cuts(T, n, 1), C, K, dtype, state, bias, 2)
    y, so = g.gdn_ssm_conv_fwd(x, w, b, cu, state=st)
    ry, rs, bound = R.conv_fwd(R.d(x), R.d(w), R.d(b), cu.cpu(), R.d(st))
    R.assert_within(y, ry, bound, "y")
    assert torch.equal(so.double().cpu(), rs)


@pytest.mark.parametrize("T,n,C,K,dtype,state,bias", CONV)
def test_conv_backward(g, T, n, C, K, dtype, state, bias):
    from linear_attention_sequence_device_gb300 import binding
    strips = binding.load().gdn_ssm_conv_bwd_workspace_size(T, C, K) // (4 * C * (K + 1))
    assert T >= 5 * 4 * strips  # more than five batches of four rows
    (x, w, b, cu, st), q = conv_inputs(cuts(T, n, 3), C, K, dtype, state, bias, 4)
    dy = rnd(q, T, C, dtype=dtype)
    dso = rnd(q, n, K - 1, C) if state else None
    r = g.gdn_ssm_conv_bwd(dy, x, w, b, cu, state=st, dstate_out=dso)
    a = [R.d(v) for v in (dy, x, w, b)] + [cu.cpu(), R.d(st), R.d(dso)]
    ref, mag = R.conv_bwd(*a), R.conv_bwd(*a, absolute=True)
    pre = 1 + float(R.conv_pre(a[1], a[2], a[3], a[4], a[5], absolute=True)[0].abs().max())
    for k in ("dx", "dstate"):
        R.assert_within(r[k], ref[k], (8 + 2 * K * pre) * R.U * mag[k], k)
    for k in ("dw", "dbias") if bias else ("dw",):
        R.assert_within(r[k], ref[k], (8 + 2 * K * pre + T) * R.U * mag[k], k)
    again = g.gdn_ssm_conv_bwd(dy, x, w, b, cu, state=st, dstate_out=dso)
    assert all(torch.equal(r[k], again[k]) for k in r if r[k] is not None)


@pytest.mark.parametrize("batch,C,K,dtype", [(300, 8192, 4, BF), (250, 8192, 4, F32), (330, 6152, 3, BF), (2000, 64, 4, F32),
                                             (2000, 1032, 2, BF), (700, 4096, 1, F32)])
def test_conv_step(g, batch, C, K, dtype):
    assert batch * ((C + 1023) // 1024) > 2 * blocks_at_once()
    q = gen(4)
    x, w, b = rnd(q, batch, C, dtype=dtype), rnd(q, C, K, dtype=dtype), rnd(q, C, dtype=dtype)
    pool = rnd(q, 3 * batch, K - 1, C, dtype=dtype)
    src, dst = slots(batch, q)
    old = pool.clone()
    y = g.gdn_ssm_conv_step(x, w, b, pool, src=src, dst=dst)
    have, keep = (src >= 0) & (src < 3 * batch), (dst >= 0) & (dst < 3 * batch)
    st = wide(old)[src.clamp(0, 3 * batch - 1).long()] * have[:, None, None]
    ry, rs, bound = R.conv_fwd(R.d(x), R.d(w), R.d(b), torch.arange(batch + 1), st.cpu())
    keep, exp = keep.cpu(), R.d(old)
    assert not y.cpu()[~keep].any()
    R.assert_within(y.cpu()[keep], ry[keep], bound[keep], "y")
    exp[dst.cpu()[keep].long()] = rs[keep]
    assert torch.equal(R.d(pool), exp)
