"""The selective scan layer's kernels against the 64-bit forms of ssm_ref.py:
lengths from zero to several segments, ragged and empty sequences, odd state
sizes, groups, strides, both types, carried states and the single-token forms.

Tolerances: half a step of the output's type, plus fp32 roundings counted per
operation times the magnitudes they apply to (ssm_ref.py)."""
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


def rows(T, C, dtype, q, pad=0, std=1.0):
    """A [T, C] device view with row stride C + pad."""
    t = (torch.randn(T, C + pad, generator=q) * std).to(dtype).cuda()
    return t[:, :C]


LENS = {"one": [1], "zero": [0], "zeros": [0, 0], "short": [5], "ragged": [0, 3, 0, 1, 70, 64, 0, 129, 2, 0],
        "long": [700], "edges": [64, 64, 128, 1, 63, 192]}


# ---- conv ----------------------------------------------------------------------

def conv_inputs(lens, C, K, dtype, state, bias, seed=0, pad=0):
    q = gen(seed)
    T, n = sum(lens), len(lens)
    x = rows(T, C, dtype, q, pad)
    w = (torch.randn(C, K, generator=q) * 0.5).to(dtype).cuda()
    b = (torch.randn(C, generator=q) * 0.1).to(dtype).cuda() if bias else None
    st = torch.randn(n, K - 1, C, generator=q).to(dtype).cuda() if state else None
    return x, w, b, cu_of(lens).cuda(), st


CONV = [("ragged", 64, 4, BF, True, True, 0), ("ragged", 24, 4, F32, True, False, 8), ("edges", 1032, 3, BF, False, True, 24),
        ("long", 64, 2, F32, True, True, 0), ("one", 8, 4, BF, True, True, 0), ("zero", 16, 4, BF, True, True, 0),
        ("zeros", 16, 3, F32, False, True, 0), ("short", 40, 1, BF, False, True, 0), ("long", 512, 4, BF, False, False, 0)]


@pytest.mark.parametrize("lens,C,K,dtype,state,bias,pad", CONV)
def test_conv_forward(g, lens, C, K, dtype, state, bias, pad):
    x, w, b, cu, st = conv_inputs(LENS[lens], C, K, dtype, state, bias, pad=pad)
    y, so = g.gdn_ssm_conv_fwd(x, w, b, cu, state=st)
    ry, rs, bound = R.conv_fwd(R.d(x), R.d(w), R.d(b), cu.cpu(), R.d(st))
    R.assert_within(y, ry, bound, "y")
    assert torch.equal(so.double().cpu(), rs)  # rows are moved, not computed


@pytest.mark.parametrize("lens,C,K,dtype,state,bias,pad", CONV)
def test_conv_backward(g, lens, C, K, dtype, state, bias, pad):
    x, w, b, cu, st = conv_inputs(LENS[lens], C, K, dtype, state, bias, seed=1, pad=pad)
    q = gen(2)
    dy = rows(x.shape[0], C, dtype, q, pad)
    dso = torch.randn(len(LENS[lens]), K - 1, C, generator=q).cuda() if state else None
    r = g.gdn_ssm_conv_bwd(dy, x, w, b, cu, state=st, dstate_out=dso)
    a = [R.d(v) for v in (dy, x, w, b)] + [cu.cpu(), R.d(st), R.d(dso)]
    ref, mag = R.conv_bwd(*a), R.conv_bwd(*a, absolute=True)
    # ds: the pre-activation's K + 1 roundings and 8 of the logistic function and the products, on factors whose
    # parts are in `mag`; then sums of K, or of T in any order
    pre = 1 + float(R.conv_pre(a[1], a[2], a[3], a[4], a[5], absolute=True)[0].abs().max()) if x.shape[0] else 1.0
    T = x.shape[0]
    for k in ("dx", "dstate"):
        R.assert_within(r[k], ref[k], (8 + 2 * K * pre) * R.U * mag[k], k)
    R.assert_within(r["dw"], ref["dw"], (8 + 2 * K * pre + T) * R.U * mag["dw"], "dw")
    if bias:
        R.assert_within(r["dbias"], ref["dbias"], (8 + 2 * K * pre + T) * R.U * mag["dbias"], "dbias")
    again = g.gdn_ssm_conv_bwd(dy, x, w, b, cu, state=st, dstate_out=dso)
    assert all(torch.equal(r[k], again[k]) for k in r if r[k] is not None)


def test_conv_in_pieces_and_steps_equals_the_whole(g):
    """A prompt fed in pieces of any length, then token by token, gives the whole prompt's outputs and state, bit for bit."""
    x, w, b, cu, _ = conv_inputs([97], 64, 4, BF, False, True)
    y, st = g.gdn_ssm_conv_fwd(x, w, b, cu)
    out, state, at = [], None, 0
    for n in (1, 2, 40, 3):
        o, state = g.gdn_ssm_conv_fwd(x[at:at + n], w, b, cu_of([n]).cuda(), state=state)
        out.append(o)
        at += n
    pool = torch.full((3, 3, 64), 7.0, dtype=BF, device="cuda")
    pool[2] = state[0]
    slot = torch.tensor([2], dtype=torch.int32, device="cuda")
    for t in range(at, 97):
        out.append(g.gdn_ssm_conv_step(x[t:t + 1], w, b, pool, src=slot, dst=slot))
    assert torch.equal(torch.cat(out), y) and torch.equal(pool[2:], st)
    assert bool((pool[:2] == 7).all())


@pytest.mark.parametrize("dtype,K,C", [(BF, 4, 1040), (F32, 3, 64), (BF, 1, 16), (F32, 2, 8)])
def test_conv_step(g, dtype, K, C):
    q = gen(4)
    x = rows(5, C, dtype, q, 8)
    w = torch.randn(C, K, generator=q).to(dtype).cuda()
    pool = torch.randn(9, K - 1, C, generator=q).to(dtype).cuda()
    # a fork, an update in place, a new request, a padded row, slot numbers out of range
    src = torch.tensor([0, 3, -1, 4, 99], dtype=torch.int32, device="cuda")
    dst = torch.tensor([8, 3, 5, -1, 6], dtype=torch.int32, device="cuda")
    old = pool.clone()
    y = g.gdn_ssm_conv_step(x, w, None, pool, src=src, dst=dst)
    st = torch.stack([R.d(old[0]), R.d(old[3]), torch.zeros(K - 1, C).double(), torch.zeros(K - 1, C).double(),
                      torch.zeros(K - 1, C).double()])
    ry, rs, bound = R.conv_fwd(R.d(x), R.d(w), None, torch.arange(6), st)
    ry[3], bound[3] = 0, 0
    R.assert_within(y, ry, bound, "y")
    exp = R.d(old)
    exp[8], exp[3], exp[5], exp[6] = rs[0], rs[1], rs[2], rs[4]
    assert torch.equal(R.d(pool), exp)


# ---- scan ------------------------------------------------------------------------

def scan_inputs(lens, ch, N, G, dtype, opts="Dzbh", seed=0, pad=0):
    q = gen(seed)
    T, n = sum(lens), len(lens)
    a = dict(x=rows(T, ch, dtype, q, pad), dt=rows(T, ch, dtype, q, pad, 0.5))
    bc = torch.randn(T, 3, G, N, generator=q).to(dtype).cuda()
    a["B"], a["C"] = bc[:, 0], bc[:, 2]
    a["A_log"] = (torch.log(torch.arange(1, N + 1.0)).expand(ch, N) + 0.1 * torch.randn(ch, N, generator=q)).cuda()
    d0 = torch.exp(torch.rand(ch, generator=q) * 4.6 - 6.9)
    a["dt_bias"] = (d0 + torch.log(-torch.expm1(-d0))).cuda() if "b" in opts else None
    a["D"] = torch.randn(ch, generator=q).cuda() if "D" in opts else None
    a["z"] = rows(T, ch, dtype, q, pad) if "z" in opts else None
    a["h0"] = torch.randn(n, ch, N, generator=q).cuda() if "h" in opts else None
    return a, cu_of(lens).cuda()


def fwd(g, a, cu, **kw):
    return g.gdn_ssm_scan_fwd(a["x"], a["dt"], a["A_log"], a["B"], a["C"], cu, D=a["D"], z=a["z"], dt_bias=a["dt_bias"],
                              h0=a["h0"], **kw)


def ref64(a, cu):
    v = {k: R.d(t) for k, t in a.items()}
    return v, (v["x"], v["dt"], v["A_log"], v["B"], v["C"], cu.cpu(), v["D"], v["z"], v["dt_bias"], v["h0"])


SCAN = [("ragged", 64, 16, 1, BF, "Dzbh", 0), ("ragged", 48, 16, 2, F32, "Dzbh", 8), ("edges", 72, 12, 1, F32, "Dzb", 0),
        ("long", 40, 16, 1, BF, "z", 16), ("long", 16, 4, 2, F32, "bh", 0), ("one", 8, 16, 1, BF, "Dzbh", 0),
        ("short", 32, 1, 1, F32, "Dzh", 0), ("zero", 16, 16, 1, BF, "Dzbh", 0), ("zeros", 8, 3, 1, F32, "Dz", 0),
        ("ragged", 32, 64, 2, F32, "Dzbh", 0), ("ragged", 40, 33, 1, BF, "Dbh", 0), ("edges", 136, 8, 1, BF, "Dzbh", 0),
        ("ragged", 200, 7, 1, F32, "zbh", 0), ("long", 24, 24, 3, F32, "Dzbh", 0), ("edges", 264, 2, 1, F32, "Dzbh", 0)]


@pytest.mark.parametrize("lens,ch,N,G,dtype,opts,pad", SCAN)
def test_scan_forward(g, lens, ch, N, G, dtype, opts, pad):
    a, cu = scan_inputs(LENS[lens], ch, N, G, dtype, opts, pad=pad)
    y, hf, ck = fwd(g, a, cu, checkpoints=True)
    v, args = ref64(a, cu)
    r = R.scan(*args)
    R.assert_within(hf, r["h_final"], r["h_bound"], "h_final")
    R.assert_within(y, r["y"], r["y_bound"], "y")
    starts = set(cu.tolist())
    for b in range(ck.shape[0]):  # the state before every 8th token, where that one goes on with a sequence
        if 8 * b not in starts:
            ref = r["before"][8 * b]
            R.assert_within(ck[b], ref, 64 * 16 * R.U * (1 + ref.abs().max()), f"checkpoint {b}")


@pytest.mark.parametrize("lens,ch,N,G,dtype,opts,pad", SCAN)
def test_scan_backward(g, lens, ch, N, G, dtype, opts, pad):
    a, cu = scan_inputs(LENS[lens], ch, N, G, dtype, opts, seed=3, pad=pad)
    _, _, ck = fwd(g, a, cu, checkpoints=True)
    q = gen(5)
    T, n = a["x"].shape[0], len(LENS[lens])
    dy = rows(T, ch, dtype, q, pad)
    dhf = torch.randn(n, ch, N, generator=q).cuda() if "h" in opts else None
    call = lambda: g.gdn_ssm_scan_bwd(dy, a["x"], a["dt"], a["A_log"], a["B"], a["C"], cu, ck, D=a["D"], z=a["z"],
                                      dt_bias=a["dt_bias"], h0=a["h0"], dh_final=dhf)
    r = call()
    v, args = ref64(a, cu)
    ref, mag = R.scan_grads(R.d(dy), R.d(dhf), *args), R.scan_grads(R.d(dy), R.d(dhf), *args, absolute=True)
    # every term is a product of a state, a gradient of a state and a few factors; the two recurrences each gather
    # 16 U a step over the sequence (ssm_ref.scan), the sums over n, channels or tokens one rounding a term, the
    # factors' own functions 16 U with arguments up to |z| = 5
    longest = max(LENS[lens])
    steps = 2 * 16 * longest + 32
    count = dict(dx=N, ddt=2 * N, dz=N, dA_log=T, dB=ch, dC=ch, dD=T, ddt_bias=T + 2 * N, dh0=0)
    for k, c in count.items():
        assert (r[k] is None) == (ref[k] is None), k
        if r[k] is not None:
            R.assert_within(r[k], ref[k], (steps + c) * R.U * mag[k], k)
    again = call()
    assert all(torch.equal(r[k], again[k]) for k in r if r[k] is not None)


def test_scan_norm_of_the_error_is_that_of_fp32(g):
    """The bounds above grow with the length; the error itself does not: in norm a few fp32 steps (a decay's
    relative error of 4 U a step over a memory of at most a thousand tokens, of random sign)."""
    a, cu = scan_inputs([2000], 32, 16, 1, F32, seed=6)
    y, hf, _ = fwd(g, a, cu)
    v, args = ref64(a, cu)
    r = R.scan(*args)
    for got, ref in ((y, r["y"]), (hf, r["h_final"])):
        assert float((R.d(got) - ref).norm() / ref.norm()) <= 4 * 1000 ** 0.5 * R.U


def test_scan_continued_and_stepped_equals_the_whole(g):
    """A prompt in two calls, then single tokens, against one call: the same recurrence, so within its bound twice."""
    a, cu = scan_inputs([150], 64, 16, 1, F32, "Dzbh", seed=7)
    y, hf, _ = fwd(g, a, cu)
    cut = lambda s, e, h0: {k: (t[s:e] if k in "xdtzBC" or k == "dt" else t) for k, t in a.items()} | {"h0": h0}
    y1, h1, _ = fwd(g, cut(0, 77, a["h0"]), cu_of([77]).cuda())
    y2, h2, _ = fwd(g, cut(77, 140, h1), cu_of([63]).cuda())
    out, pool = [y1, y2], h2.clone()
    for t in range(140, 150):
        out.append(g.gdn_ssm_scan_step(a["x"][t:t + 1], a["dt"][t:t + 1], a["A_log"], a["B"][t:t + 1], a["C"][t:t + 1],
                                       pool, D=a["D"], z=a["z"][t:t + 1], dt_bias=a["dt_bias"]))
    v, args = ref64(a, cu)
    r = R.scan(*args)
    R.assert_within(torch.cat(out), r["y"], r["y_bound"], "y in pieces")
    R.assert_within(pool, r["h_final"], r["h_bound"], "state in pieces")


@pytest.mark.parametrize("ch,N,G,dtype,opts", [(64, 16, 1, BF, "Dzb"), (48, 12, 2, F32, "Dzb"), (40, 5, 1, F32, "z"),
                                               (16, 64, 1, BF, "Db"), (264, 1, 1, F32, "Dzb"), (32, 8, 4, BF, "b")])
def test_scan_step(g, ch, N, G, dtype, opts):
    a, _ = scan_inputs([1] * 5, ch, N, G, dtype, opts, seed=8, pad=8)
    q = gen(9)
    pool = torch.randn(9, ch, N, generator=q).cuda()
    src = torch.tensor([0, 3, -1, 4, 99], dtype=torch.int32, device="cuda")
    dst = torch.tensor([8, 3, 5, -1, 6], dtype=torch.int32, device="cuda")
    old = pool.clone()
    y = g.gdn_ssm_scan_step(a["x"], a["dt"], a["A_log"], a["B"], a["C"], pool, D=a["D"], z=a["z"], dt_bias=a["dt_bias"],
                            src=src, dst=dst)
    st = torch.zeros(5, ch, N).double()
    st[0], st[1] = R.d(old[0]), R.d(old[3])
    v = {k: R.d(t) for k, t in a.items()}
    r = R.scan_step(v["x"], v["dt"], v["A_log"], v["B"], v["C"], st, v["D"], v["z"], v["dt_bias"])
    r["y"][3], r["y_bound"][3] = 0, 0
    R.assert_within(y, r["y"], r["y_bound"], "y")
    exp, bound = R.d(old), torch.zeros(9, ch, N).double()
    for i, s in ((0, 8), (1, 3), (2, 5), (4, 6)):
        exp[s], bound[s] = r["h_final"][i], r["h_bound"][i]
    R.assert_within(pool, exp, bound, "states")


def test_scan_sequences_do_not_leak(g):
    """Infinities and NaN of one sequence stay in it (its outputs, state and gradients), forward and backward."""
    lens = [40, 100, 30]
    a, cu = scan_inputs(lens, 64, 16, 1, F32, seed=10)
    a["x"][45, 3] = float("inf")
    a["h0"][1, 5] = float("nan")
    y, hf, ck = fwd(g, a, cu, checkpoints=True)
    clean = torch.ones(170, dtype=torch.bool)
    clean[40:140] = False
    assert torch.isfinite(y[clean.cuda()]).all() and torch.isfinite(hf[[0, 2]]).all()
    assert not torch.isfinite(hf[1, 5]).any() and not torch.isfinite(y[45:140, 3]).any()
    q = gen(11)
    r = g.gdn_ssm_scan_bwd(rows(170, 64, F32, q), a["x"], a["dt"], a["A_log"], a["B"], a["C"], cu, ck, D=a["D"],
                           z=a["z"], dt_bias=a["dt_bias"], h0=a["h0"])
    for k in ("dx", "ddt", "dz", "dB", "dC"):
        assert torch.isfinite(r[k][clean.cuda()]).all(), k
    assert torch.isfinite(r["dh0"][[0, 2]]).all()


def test_scan_extreme_steps(g):
    """delta from far below to above softplus's threshold: decays of 1 and of 0."""
    a, cu = scan_inputs([130], 32, 16, 1, F32, "Dzh", seed=12)
    a["dt"] = torch.linspace(-60, 60, 130).cuda()[:, None].expand(130, 32).contiguous()
    y, hf, ck = fwd(g, a, cu, checkpoints=True)
    v, args = ref64(a, cu)
    r = R.scan(*args)
    R.assert_within(y, r["y"], r["y_bound"], "y")
    R.assert_within(hf, r["h_final"], r["h_bound"], "h_final")


def test_scan_in_a_graph_on_another_stream(g):
    """Forward and backward captured on a side stream and replayed on new inputs give the eager bits."""
    a, cu = scan_inputs([300, 20], 64, 16, 1, BF, seed=13)
    b, _ = scan_inputs([300, 20], 64, 16, 1, BF, seed=14)
    dy = rows(320, 64, BF, gen(15))

    def both(a):
        y, hf, ck = fwd(g, a, cu, checkpoints=True)
        r = g.gdn_ssm_scan_bwd(dy, a["x"], a["dt"], a["A_log"], a["B"], a["C"], cu, ck, D=a["D"], z=a["z"],
                               dt_bias=a["dt_bias"], h0=a["h0"])
        return [y, hf] + [r[k] for k in sorted(r)]
    want = both(b)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        both(a)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(a)
    for k in a:
        if isinstance(a[k], torch.Tensor):
            a[k].copy_(b[k])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, w) for u, w in zip(got, want))


def test_wrong_arguments_raise(g):
    a, cu = scan_inputs([10], 64, 16, 1, BF)
    with pytest.raises(TypeError):
        fwd(g, a | {"dt": a["dt"].float()}, cu)
    with pytest.raises(ValueError):
        fwd(g, a | {"z": a["z"][:, :32]}, cu)
    with pytest.raises(ValueError):
        fwd(g, a | {"D": a["D"][:8]}, cu)
    with pytest.raises(ValueError):
        fwd(g, a | {"B": a["B"].transpose(1, 2).contiguous().transpose(1, 2).expand(10, 1, 16)[:, :, ::2]}, cu)
    with pytest.raises(ValueError):
        fwd(g, a, cu.cpu())
    with pytest.raises(g.GdnError):
        fwd(g, a, cu, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        g.gdn_ssm_conv_step(a["x"], torch.ones(64, 4, dtype=BF, device="cuda"), None,
                            torch.zeros(10, 2, 64, dtype=BF, device="cuda"))
