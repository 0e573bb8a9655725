"""No GPU: the 64-bit forms that the GPU tests compare against (their gradients
against automatic differentiation and against differences), and the refusals of
the selective scan layer's and the block norm's entry points."""
import ctypes

import pytest
import torch

from tests import ssm_ref as R

f64 = torch.float64


def rnd(*shape, seed=0, std=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=f64) * std


CU = torch.tensor([0, 0, 1, 6, 6, 11, 11])


def leaves(ts):
    return [t.clone().requires_grad_() for t in ts]


def check_grads(fn, inputs, got, weights):
    """got[i] against autograd of sum(weights * fn(inputs)) and against central differences along one direction."""
    ins = leaves(inputs)
    loss = lambda a: sum((w * o).sum() for w, o in zip(weights, fn(*a)))
    auto = torch.autograd.grad(loss(ins), ins)
    for g, a in zip(got, auto):
        assert torch.allclose(g, a, rtol=1e-10, atol=1e-11)
    for i, x in enumerate(inputs):
        v = rnd(*x.shape, seed=77 + i)
        at = lambda h: float(loss([q + h * v if j == i else q for j, q in enumerate(inputs)]).detach())
        num = (at(1e-5) - at(-1e-5)) / 2e-5
        assert abs(num - float((got[i] * v).sum())) <= 1e-6 * (1 + abs(num))


def test_conv_form_and_gradient():
    K, C, T, n = 4, 3, 11, len(CU) - 1
    x, w, b, st = rnd(T, C), rnd(C, K, seed=1), rnd(C, seed=2), rnd(n, K - 1, C, seed=3)
    y, out, _ = R.conv_fwd(x, w, b, CU, st)
    s, e = 1, 6  # a whole sequence by torch's convolution
    full = torch.cat([st[2], x[s:e]]).t()[None]
    pre = torch.nn.functional.conv1d(full, w[:, None], b, groups=C)[0].t()
    assert torch.allclose(y[s:e], torch.nn.functional.silu(pre))
    assert torch.equal(out[1], torch.cat([st[1], x[0:1]])[1:]) and torch.equal(out[3], st[3])
    dy, dso = rnd(T, C, seed=4), rnd(n, K - 1, C, seed=5)
    g = R.conv_bwd(dy, x, w, b, CU, st, dso)
    check_grads(lambda x, w, b, st: R.conv_fwd(x, w, b, CU, st)[:2], (x, w, b, st),
                (g["dx"], g["dw"], g["dbias"], g["dstate"]), (dy, dso))


def test_scan_form_and_gradient():
    T, ch, G, N, n = 11, 4, 2, 3, len(CU) - 1
    a = dict(x=rnd(T, ch), dt=rnd(T, ch, seed=1), A_log=rnd(ch, N, seed=2, std=0.5), B=rnd(T, G, N, seed=3),
             C=rnd(T, G, N, seed=4), D=rnd(ch, seed=5), z=rnd(T, ch, seed=6), dt_bias=rnd(ch, seed=7),
             h0=rnd(n, ch, N, seed=8))
    dy, dhf = rnd(T, ch, seed=9), rnd(n, ch, N, seed=10)
    g = R.scan_grads(dy, dhf, a["x"], a["dt"], a["A_log"], a["B"], a["C"], CU, a["D"], a["z"], a["dt_bias"], a["h0"])

    def fn(x, dt, A_log, B, C, D, z, dt_bias, h0):
        r = R.scan(x, dt, A_log, B, C, CU, D, z, dt_bias, h0)
        return r["y"], r["h_final"]
    check_grads(fn, list(a.values()), [g[k] for k in ("dx", "ddt", "dA_log", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")],
                (dy, dhf))


def test_norm_form_and_gradient():
    T, W = 3, 8
    o, r, wp, wq, ga, sc = rnd(T, W), rnd(T, W, seed=1), rnd(W, seed=2), rnd(W, seed=3), rnd(T, W, seed=4), rnd(W, seed=5)
    dy, dr = rnd(T, W, seed=6), rnd(T, W, seed=7)
    y, ro = R.norm_fwd(o, r, wp, wq, ga, sc, 1e-6)
    g = R.norm_bwd(dy, dr, o, ro, wp, wq, ga, sc, 1e-6)
    check_grads(lambda o, r, wp, wq, ga, sc: R.norm_fwd(o, r, wp, wq, ga, sc, 1e-6), (o, r, wp, wq, ga, sc),
                (g["do"], g["dres"], g["dw_pre"], g["dw_post"], g["dgate"], g["dscale"]), (dy, dr))


# ---- refusals -------------------------------------------------------------------

FAKE = ctypes.c_void_p(4096)       # never read: every call below fails on the host
ODD = ctypes.c_void_p(4096 + 4)


@pytest.fixture(scope="module")
def lib():
    from linear_attention_sequence_device_gb300 import build, binding
    build.build_library()
    return binding.load()


def test_conv_refusals(lib):
    def fwd(**kw):
        a = dict(x=FAKE, ldx=64, dt=1, T=8, C=64, w=FAKE, K=4, cu=FAKE, n=1, st=None, so=None, y=FAKE, ldy=64)
        a.update(kw)
        return lib.gdn_ssm_conv_fwd(a["x"], a["ldx"], a["dt"], a["T"], a["C"], a["w"], None, a["K"], a["cu"], a["n"],
                                    a["st"], a["so"], a["y"], a["ldy"], None)
    assert fwd(dt=5) == 3
    assert fwd(C=60) == 2 and fwd(K=5) == 2 and fwd(K=0) == 2
    assert fwd(T=-1) == 1 and fwd(n=0) == 1 and fwd(cu=None) == 1 and fwd(w=None) == 1
    assert fwd(ldx=56) == 1 and fwd(ldx=68) == 1 and fwd(x=ODD) == 1 and fwd(y=None) == 1
    assert fwd(st=ODD) == 1 and fwd(st=FAKE, so=FAKE) == 1

    need = lib.gdn_ssm_conv_bwd_workspace_size(256, 64, 4)
    assert need > 0 and need % 256 == 0
    assert lib.gdn_ssm_conv_bwd_workspace_size(256, 60, 4) == 0 and lib.gdn_ssm_conv_bwd_workspace_size(256, 64, 9) == 0

    def bwd(**kw):
        a = dict(dy=FAKE, lddy=64, dt=1, T=256, C=64, K=4, n=1, dx=FAKE, dw=FAKE, ws=FAKE, wb=need, st=None)
        a.update(kw)
        return lib.gdn_ssm_conv_bwd(a["dy"], a["lddy"], FAKE, 64, a["dt"], a["T"], a["C"], FAKE, None, a["K"], FAKE,
                                    a["n"], a["st"], None, a["dx"], 64, a["dw"], None, None, a["ws"], a["wb"], None)
    assert bwd(dt=2) == 3 and bwd(K=5) == 2 and bwd(n=0) == 1 and bwd(dw=None) == 1
    assert bwd(dy=ODD) == 1 and bwd(lddy=8) == 1 and bwd(dx=None) == 1 and bwd(st=ODD) == 1
    assert bwd(wb=need - 1) == 9 and bwd(ws=None) == 9 and bwd(ws=ctypes.c_void_p(4096 + 16)) == 9

    def step(**kw):
        a = dict(x=FAKE, B=4, C=64, K=4, states=FAKE, slots=4, src=None, dst=None, y=FAKE)
        a.update(kw)
        return lib.gdn_ssm_conv_step(a["x"], 64, 1, a["B"], a["C"], FAKE, None, a["K"], a["states"], a["slots"],
                                     a["src"], a["dst"], a["y"], 64, None)
    assert step(slots=3) == 1 and step(slots=3, src=FAKE) == 1 and step(slots=-1, src=FAKE, dst=FAKE) == 1
    assert step(B=65536, slots=70000) == 2 and step(C=4) == 2 and step(states=None) == 1 and step(y=ODD) == 1
    assert step(B=0) == 0  # nothing to do


def test_scan_refusals(lib):
    need = lib.gdn_ssm_scan_workspace_size(128, 64, 16, 2)
    assert need > 0 and need % 256 == 0
    assert lib.gdn_ssm_scan_ckpt_floats(65, 64, 16) == 9 * 64 * 16 and lib.gdn_ssm_scan_ckpt_floats(0, 64, 16) == 0
    for bad in ((128, 64, 65, 2), (128, 64, 0, 2), (128, 24, 16, 2), (128, 64, 16, 3), (-1, 64, 16, 2)):
        assert lib.gdn_ssm_scan_workspace_size(*bad) == 0 and lib.gdn_ssm_scan_bwd_workspace_size(*bad) == 0

    def fwd(**kw):
        a = dict(x=FAKE, ldx=64, z=None, ldz=0, B=FAKE, ldb=32, dt=1, A=FAKE, h0=None, cu=FAKE, n=1, T=128, ch=64, N=16,
                 G=2, y=FAKE, hf=None, ck=None, ws=FAKE, wb=need)
        a.update(kw)
        return lib.gdn_ssm_scan_fwd(a["x"], a["ldx"], FAKE, 64, a["z"], a["ldz"], a["B"], a["ldb"], FAKE, 32, a["dt"],
                                    a["A"], None, None, a["h0"], a["cu"], a["n"], a["T"], a["ch"], a["N"], a["G"],
                                    a["y"], 64, a["hf"], a["ck"], a["ws"], a["wb"], None)
    assert fwd(dt=2) == 3 and fwd(N=65) == 2 and fwd(N=0) == 2 and fwd(G=3) == 2 and fwd(ch=24) == 2
    assert fwd(T=-1) == 1 and fwd(n=0) == 1 and fwd(cu=None) == 1 and fwd(A=None) == 1 and fwd(B=None) == 1
    assert fwd(x=ODD) == 1 and fwd(ldx=60) == 1 and fwd(z=FAKE, ldz=32) == 1 and fwd(ldb=31) == 1 and fwd(y=None) == 1
    assert fwd(hf=ODD) == 1 and fwd(ck=ODD) == 1 and fwd(h0=FAKE, hf=FAKE) == 1
    assert fwd(wb=need - 1) == 9 and fwd(ws=None) == 9 and fwd(ws=ctypes.c_void_p(4096 + 64)) == 9

    bneed = lib.gdn_ssm_scan_bwd_workspace_size(128, 64, 16, 2)
    assert bneed > 0 and bneed % 256 == 0

    def bwd(**kw):
        a = dict(dy=FAKE, z=None, ldz=0, ck=FAKE, dhf=None, dx=FAKE, dz=None, dA=FAKE, dh0=None, N=16, ws=FAKE, wb=bneed)
        a.update(kw)
        return lib.gdn_ssm_scan_bwd(a["dy"], 64, FAKE, 64, FAKE, 64, a["z"], a["ldz"], FAKE, 32, FAKE, 32, 1, FAKE,
                                    None, None, None, a["ck"], a["dhf"], FAKE, 1, 128, 64, a["N"], 2, a["dx"], FAKE,
                                    a["dz"], FAKE, FAKE, a["dA"], None, None, a["dh0"], a["ws"], a["wb"], None)
    assert bwd(dy=None) == 1 and bwd(ck=None) == 1 and bwd(dx=None) == 1 and bwd(dx=ODD) == 1 and bwd(dA=None) == 1
    assert bwd(z=FAKE, ldz=64) == 1  # a gate without its gradient
    assert bwd(dhf=FAKE, dh0=FAKE) == 1 and bwd(N=99) == 2
    assert bwd(wb=bneed - 1) == 9 and bwd(ws=None) == 9

    def step(**kw):
        a = dict(B=4, N=16, states=FAKE, slots=4, src=None)
        a.update(kw)
        return lib.gdn_ssm_scan_step(FAKE, 64, FAKE, 64, None, 0, FAKE, 32, FAKE, 32, 1, FAKE, None, None, a["B"], 64,
                                     a["N"], 2, a["states"], a["slots"], a["src"], None, FAKE, 64, None)
    assert step(slots=3) == 1 and step(states=None) == 1 and step(states=ODD) == 1 and step(B=65536, slots=1 << 20) == 2
    assert step(N=65) == 2 and step(B=0) == 0


def test_norm_refusals(lib):
    def fwd(**kw):
        a = dict(o=FAKE, ldo=64, g=None, ldg=0, dt=1, res=FAKE, rdt=1, wq=None, wp=FAKE, eps=1e-6, T=4, W=64, ro=FAKE,
                 y=FAKE)
        a.update(kw)
        return lib.gdn_block_norm_fwd(a["o"], a["ldo"], a["g"], a["ldg"], a["dt"], a["res"], a["rdt"], a["wq"], a["wp"],
                                      None, a["eps"], a["T"], a["W"], a["ro"], a["y"], None)
    assert fwd(dt=3) == 3 and fwd(dt=0, rdt=1) == 3
    assert fwd(W=60, ldo=64) == 2 and fwd(W=16392, ldo=16392) == 2
    assert fwd(T=-1) == 1 and fwd(wp=None) == 1 and fwd(eps=-1.0) == 1 and fwd(o=None) == 1 and fwd(ldo=32) == 1
    assert fwd(g=FAKE, ldg=32) == 1 and fwd(res=ODD) == 1 and fwd(y=None) == 1 and fwd(wq=ODD) == 1
    assert fwd(T=0) == 0

    need = lib.gdn_block_norm_bwd_workspace_size(4, 64)
    assert need > 0 and need % 256 == 0 and lib.gdn_block_norm_bwd_workspace_size(4, 60) == 0

    def bwd(**kw):
        a = dict(dy=FAKE, g=None, wq=None, sc=None, do=FAKE, dwq=None, dsc=None, dwp=FAKE, ws=FAKE, wb=need)
        a.update(kw)
        return lib.gdn_block_norm_bwd(a["dy"], None, FAKE, 64, a["g"], 64, 1, FAKE, 1, a["wq"], FAKE, a["sc"], 1e-6, 4,
                                      64, a["do"], None, FAKE, a["dwp"], a["dwq"], a["dsc"], a["ws"], a["wb"], None)
    assert bwd(dy=None) == 1 and bwd(do=ODD) == 1 and bwd(dwp=None) == 1
    assert bwd(g=FAKE) == 1 and bwd(wq=FAKE) == 1 and bwd(sc=FAKE) == 1  # an input without its gradient
    assert bwd(wb=need - 1) == 9 and bwd(ws=None) == 9


@pytest.mark.parametrize("ch,N,G", [(8, 16, 1), (152, 12, 1), (1024, 16, 4), (1536, 5, 2), (4096, 16, 1), (8192, 64, 8)])
def test_workspace_sizes_do_not_fall(lib, ch, N, G):
    """A workspace for a long call serves every shorter one."""
    lens = sorted({int(1.17 ** i) + j for i in range(80) for j in (0, 1, 7)})
    for size in (lambda T: lib.gdn_ssm_scan_workspace_size(T, ch, N, G),
                 lambda T: lib.gdn_ssm_scan_bwd_workspace_size(T, ch, N, G),
                 lambda T: lib.gdn_ssm_conv_bwd_workspace_size(T, ch, 4),
                 lambda T: lib.gdn_block_norm_bwd_workspace_size(T, ch)):
        s = [size(T) for T in lens]
        assert all(a <= b for a, b in zip(s, s[1:])) and s[0] > 0
