"""The block norm (post norm, gate, residual scale, residual add, pre norm) and
its gradient against the 64-bit forms of ssm_ref.py.

Tolerances: half a step of each output's type plus counted fp32 roundings: a
mean over W values W + 4 (halved by the root), every factor one, the logistic
function 8 + 2 |gate|, on the magnitudes of the terms."""
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


def inputs(T, W, dtype, res, opts, seed=0, pad=0):
    q = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=q)
    a = dict(o=rn(T, W + pad).to(dtype).cuda()[:, :W], res=(2 * rn(T, W)).to(res).cuda(),
             w_pre=(1 + 0.1 * rn(W)).to(dtype).cuda(),
             w_post=(1 + 0.1 * rn(W)).to(dtype).cuda() if "p" in opts else None,
             gate=rn(T, W + pad).to(dtype).cuda()[:, :W] if "g" in opts else None,
             scale=(0.1 + 0.02 * rn(W)).cuda() if "s" in opts else None)
    return a, rn(T, W).to(dtype).cuda(), rn(T, W).to(res).cuda()


CASES = [(5, 64, BF, BF, "pgs", 0), (3, 8, F32, F32, "pgs", 8), (17, 4096, BF, F32, "pgs", 0), (4, 1032, BF, BF, "p", 24),
         (1, 2048, F32, F32, "gs", 0), (2, 8200, BF, F32, "pgs", 0), (3, 16384, F32, F32, "ps", 0), (700, 136, BF, BF, "", 0),
         (33, 512, F32, F32, "g", 16), (0, 64, BF, F32, "pgs", 0)]


@pytest.mark.parametrize("T,W,dtype,res,opts,pad", CASES)
def test_forward(g, T, W, dtype, res, opts, pad):
    a, _, _ = inputs(T, W, dtype, res, opts, pad=pad)
    y, r = g.gdn_block_norm_fwd(a["o"], a["res"], a["w_pre"], w_post=a["w_post"], gate=a["gate"], scale=a["scale"])
    v = {k: R.d(t) for k, t in a.items()}
    ry, rr = R.norm_fwd(v["o"], v["res"], v["w_pre"], v["w_post"], v["gate"], v["scale"], 1e-6)
    amp = 5.0  # |gate| of these draws
    bound = (W / 2 + 16 + 2 * amp) * R.U * (v["res"].abs() + (rr - v["res"]).abs())
    R.assert_within(r, rr, bound, "res_out")
    scale = (v["w_pre"].abs() / torch.sqrt(rr.square().mean(1, keepdim=True) + 1e-6)) if T else 0.0
    R.assert_within(y, ry, bound * scale + (W / 2 + 8) * R.U * ry.abs(), "y")


@pytest.mark.parametrize("T,W,dtype,res,opts,pad", CASES)
def test_backward(g, T, W, dtype, res, opts, pad):
    a, dy, dres = inputs(T, W, dtype, res, opts, seed=1, pad=pad)
    kw = dict(w_post=a["w_post"], gate=a["gate"], scale=a["scale"])
    v = {k: R.d(t) for k, t in a.items()}
    for dr in (dres, None):
        r = g.gdn_block_norm_bwd(dy, dr, a["o"], a["res"], a["w_pre"], **kw)
        args = (R.d(dy), R.d(dr), v["o"], v["res"], v["w_pre"], v["w_post"], v["gate"], v["scale"], 1e-6)
        ref, mag = R.norm_bwd(*args), R.norm_bwd(*args, absolute=True)
        # two means of W products each on top of the rms
        for k in ref:
            assert (r[k] is None) == (ref[k] is None), k
            if ref[k] is not None:
                c = 3 * W + 48 + (T if k in ("dw_pre", "dw_post", "dscale") else 0)
                R.assert_within(r[k], ref[k], c * R.U * mag[k], k)
        again = g.gdn_block_norm_bwd(dy, dr, a["o"], a["res"], a["w_pre"], **kw)
        assert all(torch.equal(r[k], again[k]) for k in r if r[k] is not None)


def test_in_place_residual(g):
    a, dy, dres = inputs(9, 256, BF, F32, "pgs", seed=2)
    kw = dict(w_post=a["w_post"], gate=a["gate"], scale=a["scale"])
    y, r = g.gdn_block_norm_fwd(a["o"], a["res"], a["w_pre"], **kw)
    y2, r2 = g.gdn_block_norm_fwd(a["o"], a["res"], a["w_pre"], res_out=a["res"], **kw)
    assert r2 is a["res"] and torch.equal(r, r2) and torch.equal(y, y2)


def test_zero_rows_and_nan_stay_in_their_row(g):
    a, _, _ = inputs(6, 64, F32, F32, "p", seed=3)
    a["o"][1] = 0
    a["res"][1] = 0
    a["o"][3, 7] = float("nan")
    y, r = g.gdn_block_norm_fwd(a["o"], a["res"], a["w_pre"], w_post=a["w_post"])
    assert bool((y[1] == 0).all()) and bool((r[1] == 0).all())
    assert torch.isfinite(y[[0, 1, 2, 4, 5]]).all() and not torch.isfinite(y[3]).any()


def test_wrong_arguments_raise(g):
    a, dy, dres = inputs(4, 64, BF, BF, "pgs")
    with pytest.raises(TypeError):
        g.gdn_block_norm_fwd(a["o"], a["res"].to(torch.float16), a["w_pre"])
    with pytest.raises(ValueError):
        g.gdn_block_norm_fwd(a["o"], a["res"], a["w_pre"][:32])
    with pytest.raises(ValueError):
        g.gdn_block_norm_fwd(a["o"], a["res"].t().contiguous().t(), a["w_pre"])
    with pytest.raises(TypeError):
        g.gdn_block_norm_bwd(dy, dres.float(), a["o"], a["res"], a["w_pre"])
