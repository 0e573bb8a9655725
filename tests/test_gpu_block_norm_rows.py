"""The block norm and its gradient with more rows than blocks, so that a block
goes from row to row (the gradient's column sums among them), at the widths
between which the vectors a thread and the ring of rows change, against the
64-bit forms of ssm_ref.py (run on the GPU).

Tolerances: those of test_gpu_block_norm.py, counted there, with the gate's
magnitude taken from the inputs."""
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


def inputs(T, W, dtype, res, opts, seed):
    q = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=q, device="cuda")
    a = dict(o=rn(T, W).to(dtype), res=(2 * rn(T, W)).to(res), w_pre=(1 + 0.1 * rn(W)).to(dtype),
             w_post=(1 + 0.1 * rn(W)).to(dtype) if "p" in opts else None, gate=rn(T, W).to(dtype) if "g" in opts else None,
             scale=0.1 + 0.02 * rn(W) if "s" in opts else None)
    return a, rn(T, W).to(dtype), rn(T, W).to(res)


def wide(t):
    return None if t is None else t.double()


def within(got, ref, bound, what):
    R.assert_within(got, ref.cpu(), bound.cpu(), what)


FORWARD = [(10000, 64, BF, BF, "pgs"), (10000, 64, F32, F32, "pg"), (10000, 264, BF, F32, "pgs"), (10000, 264, F32, F32, "gs"),
           (5000, 1032, BF, BF, "pgs"), (5000, 1032, F32, F32, "pgs"), (2500, 4096, BF, F32, "pgs"), (2500, 4096, F32, F32, "pgs"),
           (2500, 4096, BF, BF, ""), (1100, 8200, BF, BF, "ps"), (700, 16384, F32, F32, "pgs")]


@pytest.mark.parametrize("T,W,dtype,res,opts", FORWARD)
def test_forward(g, T, W, dtype, res, opts):
    # a thread takes 32 columns at most, an SM 2048 threads and 32 blocks
    assert T > torch.cuda.get_device_properties(0).multi_processor_count * min(32, 65536 // W)
    a, _, _ = inputs(T, W, dtype, res, opts, 0)
    y, r = g.gdn_block_norm_fwd(a["o"], a["res"], a["w_pre"], w_post=a["w_post"], gate=a["gate"], scale=a["scale"])
    v = {k: wide(t) for k, t in a.items()}
    with torch.device("cuda"):
        ry, rr = R.norm_fwd(v["o"], v["res"], v["w_pre"], v["w_post"], v["gate"], v["scale"], 1e-6)
    amp = float(a["gate"].abs().max()) if a["gate"] is not None else 0.0
    bound = (W / 2 + 16 + 2 * amp) * R.U * (v["res"].abs() + (rr - v["res"]).abs())
    within(r, rr, bound, "res_out")
    scale = v["w_pre"].abs() / torch.sqrt(rr.square().mean(1, keepdim=True) + 1e-6)
    within(y, ry, bound * scale + (W / 2 + 8) * R.U * ry.abs(), "y")


BACKWARD = [(7301, 64, BF, BF, "pgs"), (7301, 64, F32, F32, "pgs"), (7301, 264, F32, F32, "pgs"), (7301, 264, BF, F32, "gs"),
            (2000, 2048, BF, F32, "gs"), (1000, 4096, BF, BF, "pgs"), (1000, 4096, BF, F32, "pgs"), (1000, 4096, F32, F32, "ps"),
            (500, 4608, F32, F32, "pgs"), (500, 5632, BF, F32, "pgs"), (500, 8192, BF, F32, "pgs"), (500, 8192, BF, BF, "p"),
            (500, 8968, BF, BF, "pgs"), (500, 12296, BF, F32, "pgs"), (500, 16384, BF, BF, "g"), (500, 16384, F32, F32, "pgs")]


@pytest.mark.parametrize("T,W,dtype,res,opts", BACKWARD)
def test_backward(g, T, W, dtype, res, opts):
    from linear_attention_sequence_device_gb300 import binding
    blocks = binding.load().gdn_block_norm_bwd_workspace_size(T, W) // (12 * W)
    assert T >= 3 * blocks
    a, dy, dres = inputs(T, W, dtype, res, opts, 1)
    kw = dict(w_post=a["w_post"], gate=a["gate"], scale=a["scale"])
    v = {k: wide(t) for k, t in a.items()}
    for dr in (dres, None):
        r = g.gdn_block_norm_bwd(dy, dr, a["o"], a["res"], a["w_pre"], **kw)
        args = (wide(dy), wide(dr), v["o"], v["res"], v["w_pre"], v["w_post"], v["gate"], v["scale"], 1e-6)
        with torch.device("cuda"):
            ref, mag = R.norm_bwd(*args), R.norm_bwd(*args, absolute=True)
        for k in ref:
            assert (r[k] is None) == (ref[k] is None), k
            if ref[k] is not None:
                c = 3 * W + 48 + (T if k in ("dw_pre", "dw_post", "dscale") else 0)
                within(r[k], ref[k], c * R.U * mag[k], k)
        again = g.gdn_block_norm_bwd(dy, dr, a["o"], a["res"], a["w_pre"], **kw)
        assert all(torch.equal(r[k], again[k]) for k in r if r[k] is not None)
