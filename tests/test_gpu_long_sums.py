"""Gradients that are sums over all tokens, of millions of them.  Inputs that do
not change from token to token make every term of a sum the same, and with them
the error of each addition: n terms added one by one are off by up to n / 2 half
steps (U) of the sum.  A block, strip or segment adds up to 1024 rows, and the
sum over the blocks' partial rows goes in eight chains whose ends are added.

Each tolerance is that count, in U relative to the sum of the terms' magnitudes,
and the terms' own error.  One wave of blocks, without a limit, would have 8192
rows each here, or 4096."""
import pytest
import torch

from tests import ssm_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
WAVE = 8192  # rows for each block of one wave


def counted(parts, term):
    """U that a sum over `parts` blocks of 1024 equal terms may be off by."""
    return 1024 / 2 + parts / 8 / 2 + 8 + term


@pytest.fixture(scope="module")
def g():
    from linear_attention_sequence_device_gb300 import build
    build.build_library()
    import linear_attention_sequence_device_gb300 as pkg
    pkg.load()
    return pkg


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def close(got, ref, mag, steps, what):
    worst = float(((got.double() - ref).abs() / (mag * R.U)).max())
    assert worst <= steps, f"{what}: {worst:.0f} steps, {steps} allowed"


def test_conv(g):
    from linear_attention_sequence_device_gb300 import binding
    C, K = 64, 2
    strips = lambda t: binding.load().gdn_ssm_conv_bwd_workspace_size(t, C, K) // (4 * C * (K + 1))
    T, q = WAVE * strips(1 << 15), gen(0)
    assert T <= 1024 * strips(T)
    u = lambda *s: torch.rand(*s, generator=q, device="cuda")
    x, w, dy = 0.2 + u(C), 0.2 + u(C, K), 0.5 + u(C)  # pre-activations of 0.1 to 3, where the SiLU's slope is 0.5 to 1.1
    row = lambda v: v.expand(T, C).contiguous()
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    r = g.gdn_ssm_conv_bwd(row(dy), row(x), w, torch.zeros(C, device="cuda"), cu, state=x.expand(1, K - 1, C).contiguous())
    x, w, dy = x.double(), w.double(), dy.double()
    pre = x * w.sum(1)
    s = torch.sigmoid(pre)
    ds = T * dy * s * (1 + pre * (1 - s))
    steps = counted(strips(T), 24)  # a term: 8 + 2 K |pre|, one more for dw
    close(r["dbias"], ds, ds.abs(), steps, "dbias")
    close(r["dw"], (ds * x)[:, None], (ds * x)[:, None], steps, "dw")


def test_block_norm(g):
    from linear_attention_sequence_device_gb300 import binding
    W = 1024
    blocks = lambda t: binding.load().gdn_block_norm_bwd_workspace_size(t, W) // (12 * W)
    T, q = WAVE // 4 * blocks(1 << 15), gen(1)  # of the three types' blocks; bf16's are half as many, with 4096 rows
    assert T <= 1024 * blocks(T)
    rn = lambda *s: torch.randn(*s, generator=q, device="cuda")
    dy, o, res = (rn(1, W).to(BF) for _ in range(3))
    w_pre, w_post, scale = (1 + 0.1 * rn(W)).to(BF), (1 + 0.1 * rn(W)).to(BF), 1 + 0.1 * rn(W)
    row = lambda v: v.expand(T, W).contiguous()
    r = g.gdn_block_norm_bwd(row(dy), None, row(o), row(res), w_pre, w_post=w_post, scale=scale)
    args = [None if t is None else R.d(t) for t in (dy, None, o, res, w_pre, w_post, None, scale)]
    ref, mag = R.norm_bwd(*args, 1e-6), R.norm_bwd(*args, 1e-6, absolute=True)
    for k in ("dw_pre", "dw_post", "dscale"):
        # a term: 40 for its factors, with roots of means that are summed as trees
        close(r[k].cpu(), T * ref[k], T * mag[k], counted(blocks(T), 40), k)


def test_scan(g):
    ch, N, short = 128, 4, 400
    bc = 4 * 2 * N  # the workspace's bytes a token; the rest is a row of 2 N + 3 a segment and channel
    segments = lambda t: (g.ssm_scan_bwd_workspace_size(t, ch, N, 1) - bc * t) // (4 * ch * (2 * N + 3))
    T, q = WAVE * segments(1 << 15), gen(2)
    assert T <= 1024 * segments(T)
    rn = lambda *s: torch.randn(*s, generator=q, device="cuda")
    u = lambda *s: torch.rand(*s, generator=q, device="cuda")
    x, dt, dy, B, C = 0.5 + u(ch), 0.5 + u(ch), 0.5 + u(ch), 0.5 + u(N), 0.5 + u(N)
    A_log = 0.3 * u(ch, N)  # decays of a step of 0.05 to 0.4: the state forgets in a few tokens
    def back(t):
        row = lambda v: v.expand(t, len(v)).contiguous()
        a = (row(x), row(dt), A_log, row(B).view(t, 1, N), row(C).view(t, 1, N))
        cu = torch.tensor([0, t], dtype=torch.int32, device="cuda")
        _, _, ck = g.gdn_ssm_scan_fwd(*a, cu, checkpoints=True)
        return g.gdn_ssm_scan_bwd(row(dy), *a, cu, ck)["dA_log"]
    got = back(T)

    def exact(t):
        row = lambda v: R.d(v).expand(t, len(v))
        return R.scan_grads(row(dy), None, row(x), row(dt), R.d(A_log), row(B).reshape(t, 1, N), row(C).reshape(t, 1, N),
                            torch.tensor([0, t]))["dA_log"]
    first = exact(short)
    ref = first + (T - short) * (exact(short + 1) - first)  # one more token in the middle is one more equal term
    # a term: two recurrences, each off by 16 half steps a token over a memory of 1 / (1 - 0.4) of them, and 20 more
    close(got.cpu(), ref, ref.abs(), counted(segments(T), 75), "dA_log")
