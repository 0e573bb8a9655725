"""Elements beyond 2^31: the last sequence of a long packed batch and the last
slots of a large cache, against the 64-bit forms (ssm_ref.py) or against the same
rows alone.  What lies before is zero, so that it costs no time to make."""
import pytest
import torch

from tests import ssm_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
C, TAIL = 4096, 45
T = 2 ** 31 // C + 208 + TAIL
SL = slice(0, C, 128)  # channels whose results are checked in 64 bits


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


def far(q, dtype=BF, width=C):
    """[T, width], zero but for the last TAIL rows."""
    t = torch.zeros(T, width, dtype=dtype, device="cuda")
    t[-TAIL:] = torch.randn(TAIL, width, generator=q).to(dtype).cuda()
    return t


def gen(seed):
    return torch.Generator().manual_seed(seed)


def cu():
    return torch.tensor([0, T - TAIL, T], dtype=torch.int32, device="cuda")


def test_conv(g):
    q = gen(0)
    x, dy = far(q), far(q)
    w, b = torch.randn(C, 4, generator=q).to(BF).cuda(), torch.randn(C, generator=q).to(BF).cuda()
    one = torch.tensor([0, TAIL], dtype=torch.int32, device="cuda")
    y, st = g.gdn_ssm_conv_fwd(x, w, b, cu())
    y1, st1 = g.gdn_ssm_conv_fwd(x[-TAIL:], w, b, one)
    assert torch.equal(y[-TAIL:], y1) and torch.equal(st[1], st1[0])
    r = g.gdn_ssm_conv_bwd(dy, x, w, b, cu())
    r1 = g.gdn_ssm_conv_bwd(dy[-TAIL:], x[-TAIL:], w, b, one)
    assert torch.equal(r["dx"][-TAIL:], r1["dx"]) and torch.equal(r["dstate"][1], r1["dstate"][0])


def test_scan(g):
    q = gen(1)
    N = 16
    x, dt, z, dy = far(q), far(q), far(q), far(q)
    B, Cm = far(q, width=N).view(T, 1, N), far(q, width=N).view(T, 1, N)
    A_log = torch.log(torch.arange(1, N + 1.0)).expand(C, N).contiguous().cuda()
    D = torch.randn(C, generator=q).cuda()
    y, hf, ck = g.gdn_ssm_scan_fwd(x, dt, A_log, B, Cm, cu(), D=D, z=z, checkpoints=True)
    r = g.gdn_ssm_scan_bwd(dy, x, dt, A_log, B, Cm, cu(), ck, D=D, z=z)
    tail = lambda t: R.d(t[-TAIL:])
    v = (tail(x)[:, SL], tail(dt)[:, SL], R.d(A_log)[SL], tail(B), tail(Cm), torch.tensor([0, TAIL]), R.d(D)[SL],
         tail(z)[:, SL])
    ref = R.scan(*v)
    R.assert_within(y[-TAIL:, SL], ref["y"], ref["y_bound"], "y")
    R.assert_within(hf[1:, SL], ref["h_final"], ref["h_bound"], "h_final")
    gy = tail(dy)[:, SL]
    gr, mag = R.scan_grads(gy, None, *v), R.scan_grads(gy, None, *v, absolute=True)
    for k, c in dict(dx=N, ddt=2 * N, dz=N, dh0=0).items():  # counted as in the short sequences' test
        got = r[k][1:, SL] if k == "dh0" else r[k][-TAIL:, SL]
        R.assert_within(got, gr[k], (2 * 16 * TAIL + 32 + c) * R.U * mag[k], k)


def test_steps(g):
    q = gen(2)
    N, slots = 16, 2 ** 31 // (C * 16) + 9
    row = lambda *s: torch.randn(*s, generator=q).to(BF).cuda()
    x, dt, B, Cm = row(1, C), row(1, C), row(1, 1, N), row(1, 1, N)
    A_log = torch.log(torch.arange(1, N + 1.0)).expand(C, N).contiguous().cuda()
    last = torch.tensor([slots - 1], dtype=torch.int32, device="cuda")
    pool = torch.zeros(slots, C, N, device="cuda")
    pool[-1] = torch.randn(C, N, generator=q).cuda()
    own = pool[-1:].clone()
    y = g.gdn_ssm_scan_step(x, dt, A_log, B, Cm, pool, src=last, dst=last)
    assert torch.equal(y, g.gdn_ssm_scan_step(x, dt, A_log, B, Cm, own)) and torch.equal(pool[-1:], own)
    assert not pool[:9].any()
    del pool
    slots = 2 ** 31 // (3 * C) + 9
    last = torch.tensor([slots - 1], dtype=torch.int32, device="cuda")
    w = row(C, 4)
    pool = torch.zeros(slots, 3, C, dtype=BF, device="cuda")
    pool[-1] = row(3, C)
    own = pool[-1:].clone()
    y = g.gdn_ssm_conv_step(x, w, None, pool, src=last, dst=last)
    assert torch.equal(y, g.gdn_ssm_conv_step(x, w, None, own)) and torch.equal(pool[-1:], own)
    assert not pool[:9].any()


def test_block_norm(g):
    q = gen(3)
    o, res, gate, dy = far(q), far(q), far(q), far(q)
    w = (1 + 0.1 * torch.randn(C, generator=q)).to(BF).cuda()
    y, r = g.gdn_block_norm_fwd(o, res, w, w_post=w, gate=gate)
    d = g.gdn_block_norm_bwd(dy, None, o, res, w, w_post=w, gate=gate)
    tail = lambda t: t[-TAIL:].contiguous()
    # bf16 results: within a step of those of the rows alone, whose sums another kernel may take in another order
    y1, r1 = g.gdn_block_norm_fwd(tail(o), tail(res), w, w_post=w, gate=tail(gate))
    d1 = g.gdn_block_norm_bwd(tail(dy), None, tail(o), tail(res), w, w_post=w, gate=tail(gate))
    for got, ref in ((y, y1), (r, r1), (d["do"], d1["do"]), (d["dres"], d1["dres"]), (d["dgate"], d1["dgate"])):
        R.assert_within(got[-TAIL:], R.d(ref), 2.0 ** -8 * R.d(ref).abs() + 1e-6, "rows")
