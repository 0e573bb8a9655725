"""Parameters and states as slices of a flat buffer, four bytes behind a 16-byte
boundary: what the scan's forward takes its gradient and its single-token form
take too, with the same bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def g():
    from linear_attention_sequence_device_gb300 import build
    build.build_library()
    import linear_attention_sequence_device_gb300 as pkg
    pkg.load()
    return pkg


def shifted(t):
    flat = torch.zeros(t.numel() + 1, dtype=t.dtype, device=t.device)
    v = flat[1:].view(t.shape)
    v.copy_(t)
    assert v.is_contiguous() and v.data_ptr() % 16 == t.element_size()
    return v


def inputs(T, ch, N, dtype, seed):
    q = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=q).cuda()
    rows = dict(x=rn(T, ch).to(dtype), dt=rn(T, ch).to(dtype), B=rn(T, 1, N).to(dtype), C=rn(T, 1, N).to(dtype))
    par = dict(A_log=0.3 * rn(ch, N), D=rn(ch), dt_bias=rn(ch) - 3)
    return rows, par, rn


@pytest.mark.parametrize("T,ch,N,dtype", [(37, 24, 16, F32), (70, 40, 8, BF), (20, 16, 64, F32), (20, 16, 5, F32)])
def test_scan_and_gradient(g, T, ch, N, dtype):
    rows, par, rn = inputs(T, ch, N, dtype, 0)
    cu = torch.tensor([0, T // 3, T // 3, T], dtype=torch.int32, device="cuda")
    h0, dhf, dy = rn(3, ch, N), rn(3, ch, N), rn(T, ch).to(dtype)

    def both(f):
        p = {k: f(v) for k, v in par.items()}
        a = (rows["x"], rows["dt"], p["A_log"], rows["B"], rows["C"], cu)
        kw = dict(D=p["D"], dt_bias=p["dt_bias"], h0=f(h0))
        y, hf, ck = g.gdn_ssm_scan_fwd(*a, checkpoints=True, **kw)
        return dict(y=y, hf=hf, **g.gdn_ssm_scan_bwd(dy, *a, ck, dh_final=f(dhf), **kw))
    want, got = both(lambda t: t), both(shifted)
    assert all(torch.equal(want[k], got[k]) for k in want if want[k] is not None)


@pytest.mark.parametrize("ch,N,dtype", [(24, 16, F32), (40, 12, BF)])
def test_step(g, ch, N, dtype):
    rows, par, rn = inputs(3, ch, N, dtype, 1)
    pool = rn(3, ch, N)

    def step(f):
        p, st = {k: f(v) for k, v in par.items()}, pool.clone()
        return g.gdn_ssm_scan_step(rows["x"], rows["dt"], p["A_log"], rows["B"], rows["C"], st, D=p["D"],
                                   dt_bias=p["dt_bias"]), st
    for want, got in zip(step(lambda t: t), step(shifted)):
        assert torch.equal(want, got)
