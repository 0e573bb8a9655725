"""The gated delta rule's single tokens against the 64-bit form of lm_ref.py: head
sizes, groups, both types, new, padded and out-of-range slots, few heads and as many
as go through the ring, strides, far slots, capture, refusals.  Bounds: lm_ref.py."""
import pytest
import torch

from tests import lm_ref as L
from tests import ssm_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def g():
    from linear_attention_sequence_device_gb300 import build
    build.build_library()
    import linear_attention_sequence_device_gb300 as pkg
    pkg.load()
    yield pkg
    assert pkg.binding.device_timeouts() == 0


def inputs(B, Hk, Hv, dk, dv, dtype, seed=0, slots=None, pad=0):
    q = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=q, device="cuda")
    rows = lambda n: rn(B, n + pad).to(dtype)[:, :n]
    return dict(x=rows(2 * Hk * dk + Hv * dv), a=rows(Hv), b=rows(Hv), z=rows(Hv * dv).unflatten(1, (Hv, dv)),
                A_log=torch.rand(Hv, generator=q, device="cuda"), dt_bias=rn(Hv), norm_w=(1 + 0.1 * rn(dv)).to(dtype),
                states=0.3 * rn(2 * B if slots is None else slots, Hv, dk, dv))


def parts(i, Hk, Hv, dk, dv):
    q, k, v = i["x"].split([Hk * dk, Hk * dk, Hv * dv], 1)
    return q.unflatten(1, (Hk, dk)), k.unflatten(1, (Hk, dk)), v.unflatten(1, (Hv, dv))


def start(states, src):
    """States that the requests start from: zeros for a slot outside the cache."""
    n = len(states)
    ok = (src >= 0) & (src < n)
    return torch.where(ok[:, None, None, None], L.dbl(states)[src.long().clamp(0, n - 1)], 0.0)


def check(got, ref, bound, states, old, src, dst, new, bS, what):
    live = (dst >= 0) & (dst < len(old))
    z = torch.zeros_like(ref[:1])
    ref, bound = torch.where(live[:, None, None], ref, z), torch.where(live[:, None, None], bound, z)
    R.assert_within(got, ref.cpu(), bound.cpu(), what)
    exp, b = L.dbl(old), torch.zeros_like(L.dbl(old))
    exp[dst[live].long()], b[dst[live].long()] = new[live], bS[live]
    R.assert_within(states, exp.cpu(), b.cpu(), what + " states")


SHAPES = [(5, 1, 1, 32, 32, BF), (5, 2, 4, 32, 128, F32), (5, 2, 2, 64, 64, BF), (6, 1, 4, 64, 32, F32), (5, 2, 4, 128, 128, BF),
          (7, 1, 2, 128, 64, F32), (5, 1, 3, 64, 128, BF), (9, 2, 2, 128, 32, BF),
          # states of 28 MB and more: the ring
          (16, 16, 32, 128, 128, BF), (16, 16, 32, 128, 128, F32), (33, 8, 32, 64, 128, BF), (70, 16, 32, 64, 64, F32),
          (241, 4, 32, 32, 32, BF), (60, 16, 32, 128, 32, BF), (120, 8, 32, 32, 64, F32), (33, 16, 32, 128, 64, F32)]


def slot_numbers(B, n, seed):
    """Forks, updates in place, new requests, padded rows and numbers behind the cache."""
    perm = torch.randperm(n, generator=torch.Generator().manual_seed(seed))[:2 * B].to(torch.int32)
    src, dst = perm[:B].clone(), perm[B:].clone()
    dst[::3] = src[::3]
    src[1::5] = -1
    src[2::7] = n + 3
    dst[3::6] = -1
    dst[4::11] = n
    return src.cuda(), dst.cuda()


@pytest.mark.parametrize("B,Hk,Hv,dk,dv,dtype", SHAPES)
def test_rule(g, B, Hk, Hv, dk, dv, dtype):
    i = inputs(B, Hk, Hv, dk, dv, dtype, pad=3)
    q, k, v = parts(i, Hk, Hv, dk, dv)
    gate, beta = L.gates(*(i[n].float() for n in ("a", "b", "A_log", "dt_bias")))
    beta = beta.to(dtype)
    src, dst = slot_numbers(B, 2 * B, 1)
    for l2, scale in ((True, None), (False, 0.1)):
        old, st = i["states"], i["states"].clone()
        o = g.gdn_chunk_step(q, k, v, gate, beta, st, src=src, dst=dst, scale=scale, l2norm=l2)
        ref = L.rule_step(L.dbl(q), L.dbl(k), L.dbl(v), L.dbl(gate), L.dbl(beta), start(old, src),
                          dk ** -0.5 if scale is None else scale, l2)
        check(o, ref[0], ref[1], st, old, src, dst, ref[2], ref[3], f"rule {l2}")


@pytest.mark.parametrize("B,Hk,Hv,dk,dv,dtype", SHAPES)
def test_layer(g, B, Hk, Hv, dk, dv, dtype):
    i = inputs(B, Hk, Hv, dk, dv, dtype, seed=2, pad=5)
    src, dst = slot_numbers(B, 2 * B, 3)
    v = {n: L.dbl(t) for n, t in i.items()}
    gate, beta = L.gates(v["a"], v["b"], v["A_log"], v["dt_bias"])
    for norm in (True, False):
        old, st = i["states"], i["states"].clone()
        y = g.gdn_layer_step(i["x"], i["a"], i["b"], i["A_log"], i["dt_bias"], i["z"] if norm else None, i["norm_w"], st,
                             Hk, Hv, dk, dv, src=src, dst=dst)
        ref = L.rule_step(*parts(v, Hk, Hv, dk, dv), gate, beta, start(old, src), dk ** -0.5, True,
                          v["z"] if norm else None, v["norm_w"])
        check(y, ref[0], ref[1], st, old, src, dst, ref[2], ref[3], f"layer {norm}")


def test_steps_are_the_chunk_kernels_tokens(g):
    """Tokens one by one give the prompt's outputs and state, to the chunk kernel's bar in fp32."""
    Hk, Hv, dk, dv, n = 2, 4, 32, 32, 70
    i = inputs(n, Hk, Hv, dk, dv, F32, seed=4, slots=1)
    q, k, v = parts(i, Hk, Hv, dk, dv)
    gate, beta = L.gates(i["a"], i["b"], i["A_log"], i["dt_bias"])
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    o, S = g.gdn_chunk_fwd(q.contiguous(), k.contiguous(), v.contiguous(), gate, beta, cu, h0=i["states"], l2norm=True)
    st = i["states"].clone()
    one = torch.cat([g.gdn_chunk_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], gate[t:t + 1], beta[t:t + 1], st, l2norm=True)
                     for t in range(n)])
    assert float((one - o).norm()) <= 1e-4 * float(o.norm()) and float((st - S).norm()) <= 1e-4 * float(S.norm())


@pytest.mark.parametrize("B", [3, 20])
def test_all_rows_padded(g, B):
    i = inputs(B, 8, 32, 128, 128, BF, seed=5)
    st = i["states"].clone()
    none = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    out = torch.full((B, 32, 128), 7.0, dtype=BF, device="cuda")
    y = g.gdn_layer_step(i["x"], i["a"], i["b"], i["A_log"], i["dt_bias"], i["z"], i["norm_w"], st, 8, 32, 128, 128,
                         src=none, dst=none, out=out)
    assert y is out and not out.any() and torch.equal(st, i["states"])


@pytest.mark.parametrize("B", [4, 40])
def test_requests_do_not_leak(g, B):
    """NaN and infinities of one request, and of the slots that none reads, stay where they are; a padded row's inputs are not read."""
    Hk, Hv, d = 4, 8, 128
    if B == 40:
        Hk = Hv = 32  # the ring
    i = inputs(B, Hk, Hv, d, d, F32, seed=6)
    src = torch.arange(B, dtype=torch.int32, device="cuda")
    dst = src.clone()
    dst[2] = -1
    st = i["states"].clone()
    call = lambda s: g.gdn_layer_step(i["x"], i["a"], i["b"], i["A_log"], i["dt_bias"], i["z"], i["norm_w"], s, Hk, Hv, d, d,
                                      src=src, dst=dst)
    clean = call(clean_st := st.clone())
    st[1, 0, 3, 5] = float("nan")
    st[B:] = float("inf")
    i["x"][2] = float("nan")
    y = call(st)
    keep = [b for b in range(B) if b != 1]
    assert torch.equal(y[keep], clean[keep]) and torch.equal(y[1, 1:], clean[1, 1:])
    assert torch.equal(st[[b for b in keep if b != 2]], clean_st[[b for b in keep if b != 2]])
    assert torch.isnan(y[1, 0]).all() and torch.isinf(st[B:]).all()


def test_far_slots(g):
    """Slots beyond 2^31 elements, by blocks of their own and through the ring."""
    Hk = Hv = 32
    n = 2 ** 31 // (Hv * 128 * 128) + 40
    st = torch.empty(n, Hv, 128, 128, device="cuda")
    for B in (2, 16):
        i = inputs(B, Hk, Hv, 128, 128, BF, seed=7, slots=2 * B)
        st[-2 * B:] = i["states"]
        near = i["states"].clone()
        a = (i["x"], i["a"], i["b"], i["A_log"], i["dt_bias"], i["z"], i["norm_w"])
        src, dst = torch.arange(B, dtype=torch.int32, device="cuda"), torch.arange(B, 2 * B, dtype=torch.int32, device="cuda")
        y = g.gdn_layer_step(*a, near, Hk, Hv, 128, 128, src=src, dst=dst)
        far = g.gdn_layer_step(*a, st, Hk, Hv, 128, 128, src=src + n - 2 * B, dst=dst + n - 2 * B)
        assert torch.equal(y, far) and torch.equal(st[-2 * B:], near)
    del st
    torch.cuda.empty_cache()


@pytest.mark.parametrize("B", [3, 20])
def test_captured_on_another_stream(g, B):
    i, j = inputs(B, 8, 32, 128, 128, BF, seed=8), inputs(B, 8, 32, 128, 128, BF, seed=9)
    out = torch.empty(B, 32, 128, dtype=BF, device="cuda")

    def step(i, st):
        return g.gdn_layer_step(i["x"], i["a"], i["b"], i["A_log"], i["dt_bias"], i["z"], i["norm_w"], st, 8, 32, 128, 128,
                                out=out)
    want_st = j["states"].clone()
    want = step(j, want_st).clone()
    st = i["states"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(i, st.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(i, st)
    for n in i:
        i[n].copy_(j[n])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(st, want_st)


def test_no_requests(g):
    i = inputs(1, 1, 2, 32, 32, F32)
    y = g.gdn_layer_step(i["x"][:0], i["a"][:0], i["b"][:0], i["A_log"], i["dt_bias"], i["z"][:0], i["norm_w"], i["states"],
                         1, 2, 32, 32)
    assert y.shape == (0, 2, 32)


def test_wrong_arguments_raise(g):
    i = inputs(4, 1, 2, 32, 32, F32)
    q, k, v = parts(i, 1, 2, 32, 32)
    gate, beta = L.gates(i["a"], i["b"], i["A_log"], i["dt_bias"])
    ok = dict(q=q, k=k, v=v, g=gate, beta=beta, states=i["states"])
    call = lambda **kw: g.gdn_chunk_step(**(ok | kw))
    call()
    with pytest.raises(TypeError):
        call(g=gate.double())
    with pytest.raises(TypeError):
        call(k=k.to(BF))
    with pytest.raises(ValueError):
        call(k=k[:3])
    with pytest.raises(ValueError):
        call(states=i["states"].transpose(2, 3))
    with pytest.raises(TypeError):
        call(src=torch.zeros(4, dtype=torch.int64, device="cuda"), dst=torch.zeros(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(g.GdnError):  # fewer slots than requests
        call(states=i["states"][:3])
    with pytest.raises(g.GdnError):  # head size
        g.gdn_chunk_step(q[..., :16], k[..., :16], v, gate, beta, i["states"][:, :, :16].contiguous())
    with pytest.raises(g.GdnError):  # a norm without its weights
        g.gdn_layer_step(i["x"], i["a"], i["b"], i["A_log"], i["dt_bias"], i["z"], None, i["states"], 1, 2, 32, 32)
    with pytest.raises(ValueError):
        g.gdn_layer_step(i["x"][:, :-1], i["a"], i["b"], i["A_log"], i["dt_bias"], i["z"], i["norm_w"], i["states"], 1, 2, 32, 32)
