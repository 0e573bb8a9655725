"""The vocabulary's loss and its gradients against the 64-bit form of lm_ref.py: both
types, sizes from one to several tiles and pieces, odd widths, strides, tokens left
out, targets behind the vocabulary, scales, wide ranges in fp32, capture, refusals.
Bounds: lm_ref.py."""
import pytest
import torch

from tests import lm_ref as L
from tests import ssm_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
I32, I64 = torch.int32, torch.int64


@pytest.fixture(scope="module")
def g():
    from linear_attention_sequence_device_gb300 import build
    build.build_library()
    import linear_attention_sequence_device_gb300 as pkg
    pkg.load()
    yield pkg
    assert pkg.binding.device_timeouts() == 0


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def view(T, W, dtype, q, pad=0, skip=0, std=1.0):
    flat = (torch.randn(T * (W + pad) + skip, generator=q, device="cuda") * std).to(dtype)
    return flat[skip:].view(T, W + pad)[:, :W]


def inputs(T, V, W, dtype, seed=0, pad=0, skip=0, index=I64, know=6.0, out=0.15):
    """Hidden states that know their target more or less well; some tokens left out."""
    q = gen(seed)
    w = view(V, W, dtype, q, pad, skip, W ** -0.5)
    t = torch.randint(0, V, (T,), generator=q, device="cuda")
    h = view(T, W, dtype, q, pad, skip)
    h.copy_((h.float() + know * torch.rand(T, 1, generator=q, device="cuda") * w[t].float()).to(dtype))
    t[torch.rand(T, generator=q, device="cuda") < out] = -100
    dloss = (0.5 + torch.rand(T, generator=q, device="cuda")) / max(T, 1)
    return h, w, t.to(index), dloss


def check(g, h, w, t, dloss, scale=1.0, names=("loss", "lse", "dh", "dw")):
    loss, lse = g.gdn_vocab_loss_fwd(h, w, t, scale=scale)
    r = dict(loss=loss, lse=lse, **g.gdn_vocab_loss_bwd(dloss, h, w, t, lse, scale=scale))
    ref = L.vocab_loss(L.dbl(h), L.dbl(w), t, scale, h.dtype is F32, L.dbl(dloss))
    for n in names:
        assert r[n].dtype is (F32 if n in ("loss", "lse") else h.dtype)
        R.assert_within(r[n], ref[n].cpu(), ref[n + "_b"].cpu(), n)
    return r, ref


SIZES = [(1, 1, 1), (1, 1000, 64), (5, 3, 7), (2, 256, 8), (130, 300, 72), (256, 256, 64), (257, 513, 1001), (300, 5000, 512),
         (129, 20000, 256), (1000, 40, 200), (3, 4100, 4096)]


@pytest.mark.parametrize("T,V,W", SIZES)
@pytest.mark.parametrize("dtype,index", [(BF, I64), (F32, I32)])
def test_loss_and_gradients(g, T, V, W, dtype, index):
    check(g, *inputs(T, V, W, dtype, index=index))


@pytest.mark.parametrize("T,V,W,dtype", [(130, 300, 72, BF), (300, 2000, 520, F32)])
@pytest.mark.parametrize("scale", [0.05, -1.3])
def test_scales(g, T, V, W, dtype, scale):
    check(g, *inputs(T, V, W, dtype, seed=1), scale=scale)


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_errors_in_norm(g, dtype):
    """Element-wise bounds grow with the sums; in norm the errors are those of roundings that do not add up.  fp32:
    a logit of order ten is off by a few 2^-24 of itself, and P by as much times ten; bf16 gradients: two roundings
    of 2^-8 / sqrt(3) at the most, P's and the result's."""
    r, ref = check(g, *inputs(700, 9000, 1024, dtype, seed=2))
    assert rel(r["lse"], ref["lse"]) <= 1e-6 and rel(r["loss"], ref["loss"]) <= 1e-6
    most = 2 ** -8 * (2 / 3) ** 0.5 if dtype is BF else 2e-6
    assert rel(r["dh"], ref["dh"]) <= most and rel(r["dw"], ref["dw"]) <= most


@pytest.mark.parametrize("dtype,scale", [(BF, 1.0), (F32, 1.0), (BF, 0.7)])
@pytest.mark.parametrize("T,V,W", [(3, 500, 3200), (5, 200, 700), (60, 3000, 1100), (150, 400, 2048)])
def test_tokens_that_are_nearly_certain(g, dtype, scale, T, V, W):
    """P at a target is p - 1: where that is 1e-4, as for tokens 9 above log V, what counts is that the gradient's logits
    are off as the loss's are.  lse, of order 15, is rounded by up to 2^-21, so that p - 1 is off by that and the few
    2^-24 of its exponential and sum: 2^-20 against 1e-4 is 1 %, on the least certain of tokens, in norm, for fp32."""
    h, w, t, dloss = inputs(T, V, W, dtype, seed=20, know=0.0, out=0.0)
    x = L.dbl(h) @ L.dbl(w).t()
    n = L.dbl(w)[t].square().sum(1)
    lift = (torch.logsumexp(x, 1) + 9.2 - x.gather(1, t[:, None])[:, 0]) / n / scale
    h.copy_((h.float() / scale + lift[:, None].float() * w[t].float()).to(dtype))
    loss, lse = g.gdn_vocab_loss_fwd(h, w, t, scale=scale)
    r = g.gdn_vocab_loss_bwd(dloss, h, w, t, lse, scale=scale)
    ref = L.vocab_loss(L.dbl(h), L.dbl(w), t, scale, dtype is F32, L.dbl(dloss))
    assert 1e-5 < float(ref["loss"].min()) and float(ref["loss"].max()) < 1e-3
    most = 0.01 + (2 ** -8 * (2 / 3) ** 0.5 if dtype is BF else 0.0)
    assert rel(r["dh"], ref["dh"]) <= most and rel(r["dw"], ref["dw"]) <= most


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad,skip", [(8, 0), (3, 1), (0, 4)])
def test_strides_and_alignment(g, dtype, pad, skip):
    """Row-strided views, at any alignment, give the bits of dense rows."""
    for W in (64, 77):
        h, w, t, dloss = inputs(150, 400, W, dtype, seed=3, pad=pad, skip=skip)
        a, _ = check(g, h, w, t, dloss)
        b, _ = check(g, h.clone(memory_format=torch.contiguous_format), w.clone(memory_format=torch.contiguous_format), t, dloss)
        assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tokens_left_out(g, dtype):
    """What a token without a target holds, or one whose dloss is zero, reaches no other token and no weight."""
    h, w, t, dloss = inputs(400, 600, 136, dtype, seed=4, out=0.3)
    dloss[5] = 0
    t[5] = 7
    clean, _ = check(g, h, w, t, dloss)
    bad = t < 0
    h[bad] = float("nan")
    h[bad.nonzero()[0]] = float("inf")
    dloss[bad] = float("nan")
    loss, lse = g.gdn_vocab_loss_fwd(h, w, t)
    r = g.gdn_vocab_loss_bwd(dloss, h, w, t, lse)
    assert torch.equal(loss, clean["loss"]) and torch.equal(lse[~bad], clean["lse"][~bad])
    assert torch.equal(r["dh"], clean["dh"]) and torch.equal(r["dw"], clean["dw"]) and not r["dh"][bad].any()
    h[5] = float("nan")
    assert torch.equal(g.gdn_vocab_loss_bwd(dloss, h, w, t, clean["lse"])["dw"], clean["dw"])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_all_left_out_and_none_at_all(g, dtype):
    h, w, t, dloss = inputs(70, 100, 48, dtype, seed=5, out=1.1)
    r, _ = check(g, h, w, t, dloss)
    assert not r["loss"].any() and not r["dh"].any() and not r["dw"].any()
    loss, lse = g.gdn_vocab_loss_fwd(h[:0], w, t[:0])
    r = g.gdn_vocab_loss_bwd(dloss[:0], h[:0], w, t[:0], lse)
    assert loss.shape == (0,) and r["dh"].shape == (0, 48) and r["dw"].shape == w.shape and not r["dw"].any()


@pytest.mark.parametrize("dtype,index", [(BF, I32), (F32, I64)])
def test_targets_behind_the_vocabulary(g, dtype, index):
    h, w, t, dloss = inputs(40, 100, 48, dtype, seed=6, index=index)
    t[3], t[9] = 100, 2 ** 31 - 1
    loss, lse = g.gdn_vocab_loss_fwd(h, w, t)
    bad = t >= 100
    assert torch.isnan(loss[bad]).all() and torch.isfinite(loss[~bad]).all() and torch.isfinite(lse).all()
    r = g.gdn_vocab_loss_bwd(dloss, h, w, t, lse)
    assert torch.isnan(r["dh"][bad]).all() and torch.isfinite(r["dh"][~bad]).all() and torch.isnan(r["dw"]).all()


@pytest.mark.parametrize("T,V,dtype", [(4200, 140000, BF), (4200, 70000, F32)])
def test_pieces_of_the_vocabulary(g, T, V, dtype):
    """P of more than half a gigabyte: two pieces, the second a short one; many rows of tiles."""
    W = 40
    h, w, t, dloss = inputs(T, V, W, dtype, seed=7)
    loss, lse = g.gdn_vocab_loss_fwd(h, w, t)
    r = g.gdn_vocab_loss_bwd(dloss, h, w, t, lse)
    hd, wd = L.dbl(h), L.dbl(w)
    dw, dh = torch.zeros_like(wd), torch.zeros_like(hd)
    for a in range(0, T, 700):  # 64 bits, in blocks of tokens
        x = hd[a:a + 700] @ wd.t()
        z = torch.logsumexp(x, 1)
        assert rel(lse[a:a + 700], z) <= 1e-6
        tt, real = t[a:a + 700].clamp(min=0), t[a:a + 700] >= 0
        P = torch.exp(x - z[:, None])
        P[torch.arange(len(tt)), tt] -= 1
        P *= torch.where(real, L.dbl(dloss[a:a + 700]), 0.0)[:, None]
        dh[a:a + 700], dw = P @ wd, dw + P.t() @ hd[a:a + 700]
    most = 2 ** -8 * (2 / 3) ** 0.5 if dtype is BF else 4e-6  # (test_errors_in_norm; a sum over twice as many)
    assert rel(r["dh"], dh) <= most and rel(r["dw"], dw) <= most
    assert rel(r["dw"][-300:], dw[-300:]) <= 2 * most and rel(r["dw"][65000:66000], dw[65000:66000]) <= 2 * most


def test_wide_ranges_in_fp32(g):
    """Rows of h over 2^20, weights' elements over 2^12, dloss over 2^24: within the bounds of the scaled parts."""
    h, w, t, dloss = inputs(300, 700, 200, F32, seed=8, know=0.0)
    q = gen(9)
    h *= torch.exp2(torch.randint(-18, 2, (300, 1), generator=q, device="cuda").float())
    w *= torch.exp2(torch.randint(-10, 2, (700, 200), generator=q, device="cuda").float())
    dloss *= torch.exp2(torch.randint(-20, 4, (300,), generator=q, device="cuda").float())
    check(g, h, w, t, dloss)
    for s in (1e-20, 1e20):  # the scalings are by the inputs' own size
        check(g, h * s, w / s, t, dloss, names=("loss", "lse"))


@pytest.mark.parametrize("s", [1e-34, 1e34])
@pytest.mark.parametrize("T", [40, 300])
def test_inputs_at_the_ends_of_fp32_whose_products_are_not(g, T, s):
    h, w, t, dloss = inputs(T, 700, 200, F32, seed=19)
    check(g, h * s, w / s, t, dloss, names=("loss", "lse"))
    _, lse = g.gdn_vocab_loss_fwd(h * s, w / s, t)
    r = g.gdn_vocab_loss_bwd(dloss, h * s, w / s, t, lse)
    assert torch.isfinite(r["dh"]).all() and torch.isfinite(r["dw"]).all()


def test_large_logits(g):
    """Logits of a few hundred: sums of exponentials far from one another, tokens that are certain."""
    for dtype in (BF, F32):
        h, w, t, dloss = inputs(200, 900, 64, dtype, seed=10)
        check(g, h * 40, w, t, dloss)
    h, w = torch.zeros(3, 64, device="cuda"), torch.zeros(50, 64, device="cuda")
    check(g, h, w, torch.tensor([0, 49, -1], device="cuda"), torch.ones(3, device="cuda"))


def test_nan_reaches_its_token(g):
    h, w, t, dloss = inputs(60, 500, 64, BF, seed=11, out=0.0)
    h[7, 3] = float("nan")
    loss, lse = g.gdn_vocab_loss_fwd(h, w, t)
    keep = torch.arange(60, device="cuda") != 7
    assert torch.isnan(loss[7]) and torch.isnan(lse[7]) and torch.isfinite(loss[keep]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_equal_calls_equal_bits_and_other_workspaces(g, dtype):
    h, w, t, dloss = inputs(333, 4001, 328, dtype, seed=12)
    t[t >= 0] = t[t >= 0] % 50  # targets that several tokens have
    a = g.gdn_vocab_loss_fwd(h, w, t)
    r = g.gdn_vocab_loss_bwd(dloss, h, w, t, a[1])
    ws = torch.full((max(g.vocab_loss_bwd_workspace_size(500, 6000, 400, dtype), g.vocab_loss_fwd_workspace_size(500, 6000, 400, dtype)),),
                    255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        b = g.gdn_vocab_loss_fwd(h, w, t, workspace=ws)
        s = g.gdn_vocab_loss_bwd(dloss, h, w, t, b[1], workspace=ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and all(torch.equal(r[n], s[n]) for n in r)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_captured_on_another_stream(g, dtype):
    a, b = inputs(300, 3000, 200, dtype, seed=13), inputs(300, 3000, 200, dtype, seed=14)

    def both(h, w, t, dloss):
        loss, lse = g.gdn_vocab_loss_fwd(h, w, t)
        r = g.gdn_vocab_loss_bwd(dloss, h, w, t, lse)
        return loss, lse, r["dh"], r["dw"]
    want = both(*b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(*a)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(*a)
    for x, y in zip(a, b):
        x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_two_streams_at_once(g):
    """Two calls that overlap, each with a workspace of its own."""
    jobs = [inputs(900, 8000, 512, dt, seed=15 + i) for i, dt in enumerate((BF, F32))]

    def both(h, w, t, dloss):
        loss, lse = g.gdn_vocab_loss_fwd(h, w, t)
        return loss, lse, *g.gdn_vocab_loss_bwd(dloss, h, w, t, lse).values()
    want = [both(*j) for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    got = []
    for j, s in zip(jobs, streams):
        with torch.cuda.stream(s):
            got.append([both(*j) for _ in range(3)][-1])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))


def test_gradient_against_differences(g):
    """The loss along its gradient, by central differences: fp32 losses of order ten are good to about 4e-6 each,
    random over tokens (their weighted mean to a tenth of that), which over a step of 2e-2 is 2e-5; the third
    derivative adds the step's square, 1e-4 of a slope of order one."""
    h, w, t, dloss = inputs(120, 500, 96, F32, seed=17)
    f = lambda h, w: float((L.dbl(dloss) * L.dbl(g.gdn_vocab_loss_fwd(h, w, t, scale=0.7)[0])).sum())
    lse = g.gdn_vocab_loss_fwd(h, w, t, scale=0.7)[1]
    r = g.gdn_vocab_loss_bwd(dloss, h, w, t, lse, scale=0.7)
    slope = float(torch.sqrt(L.dbl(r["dh"]).square().sum() + L.dbl(r["dw"]).square().sum()))
    e = 1e-2 / slope
    d = (f(h + e * r["dh"], w + e * r["dw"]) - f(h - e * r["dh"], w - e * r["dw"])) / 2e-2
    assert abs(d - slope) <= 1e-3 * slope


def test_far_weights(g):
    """Weights, and their gradient, beyond 2^31 elements: the vocabulary's end is as it is alone."""
    W, V = 4096, 2 ** 31 // 4096 + 300
    q = gen(18)
    w = torch.zeros(V, W, dtype=BF, device="cuda")
    w[-300:] = view(300, W, BF, q, std=W ** -0.5)
    h, t, dloss = view(20, W, BF, q), V - 1 - torch.randint(0, 300, (20,), generator=q, device="cuda"), torch.ones(20, device="cuda")
    loss, lse = g.gdn_vocab_loss_fwd(h, w, t)
    x = L.dbl(h) @ L.dbl(w[-300:]).t()
    z = torch.logaddexp(torch.logsumexp(x, 1), torch.log(torch.tensor(V - 300.0, device="cuda").double()))
    assert rel(lse, z) <= 1e-6
    r = g.gdn_vocab_loss_bwd(dloss, h, w, t, lse)
    P = torch.exp(x - z[:, None])
    P[torch.arange(20), t - (V - 300)] -= 1
    assert rel(r["dw"][-300:], P.t() @ L.dbl(h)) <= 2 ** -8 and rel(r["dh"], P @ L.dbl(w[-300:])) <= 2 ** -8


# ---- up to 128 tokens: tiles of one CTA ------------------------------------------

ALONE = [(17, 30, 8), (20, 257, 64), (33, 3000, 520), (64, 513, 72), (65, 700, 2048), (100, 5000, 1001), (127, 20000, 256),
         (128, 1100, 640), (20, 300, 4200), (128, 256, 3)]


@pytest.mark.parametrize("T,V,W", ALONE)
@pytest.mark.parametrize("dtype,index", [(BF, I32), (F32, I64)])
def test_up_to_128_tokens(g, T, V, W, dtype, index):
    check(g, *inputs(T, V, W, dtype, seed=28, index=index))
    h, w, t, dloss = inputs(T, V, W, dtype, seed=29, index=index, out=0.0)
    a, b = (g.gdn_vocab_loss_bwd(dloss, h, w, t, g.gdn_vocab_loss_fwd(h, w, t)[1]) for _ in range(2))
    assert torch.equal(a["dh"], b["dh"]) and torch.equal(a["dw"], b["dw"])


# ---- few tokens: kernels of their own up to 16 of fp32, 4 or 8 of bf16 ------------

FEW = [(1, 8, 1), (1, 9, 3), (2, 100, 8), (3, 513, 66), (4, 1000, 1001), (5, 3001, 520), (7, 700, 4096), (8, 4099, 64),
       (9, 800, 130), (13, 2000, 34), (16, 1023, 2048), (17, 300, 100), (4, 7, 64), (1, 140, 20000), (8, 160, 8200), (8, 700, 1001), (6, 64, 66), (9, 65, 67)]


@pytest.mark.parametrize("T,V,W", FEW)
@pytest.mark.parametrize("dtype,index", [(BF, I32), (F32, I64)])
@pytest.mark.parametrize("scale", [1.0, -0.7])
def test_few_tokens(g, T, V, W, dtype, index, scale):
    check(g, *inputs(T, V, W, dtype, seed=21, index=index, out=0.2), scale=scale)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 4, 6, 15])
@pytest.mark.parametrize("W,pad,skip", [(66, 2, 2), (66, 1, 1), (64, 4, 4), (65, 0, 0), (128, 8, 0), (1346, 0, 0)])
def test_few_tokens_with_rows_of_any_alignment(g, dtype, T, W, pad, skip):
    check(g, *inputs(T, 777, W, dtype, seed=22, pad=pad, skip=skip))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("W", [72, 1001])
def test_few_tokens_left_out_and_behind_the_vocabulary(g, dtype, W):
    h, w, t, dloss = inputs(6, 500, W, dtype, seed=23, out=0.0)
    t[2], dloss[3] = -5, 0.0
    h[2:4] = float("nan")
    loss, lse = g.gdn_vocab_loss_fwd(h, w, t)
    assert loss[2] == 0 and torch.isnan(loss[3])
    r = g.gdn_vocab_loss_bwd(dloss, h, w, t, lse)
    assert (r["dh"][2:4] == 0).all()
    keep = torch.tensor([0, 1, 4, 5], device="cuda")
    one = g.gdn_vocab_loss_bwd(dloss[keep], h[keep], w, t[keep], lse[keep])
    ref = L.vocab_loss(L.dbl(h[keep]), L.dbl(w), t[keep], 1.0, dtype is F32, L.dbl(dloss[keep]))
    for x, n in ((r["dh"][keep], "dh"), (r["dw"], "dw"), (one["dw"], "dw")):
        R.assert_within(x, ref[n].cpu(), ref[n + "_b"].cpu(), n)
    h, w, t, dloss = inputs(3, 500, W, dtype, seed=24, out=0.0)
    t[1] = 500
    loss, lse = g.gdn_vocab_loss_fwd(h, w, t)
    r = g.gdn_vocab_loss_bwd(dloss, h, w, t, lse)
    assert torch.isnan(loss[1]) and torch.isfinite(loss[0::2]).all() and torch.isfinite(lse).all()
    assert torch.isnan(r["dh"][1]).all() and torch.isfinite(r["dh"][0::2]).all() and torch.isnan(r["dw"]).all()


@pytest.mark.parametrize("dtype,T", [(BF, 1), (BF, 7), (F32, 4), (F32, 16)])
def test_few_tokens_in_errors_in_norm_equal_bits_and_captured(g, dtype, T):
    """Errors in norm: dh and dw are fp32 sums, rounded once for bf16 (2^-8 at most, by 1 / sqrt(3) of that in norm
    and less)."""
    h, w, t, dloss = inputs(T, 5003, 1024, dtype, seed=25, out=0.0)
    ref = L.vocab_loss(L.dbl(h), L.dbl(w), t, 1.0, dtype is F32, L.dbl(dloss))
    def both():
        loss, lse = g.gdn_vocab_loss_fwd(h, w, t)
        return dict(loss=loss, lse=lse, **g.gdn_vocab_loss_bwd(dloss, h, w, t, lse))
    a = both()
    for n in ("dh", "dw"):
        assert rel(a[n], ref[n]) <= (2 ** -8 / 3 ** 0.5 if dtype is BF else 2e-6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = both()
    for x in b.values():
        x.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_few_tokens_rows_around_stay_and_far_weights(g):
    """dh and dw of the C ABI in wider rows: what lies between stays; weights beyond 2^31 elements."""
    from linear_attention_sequence_device_gb300 import binding
    lib = binding.load()
    T, V, W = 5, 301, 70
    h, w, t, dloss = inputs(T, V, W, F32, seed=26)
    _, lse = g.gdn_vocab_loss_fwd(h, w, t)
    want = g.gdn_vocab_loss_bwd(dloss, h, w, t, lse)
    dh, dw = torch.full((T, W + 3), 9.0, device="cuda"), torch.full((V, W + 5), 9.0, device="cuda")
    ws = torch.empty(g.vocab_loss_bwd_workspace_size(T, V, W, F32), dtype=torch.uint8, device="cuda")
    st = lib.gdn_vocab_loss_bwd(dloss.data_ptr(), h.data_ptr(), h.stride(0), w.data_ptr(), w.stride(0), 0, t.data_ptr(),
                                64, lse.data_ptr(), T, V, W, 1.0, dh.data_ptr(), W + 3, dw.data_ptr(), W + 5,
                                ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert (dh[:, W:] == 9).all() and (dw[:, W:] == 9).all()
    assert rel(dh[:, :W], L.dbl(want["dh"])) <= 1e-6 and rel(dw[:, :W], L.dbl(want["dw"])) <= 1e-6
    V, W, q = (1 << 19) + 200, 4160, gen(27)
    w = torch.zeros(V, W, dtype=BF, device="cuda")
    w[-300:] = view(300, W, BF, q, std=W ** -0.5)
    h, t, dloss = view(3, W, BF, q), V - 1 - torch.randint(0, 300, (3,), generator=q, device="cuda"), torch.ones(3, device="cuda")
    loss, lse = g.gdn_vocab_loss_fwd(h, w, t)
    x = L.dbl(h) @ L.dbl(w[-300:]).t()
    z = torch.logaddexp(torch.logsumexp(x, 1), torch.log(torch.tensor(V - 300.0, device="cuda").double()))
    assert rel(lse, z) <= 1e-6
    r = g.gdn_vocab_loss_bwd(dloss, h, w, t, lse)
    P = torch.exp(x - z[:, None])
    P[torch.arange(3), t - (V - 300)] -= 1
    assert rel(r["dw"][-300:], P.t() @ L.dbl(h)) <= 2 ** -8 and rel(r["dh"], P @ L.dbl(w[-300:])) <= 2 ** -8


def test_wrong_arguments_raise(g):
    h, w, t, dloss = inputs(10, 30, 16, BF, seed=19)
    lse = torch.zeros(10, device="cuda")
    with pytest.raises(TypeError):
        g.gdn_vocab_loss_fwd(h, w.float(), t)
    with pytest.raises(ValueError):
        g.gdn_vocab_loss_fwd(h, w[:, :8], t)
    with pytest.raises(ValueError):
        g.gdn_vocab_loss_fwd(h, w, t[:9])
    with pytest.raises(TypeError):
        g.gdn_vocab_loss_fwd(h, w, t.float())
    with pytest.raises(ValueError):
        g.gdn_vocab_loss_fwd(h, w, t.cpu())
    with pytest.raises(g.GdnError):
        g.gdn_vocab_loss_fwd(h, w[:0], t)
    with pytest.raises(g.GdnError):
        g.gdn_vocab_loss_fwd(h, w, t, scale=float("inf"))
    with pytest.raises(g.GdnError):
        g.gdn_vocab_loss_bwd(dloss, h, w, t, lse, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        g.gdn_vocab_loss_bwd(dloss[:9], h, w, t, lse)
    with pytest.raises(TypeError):
        g.gdn_vocab_loss_bwd(dloss.double(), h, w, t, lse)
    with pytest.raises(TypeError):
        g.gdn_vocab_loss_fwd(h.half(), w.half(), t)
