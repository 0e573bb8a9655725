"""The vocabulary's loss of tokens that are nearly certain: losses of 1e-5 beside logits
of 15 to 300 keep their digits, and so do the gradients that are told the loss."""
import pytest
import torch

from tests import lm_ref as L
from tests import ssm_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
CASES = [(T, V, W, dtype, lse) for T, V, W in ((3, 700, 64), (60, 3000, 256), (300, 900, 136)) for dtype in (BF, F32)
         for lse in (15.0, 30.0, 100.0, 300.0)]


@pytest.fixture(scope="module")
def g():
    from linear_attention_sequence_device_gb300 import build
    build.build_library()
    import linear_attention_sequence_device_gb300 as pkg
    pkg.load()
    yield pkg
    assert pkg.binding.device_timeouts() == 0


def certain(T, V, W, dtype, lse, seed=0):
    """Tokens whose other words' probabilities sum to 1e-6 to 1e-3, with log sums of exponentials near lse: column 0
    shifts all logits of a token alike."""
    q = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=q, device="cuda")
    w = rn(V, W) * W ** -0.5
    w[:, 0] = 1.0
    w = w.to(dtype)
    t = torch.randint(0, V, (T,), generator=q, device="cuda")
    h = rn(T, W)
    h[:, 0] = 0.0
    wt = w[t].float()
    wt[:, 0] = 0.0
    for _ in range(3):  # (the lift moves the other words' logits too)
        x = L.dbl(h) @ L.dbl(w).t()
        others = torch.logsumexp(x.scatter(1, t[:, None], -torch.inf), 1)
        h += ((others + 11.0 - x.gather(1, t[:, None])[:, 0]).float() / wt.square().sum(1))[:, None] * wt
    h[:, 0] = lse - 11.0 - others.float()
    return h.to(dtype), w, t, (0.5 + torch.rand(T, generator=q, device="cuda")) / T


def reference(h, w, t, dloss):
    """The 64-bit form, and how far 1 - p of any token may be off, relative to itself: by what two logits are (lm_ref.py:
    K in steps of 16 terms, each cut by 2^-22 of the terms' magnitudes, as many more of joining, and for fp32 the parts'
    2^-21 of them and 2^-38 of the largest products), by the exponentials' 2^-20, and by roundings of the sums and of
    the logarithm."""
    ref = L.vocab_loss(L.dbl(h), L.dbl(w), t, 1.0, h.dtype is F32, L.dbl(dloss))
    V, W = w.shape
    mag = float((L.dbl(h).abs() @ L.dbl(w).abs().t()).max())
    ex = (W / 16 + 16) * 2.0 ** -22 * mag
    if h.dtype is F32:
        ex += 2.0 ** -21 * mag + 2.0 ** -38 * W * float(L.dbl(h).abs().max() * L.dbl(w).abs().max())
    assert 1e-6 < float(ref["loss"].min()) and float(ref["loss"].max()) < 1e-3
    return ref, 2 * ex + 2.0 ** -20 + (96 + V / 256) * L.U


@pytest.mark.parametrize("T,V,W,dtype,lse", CASES)
def test_small_losses_keep_their_digits(g, T, V, W, dtype, lse):
    h, w, t, dloss = certain(T, V, W, dtype, lse)
    ref, most = reference(h, w, t, dloss)
    loss, got = g.gdn_vocab_loss_fwd(h, w, t)
    assert ((L.dbl(loss) - ref["loss"]).abs() <= most * ref["loss"]).all()
    assert ((L.dbl(got) - ref["lse"]).abs() <= ref["lse_b"]).all()


@pytest.mark.parametrize("T,dtype", [(3, BF), (40, BF), (300, BF), (3, F32)])
def test_infinite_logits(g, T, dtype):
    """A target that is impossible has an infinite loss, one that alone is possible has none; an infinite logit gives NaN."""
    h, w = torch.zeros(T, 64, dtype=dtype, device="cuda"), torch.zeros(300, 64, dtype=dtype, device="cuda")
    h[:, 0] = 1.0
    w[5, 0] = -torch.inf
    t = torch.full((T,), 5, device="cuda")
    t[1], t[2] = 7, -1
    loss, lse = g.gdn_vocab_loss_fwd(h, w, t)
    keep = torch.arange(T, device="cuda") != 1
    keep[2] = False
    assert (loss[keep] == torch.inf).all() and loss[2] == 0
    some = torch.log(torch.tensor(299.0))
    assert abs(float(loss[1] - some)) <= 1e-5 and ((lse - some).abs() <= 1e-5).all()
    w[:, 0] = -torch.inf
    w[7, 0] = 2.0
    loss, lse = g.gdn_vocab_loss_fwd(h, w, t)
    assert loss[1] == 0 and (lse == 2).all() and (loss[keep] == torch.inf).all()
    w[:, 0] = 0.0
    w[5, 0] = torch.inf
    loss, lse = g.gdn_vocab_loss_fwd(h, w, t)
    assert torch.isnan(loss[keep]).all() and torch.isnan(lse).all() and loss[2] == 0


# ---- gradients that are told the loss ---------------------------------------------------

def both(g, h, w, t, dloss, scale=1.0):
    loss, lse = g.gdn_vocab_loss_fwd(h, w, t, scale=scale)
    return dict(loss=loss, lse=lse, **g.gdn_vocab_loss_bwd(dloss, h, w, t, lse, scale=scale, loss=loss))


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("T,V,W,dtype,lse", CASES)
def test_gradients_of_small_losses_keep_their_digits(g, T, V, W, dtype, lse):
    """A token's P is off by as much of itself as its 1 - p, in norm with bf16's two roundings (P's and the result's,
    2^-8 / sqrt(3) at the most), or 2e-6 of fp32's parts and sums; and by the rounded lse, 2^-24 of it, all of it alike."""
    h, w, t, dloss = certain(T, V, W, dtype, lse, seed=1)
    ref, most = reference(h, w, t, dloss)
    r = both(g, h, w, t, dloss)
    most += (2 ** -8 * (2 / 3) ** 0.5 if dtype is BF else 2e-6) + 2 * L.U * float(ref["lse"].max())
    assert rel(r["dh"], ref["dh"]) <= most and rel(r["dw"], ref["dw"]) <= most


@pytest.mark.parametrize("T,V,W", [(1, 1, 1), (1, 9, 3), (4, 300, 64), (9, 300, 77), (16, 1000, 520), (40, 257, 72), (128, 513, 1001),
                                   (130, 5000, 256), (300, 700, 40)])
@pytest.mark.parametrize("dtype,index,scale", [(BF, torch.int32, 1.0), (F32, torch.int64, -0.7)])
def test_ordinary_gradients(g, T, V, W, dtype, index, scale):
    """Within lm_ref.py's bounds, tokens left out among them, as without the loss."""
    h, w, t, dloss = certain_or_not(T, V, W, dtype, index)
    r = both(g, h, w, t, dloss, scale)
    ref = L.vocab_loss(L.dbl(h), L.dbl(w), t, scale, dtype is F32, L.dbl(dloss))
    for n in ("dh", "dw"):
        R.assert_within(r[n], ref[n].cpu(), ref[n + "_b"].cpu(), n)


def certain_or_not(T, V, W, dtype, index, seed=2):
    q = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=q, device="cuda")
    w = (rn(V, W) * W ** -0.5).to(dtype)
    t = torch.randint(0, V, (T,), generator=q, device="cuda")
    h = (rn(T, W) + 6.0 * torch.rand(T, 1, generator=q, device="cuda") * w[t].float()).to(dtype)
    if T > 2:
        t[torch.rand(T, generator=q, device="cuda") < 0.15] = -100
    return h, w, t.to(index), (0.5 + torch.rand(T, generator=q, device="cuda")) / T


@pytest.mark.parametrize("T,V,dtype", [(4200, 140000, BF), (4200, 70000, F32)])
def test_pieces_of_the_vocabulary(g, T, V, dtype):
    """P of more than half a gigabyte, in two pieces: what the loss tells about ordinary tokens is what lse tells, up to
    the latter's rounding (2^-20, of p - 1 of order one) and, for bf16, steps of the results that fall the other way."""
    h, w, t, dloss = certain_or_not(T, V, 40, dtype, torch.int64)
    r = both(g, h, w, t, dloss)
    s = g.gdn_vocab_loss_bwd(dloss, h, w, t, r["lse"])
    for n in ("dh", "dw"):
        assert rel(r[n], s[n].double()) <= (2 ** -9 if dtype is BF else 1e-5)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [4, 60, 300])
def test_tokens_left_out_and_equal_bits_in_a_graph(g, T, dtype):
    """What a token without a target or with a dloss of zero holds, its loss among it, reaches nothing; replayed, the bits
    are those of eager calls."""
    h, w, t, dloss = certain(T, 600, 72, dtype, 30.0, seed=3)
    t[1], dloss[2] = -(2 ** 63), 0.0
    a = both(g, h, w, t, dloss)
    h[1:3] = float("nan")
    loss, lse = g.gdn_vocab_loss_fwd(h, w, t)
    assert loss[1] == 0 and torch.isnan(loss[2])
    dloss[1] = float("nan")
    b = g.gdn_vocab_loss_bwd(dloss, h, w, t, lse, loss=loss)
    assert torch.equal(a["dh"], b["dh"]) and torch.equal(a["dw"], b["dw"]) and not b["dh"][1:3].any()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(g, h, w, t, dloss)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = both(g, h, w, t, dloss)
    for x in c.values():
        x.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c["dh"], a["dh"]) and torch.equal(c["dw"], a["dw"])


def test_targets_behind_the_vocabulary(g):
    for T, dtype in ((3, F32), (40, BF), (40, F32)):
        h, w, t, dloss = certain_or_not(T, 100, 48, dtype, torch.int64)
        t[1] = 100
        r = both(g, h, w, t, dloss)
        keep = torch.arange(T, device="cuda") != 1
        assert torch.isnan(r["dh"][1]).all() and torch.isfinite(r["dh"][keep]).all() and torch.isnan(r["dw"]).all()


def test_wrong_losses_raise(g):
    h, w, t, dloss = certain_or_not(10, 30, 16, BF, torch.int64)
    loss, lse = g.gdn_vocab_loss_fwd(h, w, t)
    with pytest.raises(ValueError):
        g.gdn_vocab_loss_bwd(dloss, h, w, t, lse, loss=loss[:9])
    with pytest.raises(TypeError):
        g.gdn_vocab_loss_bwd(dloss, h, w, t, lse, loss=loss.double())
    with pytest.raises(ValueError):
        g.gdn_vocab_loss_bwd(dloss, h, w, t, lse, loss=loss.cpu())
