"""The vocabulary's loss of tokens that are nearly certain: losses of 1e-5 beside logits
of 15 to 300 keep their digits, and so do the gradients that are told the loss."""
import pytest
import torch

from tests import lm_ref as L

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
