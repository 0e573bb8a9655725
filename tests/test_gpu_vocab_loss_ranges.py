"""The vocabulary's loss in fp32 where h, w and dloss lie near the ends of fp32's range
and their products do not: gradients against the 64-bit form, in norm."""
import pytest
import torch

from tests import lm_ref as L
from tests import ssm_ref as R

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.fixture(scope="module")
def g():
    from linear_attention_sequence_device_gb300 import build
    build.build_library()
    import linear_attention_sequence_device_gb300 as pkg
    pkg.load()
    yield pkg
    assert pkg.binding.device_timeouts() == 0


def inputs(T, V, W, seed):
    q = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=q, device="cuda")
    w = rn(V, W) * W ** -0.5
    t = torch.randint(0, V, (T,), generator=q, device="cuda")
    h = rn(T, W) + 6.0 * torch.rand(T, 1, generator=q, device="cuda") * w[t]
    t[torch.rand(T, generator=q, device="cuda") < 0.15] = -100
    return h, w, t, (0.5 + torch.rand(T, generator=q, device="cuda")) / T


def off(a, b):
    """How far a is from b in norm, less what results below fp32's normal numbers lose (two roundings of 2^-150)."""
    err = float((a.double() - b).norm()) - 2 * 2.0 ** -150 * b.numel() ** 0.5
    return err / float(b.norm())


@pytest.mark.parametrize("T", [40, 300])
@pytest.mark.parametrize("s", [1e-34, 1e-32, 1e-20, 1e20, 1e34])
@pytest.mark.parametrize("less", [1.0, 1e-3])
def test_gradients(g, T, s, less):
    """Scalings by powers of two take no digits: fp32 errors as for inputs of order one (a logit of order ten is off by a
    few 2^-24 of itself, P by as much times ten)."""
    h, w, t, dloss = inputs(T, 700, 200, 19)
    h, w, dloss = h * s, w / s, dloss * less
    ref = L.vocab_loss(L.dbl(h), L.dbl(w), t, 1.0, True, L.dbl(dloss))
    loss, lse = g.gdn_vocab_loss_fwd(h, w, t)
    for r in (g.gdn_vocab_loss_bwd(dloss, h, w, t, lse), g.gdn_vocab_loss_bwd(dloss, h, w, t, lse, loss=loss)):
        assert off(r["dh"], ref["dh"]) <= 2e-6 and off(r["dw"], ref["dw"]) <= 2e-6


@pytest.mark.parametrize("T", [40, 300])
def test_tokens_of_very_different_sizes(g, T):
    """dw where single tokens' h and dloss are far from the others', one row subnormal, one zero, one token without a
    gradient larger than all."""
    h, w, t, dloss = inputs(T, 300, 136, 20)
    t = t.clamp(min=0)
    h[0], h[1], dloss[2] = 0.0, h[1] * 1e-40, 0.0
    h[2] *= 1e4
    dloss[3] *= 1e-30
    h[4], dloss[4] = h[4] * 1e-20, dloss[4] * 1e20
    ref = L.vocab_loss(L.dbl(h), L.dbl(w), t, 1.0, True, L.dbl(dloss))
    _, lse = g.gdn_vocab_loss_fwd(h, w, t)
    r = g.gdn_vocab_loss_bwd(dloss, h, w, t, lse)
    assert off(r["dw"], ref["dw"]) <= 2e-6
    keep = dloss < 1e10  # (token 4's dh outweighs the others')
    assert off(r["dh"][keep], ref["dh"][keep]) <= 2e-6 and off(r["dh"][~keep], ref["dh"][~keep]) <= 2e-6


@pytest.mark.parametrize("T", [9, 40, 300])
@pytest.mark.parametrize("s", [2.0 ** 6, 2.0 ** 12, 2.0 ** 20])
def test_one_large_row_of_w(g, T, s):
    """A word far larger than all others that no token has as its target, and none likely.  The forward scales w by its
    rows; the gradients by one for all, under which the others keep what the largest leaves them: within lm_ref.py's
    bounds, which count 2^-38 of it, and in norm by as much more as that is of the other rows' elements (of size 200^-0.5)."""
    h, w, t, dloss = inputs(T, 700, 200, 21)
    h[:, 0] = 1.0
    w[:, 0] = 0.0
    row = int(torch.arange(700, device="cuda")[~torch.isin(torch.arange(700, device="cuda"), t)][0])
    w[row] = 0.0
    w[row, 0] = -s
    ref = L.vocab_loss(L.dbl(h), L.dbl(w), t, 1.0, True, L.dbl(dloss))
    loss, lse = g.gdn_vocab_loss_fwd(h, w, t)
    assert off(loss, ref["loss"]) <= 1e-6 and off(lse, ref["lse"]) <= 1e-6
    for r in (g.gdn_vocab_loss_bwd(dloss, h, w, t, lse), g.gdn_vocab_loss_bwd(dloss, h, w, t, lse, loss=loss)):
        for n in ("dh", "dw"):
            R.assert_within(r[n], ref[n].cpu(), ref[n + "_b"].cpu(), n)
            assert off(r[n], ref[n]) <= 2e-6 + 2.0 ** -38 * s * 200 ** 0.5
