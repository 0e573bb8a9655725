"""The vocabulary's gradients in bf16 as sums over a million tokens or words: the tensor
cores cut every step's sum towards zero, which must not add up over the whole of them."""
import pytest
import torch

from tests import lm_ref as L
from tests import ssm_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
# Of a chunk of 4096 terms, in steps of 16, every term may lose 2^-24 of the sum so far, half of the last one's on average
# (2^-13 of it in all), and of the 16384 that short chains and those of up to 128 tokens have four times that.
CHUNK = 2.0 ** -13


@pytest.fixture(scope="module")
def g():
    from linear_attention_sequence_device_gb300 import build
    build.build_library()
    import linear_attention_sequence_device_gb300 as pkg
    pkg.load()
    yield pkg
    assert pkg.binding.device_timeouts() == 0
    torch.cuda.empty_cache()


def gradients(g, h, w, t, dloss):
    loss, lse = g.gdn_vocab_loss_fwd(h, w, t)
    return g.gdn_vocab_loss_bwd(dloss, h, w, t, lse, loss=loss)


def along(got, ref):
    """got's part along ref, less one."""
    return float((got.double() * ref).sum() / ref.square().sum()) - 1.0


def ones_to_twos(*shape, seed=0):
    q = torch.Generator(device="cuda").manual_seed(seed)
    return (1.0 + torch.rand(*shape, generator=q, device="cuda")).to(BF)


@pytest.mark.parametrize("T", [1 << 17, 1 << 20])
def test_dw_over_many_tokens(g, T):
    """Logits of zero: P is 2^-8 for all words but the target, exactly.  The columns' sums, of T numbers between 1 and 2,
    lie within 2^-9 of one another (their spread is 0.3 / sqrt(T), below 2^-10), closer than the steps of bf16: all may be
    rounded the same way, by 2^-8."""
    V, W = 256, 256
    h, w = ones_to_twos(T, W), torch.zeros(V, W, dtype=BF, device="cuda")
    t = torch.full((T,), 3, device="cuda")
    r = gradients(g, h, w, t, torch.ones(T, device="cuda"))
    ref = torch.zeros(W, dtype=torch.float64, device="cuda")
    for a in range(0, T, 1 << 16):
        ref += h[a:a + (1 << 16)].double().sum(0)
    assert abs(along(r["dw"][0], ref / V)) <= CHUNK + 2.0 ** -8
    assert abs(along(r["dw"][3], ref / V - ref)) <= CHUNK + 2.0 ** -8
    assert torch.equal(r["dw"][0], r["dw"][255])


@pytest.mark.parametrize("T,chunks", [(100, 4), (140, 1)])
@pytest.mark.parametrize("V", [1 << 17, 1 << 20])
def test_dh_over_many_words(g, T, V, chunks):
    """The words' mean under softmax, which is dh and the target's row.  Beside the chunks: P's roundings, 2^-8 each, over V
    of them, and dh's, 2^-8 of the rows' differences over T x 64, which differ from one another: below 2^-16 both."""
    W = 64
    q = torch.Generator(device="cuda").manual_seed(2)
    w = (torch.randn(V, W, generator=q, device="cuda") * W ** -0.5 + 0.5).to(BF)
    h, t = torch.randn(T, W, generator=q, device="cuda").to(BF), torch.randint(0, V, (T,), generator=q, device="cuda")
    r = gradients(g, h, w, t, torch.ones(T, device="cuda"))
    mean = torch.softmax(h.double() @ w.double().t(), 1) @ w.double()
    assert abs(along(r["dh"].double() + w[t].double(), mean)) <= chunks * CHUNK + 2.0 ** -15


@pytest.mark.parametrize("T,V,W", [(16385, 300, 77), (20000, 300, 72), (17000, 700, 264), (200, 20000, 72), (130, 300000, 9)])
def test_long_chains_of_ordinary_tokens(g, T, V, W):
    """Results that leave the chunks by copies of boxes and by rows, targets of one and of many tokens, tokens left out:
    within lm_ref.py's bounds."""
    q = torch.Generator(device="cuda").manual_seed(3)
    w = (torch.randn(V, W, generator=q, device="cuda") * W ** -0.5).to(BF)
    t = torch.randint(0, V, (T,), generator=q, device="cuda")
    t[: T // 2] = t[: T // 2] % 7  # (the others' words mostly have one token, or none, where V is large)
    h = (torch.randn(T, W, generator=q, device="cuda") + 6.0 * torch.rand(T, 1, generator=q, device="cuda") * w[t].float()).to(BF)
    t[torch.rand(T, generator=q, device="cuda") < 0.1] = -1
    dloss = (0.5 + torch.rand(T, generator=q, device="cuda")) / T
    r = gradients(g, h, w, t, dloss)
    ref = L.vocab_loss(L.dbl(h), L.dbl(w), t, 1.0, False, L.dbl(dloss))
    for n in ("dh", "dw"):
        R.assert_within(r[n], ref[n].cpu(), ref[n + "_b"].cpu(), n)
        assert float((r[n].double() - ref[n]).norm()) <= (2 ** -8 * (2 / 3) ** 0.5 + 4 * CHUNK) * float(ref[n].norm())
