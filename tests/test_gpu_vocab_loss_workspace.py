"""One workspace, of the longest call, serves the vocabulary's loss of all shorter ones,
which leave alone what lies behind it."""
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
    yield pkg
    assert pkg.binding.device_timeouts() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V,W", [(3000, 200), (20000, 77), (300, 1024)])
def test_the_longest_calls_workspace_serves_all(g, dtype, V, W):
    q = torch.Generator(device="cuda").manual_seed(0)
    h = torch.randn(513, W, generator=q, device="cuda").to(dtype)
    w = (torch.randn(V, W, generator=q, device="cuda") * W ** -0.5).to(dtype)
    t, dloss = torch.randint(0, V, (513,), generator=q, device="cuda"), torch.rand(513, generator=q, device="cuda")
    n = [f(513, V, W, dtype) for f in (g.vocab_loss_fwd_workspace_size, g.vocab_loss_bwd_workspace_size)]
    room = [torch.full((m + 4096,), 0xAB, dtype=torch.uint8, device="cuda") for m in n]
    fwd, bwd = (r[:m] for r, m in zip(room, n))
    for T in (513, 512, 300, 257, 256, 129, 128, 65, 17, 16, 9, 8, 5, 4, 1):
        a, b, c = h[:T], t[:T], dloss[:T]
        loss, lse = g.gdn_vocab_loss_fwd(a, w, b)
        r = g.gdn_vocab_loss_bwd(c, a, w, b, lse, loss=loss)
        got = g.gdn_vocab_loss_fwd(a, w, b, workspace=fwd)
        assert torch.equal(got[0], loss) and torch.equal(got[1], lse)
        s = g.gdn_vocab_loss_bwd(c, a, w, b, lse, loss=loss, workspace=bwd)
        assert torch.equal(r["dh"], s["dh"]) and torch.equal(r["dw"], s["dw"])
        assert all((x[m:] == 0xAB).all() for x, m in zip(room, n))
