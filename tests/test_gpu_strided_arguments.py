"""Arguments that the binding copies to be contiguous: several in one call keep
memory of their own (a and b, or g and beta, as slices of one projection)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    from linear_attention_sequence_device_gb300 import build
    build.build_library()
    import linear_attention_sequence_device_gb300 as pkg
    pkg.load()
    return pkg


def rnd(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda()


def test_layer_gates_as_slices(g):
    T, H, d = 40, 2, 32
    cu = torch.tensor([0, 15, T], dtype=torch.int32, device="cuda")
    x, w, ab = rnd(T, 3 * H * d, seed=0), rnd(3 * H * d, 4, seed=1), rnd(T, 2 * H, seed=2)
    rest = (rnd(H, seed=3), rnd(H, seed=4), rnd(T, H, d, seed=5), rnd(d, seed=6), cu, H, H, d, d, 1)
    y, S, _ = g.gdn_layer_fwd(x, w, None, ab[:, :H], ab[:, H:], *rest)
    y2, S2, _ = g.gdn_layer_fwd(x, w, None, ab[:, :H].contiguous(), ab[:, H:].contiguous(), *rest)
    assert torch.equal(y, y2) and torch.equal(S, S2)


def test_chunk_gates_as_slices(g):
    T, H, d = 40, 2, 32
    cu = torch.tensor([0, 15, T], dtype=torch.int32, device="cuda")
    q, k, v = (rnd(T, H, d, seed=i) for i in range(3))
    gb = torch.sigmoid(rnd(T, 2 * H, seed=3))
    o, S = g.gdn_chunk_fwd(q, k, v, -gb[:, :H], gb[:, H:], cu, l2norm=True)
    gate = gb - 0.0
    o1, S1 = g.gdn_chunk_fwd(q, k, v, (-gate[:, :H]).contiguous(), gate[:, H:].contiguous(), cu, l2norm=True)
    o2, S2 = g.gdn_chunk_fwd(q, k, v, torch.neg(gate)[:, :H], gate[:, H:], cu, l2norm=True)
    assert torch.equal(o, o1) and torch.equal(o1, o2) and torch.equal(S1, S2) and torch.equal(S, S1)
