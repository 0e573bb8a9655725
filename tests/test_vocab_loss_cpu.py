"""No GPU: what the vocabulary's loss refuses and sizes on the host, beside test_lm_cpu.py."""
import pytest

from tests.test_lm_cpu import FAKE, INVALID, SHAPE, WORKSPACE, ODD, defaults, lib  # noqa: F401


def from_loss(lib, **kw):  # noqa: F811
    return lib.gdn_vocab_loss_bwd_from_loss(*defaults(
        "dloss h ldh w ldw dt t bits loss lse T V W scale dh lddh dw lddw ws bytes stream",
        [FAKE, FAKE, 16, FAKE, 16, 1, FAKE, 64, FAKE, FAKE, 5, 9, 16, 1.0, FAKE, 16, FAKE, 16, FAKE, 1 << 62, None], kw))


@pytest.mark.parametrize("kw,status", [(dict(loss=None), INVALID), (dict(lse=None), INVALID), (dict(dloss=None), INVALID),
                                       (dict(V=0), INVALID), (dict(V=(1 << 28) + 1), SHAPE), (dict(ws=ODD), WORKSPACE),
                                       (dict(bytes=1000), WORKSPACE), (dict(lddw=15), INVALID)])
def test_refusals_of_the_gradient_from_the_loss(lib, kw, status):  # noqa: F811
    assert from_loss(lib, **kw) == status
    assert lib.gdn_last_error()


@pytest.mark.parametrize("V,W", [(32000, 2048), (1000, 64), (300, 72), (131072, 1001), (64, 20), (20, 4096), (5310, 3498), (50021, 12800)])
@pytest.mark.parametrize("dt", [0, 1])
def test_workspaces_do_not_fall_with_the_tokens(lib, V, W, dt):  # noqa: F811
    """One for the longest call serves all."""
    Ts = [*range(0, 1400), *(256 * n + d for n in range(6, 78) for d in (0, 1)), *range(20000, 300000, 7919), 1 << 20, 1 << 28]
    assert Ts == sorted(Ts)
    for size in (lib.gdn_vocab_loss_fwd_workspace_size, lib.gdn_vocab_loss_bwd_workspace_size):
        n = [size(T, V, W, dt) for T in Ts]
        assert n == sorted(n) and all(v > 0 and v % 256 == 0 for v in n)
