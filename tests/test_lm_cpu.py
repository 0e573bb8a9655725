"""No GPU: refusals of the single-token rule, the embedding and the vocabulary's loss
on the host, their workspaces' sizes, and the 64-bit forms that the GPU tests use."""
import ctypes

import pytest
import torch

import linear_attention_sequence_device_gb300 as g
from linear_attention_sequence_device_gb300 import binding, lm, ssm
from tests import lm_ref as L

FAKE = ctypes.c_void_p(4096)  # never read: every call below fails on the host
ODD = ctypes.c_void_p(4098)


@pytest.fixture(scope="module")
def lib():
    from linear_attention_sequence_device_gb300 import build
    build.build_library()
    return binding.load()


def defaults(names, values, kw):
    a = dict(zip(names.split(), values))
    assert not set(kw) - set(a)
    return list((a | kw).values())


def chunk_step(lib, **kw):
    return lib.gdn_chunk_step(*defaults(
        "q k v ldq ldk ldv dt g beta B Hk Hv dk dv scale flags states slots src dst o stream",
        [FAKE, FAKE, FAKE, 64, 64, 128, 1, FAKE, FAKE, 4, 2, 4, 32, 32, 0.1, 1, FAKE, 9, FAKE, FAKE, FAKE, None], kw))


def layer_step(lib, **kw):
    return lib.gdn_layer_step(*defaults(
        "x ldx a lda b ldb dt A_log dt_bias z ldz norm_w eps B Hk Hv dk dv scale states slots src dst y stream",
        [FAKE, 256, FAKE, 4, FAKE, 4, 1, FAKE, FAKE, FAKE, 128, FAKE, 1e-6, 4, 2, 4, 32, 32, 0.1, FAKE, 9, FAKE, FAKE, FAKE, None], kw))


def embed_fwd(lib, **kw):
    return lib.gdn_embed_fwd(*defaults("tokens bits table ldt dt V T W scale y ldy stream",
                                       [FAKE, 64, FAKE, 16, 1, 9, 5, 16, 1.0, FAKE, 16, None], kw))


def embed_bwd(lib, **kw):
    return lib.gdn_embed_bwd(*defaults("dy lddy dt tokens bits V T W scale acc d ldd ws bytes stream",
                                       [FAKE, 16, 1, FAKE, 64, 9, 5, 16, 1.0, 0, FAKE, 16, FAKE, 1 << 62, None], kw))


def loss_fwd(lib, **kw):
    return lib.gdn_vocab_loss_fwd(*defaults("h ldh w ldw dt t bits T V W scale loss lse ws bytes stream",
                                            [FAKE, 16, FAKE, 16, 1, FAKE, 64, 5, 9, 16, 1.0, FAKE, FAKE, FAKE, 1 << 62, None], kw))


def loss_bwd(lib, **kw):
    return lib.gdn_vocab_loss_bwd(*defaults(
        "dloss h ldh w ldw dt t bits lse T V W scale dh lddh dw lddw ws bytes stream",
        [FAKE, FAKE, 16, FAKE, 16, 1, FAKE, 64, FAKE, 5, 9, 16, 1.0, FAKE, 16, FAKE, 16, FAKE, 1 << 62, None], kw))


INVALID, SHAPE, DTYPE, WORKSPACE = 1, 2, 3, 9
REFUSED = [
    (chunk_step, dict(dt=7), DTYPE), (chunk_step, dict(dk=48), SHAPE), (chunk_step, dict(dv=256), SHAPE), (chunk_step, dict(Hk=3), SHAPE),
    (chunk_step, dict(B=-1), INVALID), (chunk_step, dict(B=1 << 30), SHAPE), (chunk_step, dict(states=ODD), INVALID),
    (chunk_step, dict(states=None), INVALID), (chunk_step, dict(src=None, slots=3), INVALID), (chunk_step, dict(ldq=63), INVALID),
    (chunk_step, dict(ldv=127), INVALID), (chunk_step, dict(k=None), INVALID), (chunk_step, dict(g=None), INVALID),
    (chunk_step, dict(o=None), INVALID), (chunk_step, dict(flags=2), INVALID), (chunk_step, dict(slots=-1), INVALID),
    (layer_step, dict(dt=7), DTYPE), (layer_step, dict(ldx=255), INVALID), (layer_step, dict(lda=3), INVALID), (layer_step, dict(b=None), INVALID),
    (layer_step, dict(norm_w=None), INVALID), (layer_step, dict(ldz=127), INVALID), (layer_step, dict(A_log=None), INVALID),
    (layer_step, dict(dst=None, slots=3), INVALID), (layer_step, dict(y=None), INVALID), (layer_step, dict(dk=33), SHAPE),
    (embed_fwd, dict(dt=2), DTYPE), (embed_fwd, dict(bits=16), DTYPE), (embed_fwd, dict(T=-1), INVALID), (embed_fwd, dict(W=0), INVALID),
    (embed_fwd, dict(V=-1), INVALID), (embed_fwd, dict(T=2 ** 31 - 1), SHAPE), (embed_fwd, dict(W=(1 << 20) + 1), SHAPE),
    (embed_fwd, dict(V=(1 << 30) + 1), SHAPE), (embed_fwd, dict(tokens=None), INVALID), (embed_fwd, dict(table=None), INVALID),
    (embed_fwd, dict(ldt=15), INVALID), (embed_fwd, dict(ldy=15), INVALID),
    (embed_bwd, dict(dt=2), DTYPE), (embed_bwd, dict(bits=0), DTYPE), (embed_bwd, dict(dy=None), INVALID), (embed_bwd, dict(d=None), INVALID),
    (embed_bwd, dict(lddy=15), INVALID), (embed_bwd, dict(ldd=15), INVALID), (embed_bwd, dict(ws=None), WORKSPACE),
    (embed_bwd, dict(bytes=300), WORKSPACE), (embed_bwd, dict(ws=ODD), WORKSPACE),
    (loss_fwd, dict(dt=2), DTYPE), (loss_fwd, dict(bits=8), DTYPE), (loss_fwd, dict(V=0), INVALID), (loss_fwd, dict(T=-1), INVALID),
    (loss_fwd, dict(W=0), INVALID), (loss_fwd, dict(T=(1 << 28) + 1), SHAPE), (loss_fwd, dict(V=(1 << 28) + 1), SHAPE),
    (loss_fwd, dict(W=(1 << 20) + 8), SHAPE), (loss_fwd, dict(h=None), INVALID), (loss_fwd, dict(w=None), INVALID), (loss_fwd, dict(t=None), INVALID),
    (loss_fwd, dict(ldh=15), INVALID), (loss_fwd, dict(h=ODD), INVALID), (loss_fwd, dict(ldw=20), INVALID),
    (loss_fwd, dict(scale=float("nan")), INVALID), (loss_fwd, dict(loss=None), INVALID), (loss_fwd, dict(ws=None), WORKSPACE),
    (loss_fwd, dict(bytes=100), WORKSPACE),
    (loss_bwd, dict(dloss=None), INVALID), (loss_bwd, dict(lse=None), INVALID), (loss_bwd, dict(dh=None), INVALID), (loss_bwd, dict(dw=None), INVALID),
    (loss_bwd, dict(lddh=15), INVALID), (loss_bwd, dict(lddw=15), INVALID), (loss_bwd, dict(ws=ODD), WORKSPACE), (loss_bwd, dict(bytes=1000), WORKSPACE),
    (loss_bwd, dict(w=ODD), INVALID)]


@pytest.mark.parametrize("call,kw,status", REFUSED, ids=lambda v: v.__name__ if callable(v) else None)
def test_refusals(lib, call, kw, status):
    assert call(lib, **kw) == status
    assert lib.gdn_last_error()


def test_nothing_to_do(lib):
    """No requests or tokens, or no vocabulary to fill: nothing is launched."""
    assert chunk_step(lib, B=0, states=None) == 0 and layer_step(lib, B=0) == 0
    assert embed_fwd(lib, T=0, tokens=None) == 0 and embed_bwd(lib, V=0) == 0 and loss_fwd(lib, T=0, h=None, t=None) == 0


def test_workspaces(lib):
    """Sizes are multiples of 256 that do not fall with the tokens, and zero for sizes that are refused."""
    Ts = [0, 1, 100, 4096, 4097, 32768, 32769, 65536, 10 ** 6]
    for W in (1, 64, 1001):
        e = [lib.gdn_embed_bwd_workspace_size(T, 50, W) for T in Ts]
        assert e == sorted(e) and all(v % 256 == 0 for v in e)
    assert lib.gdn_embed_bwd_workspace_size(-1, 9, 8) == lib.gdn_embed_bwd_workspace_size(5, 9, 0) == lib.gdn_embed_bwd_workspace_size(5, -1, 8) == 0
    for dt in (0, 1):
        for size in (lib.gdn_vocab_loss_fwd_workspace_size, lib.gdn_vocab_loss_bwd_workspace_size):
            assert all(size(T, 1000, 64, dt) % 256 == 0 and size(T, 1000, 64, dt) > 0 for T in Ts)
            assert size(5, 0, 64, dt) == size(5, 9, 0, dt) == size(-1, 9, 8, dt) == 0
    assert lib.gdn_vocab_loss_fwd_workspace_size(5, 9, 8, 3) == 0


class Elsewhere:
    """What the front end may ask of a tensor on device 1 before it refuses it."""
    dtype = torch.bfloat16
    is_cuda = True

    def get_device(self):
        return 1


X = Elsewhere()
CALLS = dict(chunk_step=lambda: g.gdn_chunk_step(X, X, X, X, X, X),
             layer_step=lambda: g.gdn_layer_step(X, X, X, X, X, X, X, X, 1, 1, 32, 32), embed_fwd=lambda: g.gdn_embed_fwd(X, X),
             embed_bwd=lambda: g.gdn_embed_bwd(X, X, 5), loss_fwd=lambda: g.gdn_vocab_loss_fwd(X, X, X),
             loss_bwd=lambda: g.gdn_vocab_loss_bwd(X, X, X, X, X))


@pytest.mark.parametrize("name", CALLS)
def test_another_device_is_refused(name, monkeypatch):
    monkeypatch.setattr(binding, "_current_device", lambda: 0)

    def used(*a, **kw):
        raise AssertionError("allocated or launched")
    for n in ("empty", "empty_like"):
        monkeypatch.setattr(torch, n, used)
    monkeypatch.setattr(lm, "_run", used)
    monkeypatch.setattr(lm, "_raw_stream", used)
    with pytest.raises(ValueError, match="current device"):
        CALLS[name]()
    monkeypatch.setattr(ssm, "_run", used)


def test_tensors_on_the_host_are_refused():
    x = torch.zeros(3, 8)
    for call in (lambda: g.gdn_embed_fwd(torch.zeros(2, dtype=torch.int64), x), lambda: g.gdn_embed_bwd(x, torch.zeros(3, dtype=torch.int64), 4),
                 lambda: g.gdn_vocab_loss_fwd(x, x, torch.zeros(3, dtype=torch.int64)),
                 lambda: g.gdn_chunk_step(x[:, None], x[:, None], x[:, None], x, x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


# ---- the 64-bit forms --------------------------------------------------------------

def test_rule_form_by_matrices():
    q = torch.Generator().manual_seed(0)
    rn = lambda *s: torch.randn(*s, generator=q, dtype=torch.float64)
    B, Hk, Hv, dk, dv = 2, 1, 2, 5, 4
    qq, k, v, S = rn(B, Hk, dk), rn(B, Hk, dk), rn(B, Hv, dv), rn(B, Hv, dk, dv)
    gate, beta = L.gates(rn(B, Hv), rn(B, Hv), rn(Hv), rn(Hv))
    o, _, new, _ = L.rule_step(qq, k, v, gate, beta, S, 0.3, True)
    for b in range(B):
        for h in range(Hv):
            kk = k[b, 0] / torch.sqrt(k[b, 0] @ k[b, 0] + 1e-6)
            qn = qq[b, 0] / torch.sqrt(qq[b, 0] @ qq[b, 0] + 1e-6)
            M = (torch.eye(dk, dtype=torch.float64) - beta[b, h] * torch.outer(kk, kk)) @ S[b, h] * gate[b, h].exp()
            M = M + beta[b, h] * torch.outer(kk, v[b, h])
            assert torch.allclose(new[b, h], M) and torch.allclose(o[b, h], 0.3 * qn @ M)


def test_loss_form_by_autograd():
    q = torch.Generator().manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=q, dtype=torch.float64)
    h, w, t = rn(7, 5).requires_grad_(), rn(9, 5).requires_grad_(), torch.tensor([0, 8, -100, 3, 3, -1, 2])
    dl = torch.rand(7, generator=q, dtype=torch.float64)
    loss = torch.nn.functional.cross_entropy(0.4 * h @ w.t(), t.clamp(min=-100).where(t >= 0, torch.tensor(-100)), reduction="none")
    dh, dw = torch.autograd.grad(loss, (h, w), dl)
    r = L.vocab_loss(h.detach(), w.detach(), t, 0.4, True, dl)
    assert torch.allclose(r["loss"], loss.detach()) and torch.allclose(r["dh"], dh) and torch.allclose(r["dw"], dw)


def test_embedding_form_by_autograd():
    q = torch.Generator().manual_seed(2)
    table = torch.randn(6, 3, generator=q, dtype=torch.float64).requires_grad_()
    tok, dy = torch.tensor([0, 5, 2, 2, 0]), torch.randn(5, 3, generator=q, dtype=torch.float64)
    d, = torch.autograd.grad(table[tok] * 2.0, table, dy)
    got, _ = L.embed_bwd(torch.cat([dy, dy[:2]]), torch.cat([tok, torch.tensor([-1, 6])]), 6, 2.0)
    assert torch.allclose(got, d)
