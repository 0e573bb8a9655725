"""Front end of a language model's two ends and of the gated delta rule's single
tokens (see gdn_cp.h): the embedding lookup, the cross entropy over a vocabulary
from hidden states and output weights, each with its gradient, and the rule and
its layer for one token of each request over a cache of states.

Argument marshalling only, as in ssm.py: on the current stream of the current
device, which has to be the tensors'; wrong arguments raise before anything is
launched, and results have no autograd history.  Tokens and targets are int64 or
int32.
"""
from __future__ import annotations

import torch

from .binding import GDN_QK_L2NORM, load
from .ssm import _CODE, _F32, _I32, _c, _dense, _lead, _lib, _ptr, _raw_stream, _rows, _run, _workspace, _wrong

_BITS = {torch.int64: 64, torch.int32: 32}


def _index(t, name, dev):
    """Address and bits of a vector of tokens."""
    bits = _BITS.get(t.dtype)
    if bits is None:
        raise TypeError(f"{name} must be int64 or int32, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on CUDA device {dev}")
    if t.dim() != 1:
        raise ValueError(f"{name} must be a vector, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr(), bits


def _heads(t, name, dtype, dev, shape):
    """Address and row stride of a [B, H, d] view whose (H, d) part is dense."""
    if t is None:
        return None, 0
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        _wrong(t, name, dtype, dev, shape)
    s = t.stride()
    n, H, d = shape
    if (d > 1 and s[2] != 1) or (H > 1 and s[1] != d):
        raise ValueError(f"{name} must be a [B, H, d] view with dense heads")
    return t.data_ptr(), s[0] if n > 1 else H * d


# ----------------------------------------------------------------------------
# the gated delta rule, single tokens
# ----------------------------------------------------------------------------

def gdn_chunk_step(q, k, v, g, beta, states, src=None, dst=None, scale=None, l2norm=False, out=None):
    """One token of each request through the gated delta rule: q, k [B, Hk, dk],
    v [B, Hv, dv] (row-strided views will do), g [B, Hv] fp32, beta [B, Hv];
    states [slots, Hv, dk, dv] fp32, updated in place; src, dst int32 [B]: the
    slot that request i reads and the one it writes (None: slot i; src < 0: a
    zero state; dst < 0: a padded row).  Returns o [B, Hv, dv]."""
    dev, code = _lead(q, "q")
    e, (B, Hk, dk), (Hv, dv), n = q.dtype, q.shape, v.shape[1:], states.shape[0]
    g, beta = _c(g), _c(beta)
    o = torch.empty((B, Hv, dv), dtype=e, device=q.device) if out is None else out
    (qp, ldq), (kp, ldk) = _heads(q, "q", e, dev, (B, Hk, dk)), _heads(k, "k", e, dev, (B, Hk, dk))
    vp, ldv = _heads(v, "v", e, dev, (B, Hv, dv))
    _run(_lib().gdn_chunk_step(qp, kp, vp, ldq, ldk, ldv, code, _ptr(g, "g", _F32, dev, (B, Hv)),
                               _ptr(beta, "beta", e, dev, (B, Hv)), B, Hk, Hv, dk, dv,
                               dk ** -0.5 if scale is None else scale, GDN_QK_L2NORM if l2norm else 0,
                               _dense(states, "states", _F32, dev, (n, Hv, dk, dv)), n,
                               _dense(src, "src", _I32, dev, (B,)), _dense(dst, "dst", _I32, dev, (B,)),
                               _dense(o, "out", e, dev, (B, Hv, dv)), _raw_stream(dev)))
    return o


def gdn_layer_step(x, a, b, A_log, dt_bias, z, norm_w, states, Hk, Hv, dk, dv, src=None, dst=None, eps=1e-6,
                   scale=None, out=None):
    """One token of each request through the layer behind its short conv
    (gdn_ssm_conv_step): x [B, 2 Hk dk + Hv dv], the conv's output; a, b [B, Hv],
    the gates' raw projections; A_log, dt_bias [Hv] fp32; z [B, Hv, dv] or None
    (no norm), norm_w [dv].  x, a, b and z may be row-strided views.  q and k are
    normalised; states, src and dst as in gdn_chunk_step.  Returns y [B, Hv, dv]."""
    dev, code = _lead(x, "x")
    e, B, n = x.dtype, x.shape[0], states.shape[0]
    A_log, dt_bias, norm_w = _c(A_log), _c(dt_bias), _c(norm_w)
    y = torch.empty((B, Hv, dv), dtype=e, device=x.device) if out is None else out
    zp, ldz = _heads(z, "z", e, dev, (B, Hv, dv))
    _run(_lib().gdn_layer_step(*_rows(x, "x", e, dev, (B, 2 * Hk * dk + Hv * dv)), *_rows(a, "a", e, dev, (B, Hv)),
                               *_rows(b, "b", e, dev, (B, Hv)), code, _ptr(A_log, "A_log", _F32, dev, (Hv,)),
                               _ptr(dt_bias, "dt_bias", _F32, dev, (Hv,)), zp, ldz,
                               _ptr(norm_w, "norm_w", e, dev, (dv,)), eps, B, Hk, Hv, dk, dv,
                               dk ** -0.5 if scale is None else scale,
                               _dense(states, "states", _F32, dev, (n, Hv, dk, dv)), n,
                               _dense(src, "src", _I32, dev, (B,)), _dense(dst, "dst", _I32, dev, (B,)),
                               _dense(y, "out", e, dev, (B, Hv, dv)), _raw_stream(dev)))
    return y


# ----------------------------------------------------------------------------
# embedding
# ----------------------------------------------------------------------------

def gdn_embed_fwd(tokens, table, scale=1.0, out=None):
    """Rows of table [V, W] (a row-strided view will do) times scale; tokens [T].
    A token outside [0, V) gives a row of zeros.  Returns [T, W]."""
    dev, code = _lead(table, "table")
    e, (V, W), T = table.dtype, table.shape, tokens.shape[0]
    y = torch.empty((T, W), dtype=e, device=table.device) if out is None else out
    _run(_lib().gdn_embed_fwd(*_index(tokens, "tokens", dev), *_rows(table, "table", e, dev, (V, W)), code, V, T, W,
                              scale, *_rows(y, "out", e, dev, (T, W)), _raw_stream(dev)))
    return y


def embed_bwd_workspace_size(T, vocab, width) -> int:
    return int(load().gdn_embed_bwd_workspace_size(T, vocab, width))


def gdn_embed_bwd(dy, tokens, vocab, scale=1.0, into=None, workspace=None):
    """Gradient of gdn_embed_fwd's table for dy [T, W] (a row-strided view will
    do): a token's rows added in fp32 in their order, rounded once.  into [V, W]:
    adds to it (the rows of the tokens alone are touched), as where the output
    weights are the table.  Returns the gradient [V, W], dtype of dy."""
    dev, code = _lead(dy, "dy")
    e, (T, W) = dy.dtype, dy.shape
    lib = _lib()
    ws = _workspace(lib.gdn_embed_bwd_workspace_size(T, vocab, W), workspace, dev)
    tp, bits = _index(tokens, "tokens", dev)
    if tokens.shape[0] != T:
        raise ValueError(f"tokens must have {T} elements, got {tokens.shape[0]}")
    d = torch.empty((vocab, W), dtype=e, device=dy.device) if into is None else into
    _run(lib.gdn_embed_bwd(*_rows(dy, "dy", e, dev, (T, W)), code, tp, bits, vocab, T, W, scale,
                           0 if into is None else 1, *_rows(d, "into", e, dev, (vocab, W)), ws.data_ptr(), ws.numel(),
                           _raw_stream(dev)))
    return d


# ----------------------------------------------------------------------------
# cross entropy over the vocabulary
# ----------------------------------------------------------------------------

def _readable(t):
    """t, or a dense copy where the tensor maps could not read it: rows of whole
    16-byte pieces that do not start at one."""
    if t.dim() == 2 and t.dtype is torch.bfloat16 and t.shape[1] % 8 == 0 and \
            (t.stride(1) != 1 or (t.shape[0] > 1 and t.stride(0) % 8) or t.data_ptr() % 16):
        return t.clone(memory_format=torch.contiguous_format)
    return t


def vocab_loss_fwd_workspace_size(T, vocab, width, dtype) -> int:
    return int(load().gdn_vocab_loss_fwd_workspace_size(T, vocab, width, _CODE[dtype]))


def vocab_loss_bwd_workspace_size(T, vocab, width, dtype) -> int:
    return int(load().gdn_vocab_loss_bwd_workspace_size(T, vocab, width, _CODE[dtype]))


def gdn_vocab_loss_fwd(h, w, targets, scale=1.0, workspace=None):
    """Cross entropy of the logits scale h w^T without the logits: h [T, W], w [V,
    W] (row-strided views will do), targets [T].  A negative target leaves its
    token out (loss 0); one of V or more gives NaN.  Returns (loss [T], lse [T]),
    fp32."""
    dev, code = _lead(h, "h")
    e, (T, W), V = h.dtype, h.shape, w.shape[0]
    h, w = _readable(h), _readable(w)
    lib = _lib()
    ws = _workspace(lib.gdn_vocab_loss_fwd_workspace_size(T, V, W, code), workspace, dev)
    tp, bits = _index(targets, "targets", dev)
    if targets.shape[0] != T:
        raise ValueError(f"targets must have {T} elements, got {targets.shape[0]}")
    loss, lse = torch.empty(T, dtype=_F32, device=h.device), torch.empty(T, dtype=_F32, device=h.device)
    _run(lib.gdn_vocab_loss_fwd(*_rows(h, "h", e, dev, (T, W)), *_rows(w, "w", e, dev, (V, W)), code, tp, bits, T, V, W,
                                scale, loss.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(dev)))
    return loss, lse


def gdn_vocab_loss_bwd(dloss, h, w, targets, lse, scale=1.0, workspace=None, loss=None):
    """Gradients of gdn_vocab_loss_fwd's loss for dloss [T] fp32, with its lse and
    loss.  Without the loss the gradients of tokens that are nearly certain lose
    digits, as far as softmax - 1 does by the rounded lse.  Returns a dict: dh
    [T, W], dw [V, W], in the inputs' dtype."""
    dev, code = _lead(h, "h")
    e, (T, W), V = h.dtype, h.shape, w.shape[0]
    h, w, dloss, lse = _readable(h), _readable(w), _c(dloss), _c(lse)
    lib = _lib()
    ws = _workspace(lib.gdn_vocab_loss_bwd_workspace_size(T, V, W, code), workspace, dev)
    tp, bits = _index(targets, "targets", dev)
    if targets.shape[0] != T:
        raise ValueError(f"targets must have {T} elements, got {targets.shape[0]}")
    call, more = lib.gdn_vocab_loss_bwd, ()
    if loss is not None:
        loss = _c(loss)
        call, more = lib.gdn_vocab_loss_bwd_from_loss, (_ptr(loss, "loss", _F32, dev, (T,)),)
    r = dict(dh=torch.empty((T, W), dtype=e, device=h.device), dw=torch.empty((V, W), dtype=e, device=h.device))
    _run(call(_ptr(dloss, "dloss", _F32, dev, (T,)), *_rows(h, "h", e, dev, (T, W)), *_rows(w, "w", e, dev, (V, W)), code,
              tp, bits, *more, _ptr(lse, "lse", _F32, dev, (T,)), T, V, W, scale, r["dh"].data_ptr(), W,
              r["dw"].data_ptr(), W, ws.data_ptr(), ws.numel(), _raw_stream(dev)))
    return r
