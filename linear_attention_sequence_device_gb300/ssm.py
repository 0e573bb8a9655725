"""Front end of the selective scan layer and the block norm (see gdn_cp.h):
the short causal convolution with a state per sequence, the selective state
space scan and the norms between two blocks, each with its gradient, and the
single-token forms over a cache of states.

Argument marshalling only, on the current stream; wrong arguments raise before
anything is launched.
"""
from __future__ import annotations

import torch

from .binding import _check, _dt, _need, _p, _stream, load


def _same(dt, /, **tensors):
    for name, t in tensors.items():
        _need(t, name, dt)


def _shape(t, name, *dims):
    if t is not None and tuple(t.shape) != dims:
        raise ValueError(f"{name} must have shape {dims}, got {tuple(t.shape)}")


def _rows(t, name):
    """Row stride of a [T, C] view with unit column stride."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a 2-d view with unit column stride")
    # a single row's stride is free: any valid one will do
    return t.stride(0) if t.shape[0] > 1 else (t.shape[1] + 7) // 8 * 8


def _dense(t, name):
    if t is not None and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _c(t):
    return None if t is None else t.contiguous()


def _empty(shape, dtype, dev):
    return torch.empty(shape, dtype=dtype, device=dev)


def _workspace(need, given, dev):
    if given is None:
        return _empty(max(int(need), 256), torch.uint8, dev)
    _need(given, "workspace", torch.uint8)
    return _dense(given, "workspace")


def _slots(src, dst, batch):
    for t, n in ((src, "src"), (dst, "dst")):
        _need(t, n, torch.int32)
        _shape(t, n, batch)
        _dense(t, n)


def _lens(cu_seqlens):
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a vector of num_seqs + 1 offsets")
    return _dense(cu_seqlens, "cu_seqlens").numel() - 1


def _on_one_device(first, *rest):
    for t in rest:
        if t is not None and t.device != first.device:
            raise ValueError(f"tensors on different devices: {first.device} and {t.device}")


# ----------------------------------------------------------------------------
# short convolution
# ----------------------------------------------------------------------------

def gdn_ssm_conv_fwd(x, w, bias, cu_seqlens, state=None, output_state=True, out=None):
    """Causal depthwise conv1d + SiLU over packed sequences; x [T, C] (a
    row-strided view will do), w [C, K], bias [C] or None, state [N, K - 1, C]:
    the rows before each sequence (None: zeros).  Returns (y [T, C], the state
    after each sequence or None)."""
    dt = x.dtype
    _same(dt, x=x, w=w, bias=bias, state=state, out=out)
    n = _lens(cu_seqlens)
    T, C = x.shape
    K = w.shape[1]
    _shape(w, "w", C, K)
    _shape(bias, "bias", C)
    _shape(state, "state", n, K - 1, C)
    _shape(out, "out", T, C)
    _on_one_device(x, w, bias, cu_seqlens, state, out)
    y = _empty((T, C), dt, x.device) if out is None else out
    st = _empty((n, K - 1, C), dt, x.device) if output_state else None
    w, bias, state = w.contiguous(), _c(bias), _c(state)
    _check(load().gdn_ssm_conv_fwd(_p(x), _rows(x, "x"), _dt(x), T, C, _p(w), _p(bias), K, _p(cu_seqlens), n,
                                   _p(state), _p(st), _p(y), _rows(y, "out"), _stream()))
    return y, st


def gdn_ssm_conv_bwd(dy, x, w, bias, cu_seqlens, state=None, dstate_out=None, workspace=None):
    """Gradients of gdn_ssm_conv_fwd for dy [T, C] and dstate_out [N, K - 1, C]
    fp32 (None: zero).  Returns a dict: dx [T, C] (dtype of x), dw [C, K], dbias
    [C] (None without bias), dstate [N, K - 1, C], the last three fp32."""
    dt = x.dtype
    _same(dt, dy=dy, x=x, w=w, bias=bias, state=state)
    _need(dstate_out, "dstate_out", torch.float32)
    n = _lens(cu_seqlens)
    T, C = x.shape
    K = w.shape[1]
    _shape(dy, "dy", T, C)
    _shape(w, "w", C, K)
    _shape(bias, "bias", C)
    _shape(state, "state", n, K - 1, C)
    _shape(dstate_out, "dstate_out", n, K - 1, C)
    _on_one_device(x, dy, w, bias, cu_seqlens, state, dstate_out, workspace)
    dev, f32 = x.device, torch.float32
    lib = load()
    ws = _workspace(lib.gdn_ssm_conv_bwd_workspace_size(T, C, K), workspace, dev)
    r = dict(dx=_empty((T, C), dt, dev), dw=_empty((C, K), f32, dev),
             dbias=None if bias is None else _empty((C,), f32, dev), dstate=_empty((n, K - 1, C), f32, dev))
    w, bias, state, dstate_out = w.contiguous(), _c(bias), _c(state), _c(dstate_out)
    _check(lib.gdn_ssm_conv_bwd(_p(dy), _rows(dy, "dy"), _p(x), _rows(x, "x"), _dt(x), T, C, _p(w), _p(bias), K,
                                _p(cu_seqlens), n, _p(state), _p(dstate_out), _p(r["dx"]), _rows(r["dx"], "dx"),
                                _p(r["dw"]), _p(r["dbias"]), _p(r["dstate"]), _p(ws), ws.numel(), _stream()))
    return r


def gdn_ssm_conv_step(x, w, bias, states, src=None, dst=None, out=None):
    """One token of each request: x [B, C]; states [slots, K - 1, C], updated in
    place; src, dst int32 [B]: the slot that request i reads and the one it
    writes (None: slot i; src < 0: a zero state; dst < 0: a padded row).
    Returns y [B, C]."""
    dt = x.dtype
    _same(dt, x=x, w=w, bias=bias, states=states, out=out)
    Bt, C = x.shape
    K = w.shape[1]
    _shape(w, "w", C, K)
    _shape(bias, "bias", C)
    _shape(states, "states", states.shape[0], K - 1, C)
    _shape(out, "out", Bt, C)
    _slots(src, dst, Bt)
    _on_one_device(x, w, bias, states, src, dst, out)
    _dense(states, "states")
    y = _empty((Bt, C), dt, x.device) if out is None else out
    w, bias = w.contiguous(), _c(bias)
    _check(load().gdn_ssm_conv_step(_p(x), _rows(x, "x"), _dt(x), Bt, C, _p(w), _p(bias), K, _p(states),
                                    states.shape[0], _p(src), _p(dst), _p(y), _rows(y, "out"), _stream()))
    return y


# ----------------------------------------------------------------------------
# selective scan
# ----------------------------------------------------------------------------

def _bc(t, name, T, G, N):
    """Row stride of B or C, a [T, G, N] view whose (G, N) part is dense."""
    _shape(t, name, T, G, N)
    if (N > 1 and t.stride(2) != 1) or (G > 1 and t.stride(1) != N):
        raise ValueError(f"{name} must be a [T, groups, N] view with a dense (groups, N) part")
    return t.stride(0) if T > 1 else G * N


def _scan_args(x, dt, A_log, B, C, D, z, dt_bias):
    e = x.dtype
    _same(e, x=x, dt=dt, B=B, C=C, z=z)
    _same(torch.float32, A_log=A_log, D=D, dt_bias=dt_bias)
    T, ch = x.shape
    if B.dim() != 3 or A_log.dim() != 2:
        raise ValueError("B must be [T, groups, N] and A_log [channels, N]")
    G, N = B.shape[1], A_log.shape[1]
    _shape(dt, "dt", T, ch)
    _shape(z, "z", T, ch)
    _shape(A_log, "A_log", ch, N)
    _shape(D, "D", ch)
    _shape(dt_bias, "dt_bias", ch)
    ldb, ldc = _bc(B, "B", T, G, N), _bc(C, "C", T, G, N)
    _on_one_device(x, dt, A_log, B, C, D, z, dt_bias)
    lead = (_p(x), _rows(x, "x"), _p(dt), _rows(dt, "dt"), _p(z), 0 if z is None else _rows(z, "z"), _p(B), ldb,
            _p(C), ldc, _dt(x))
    return T, ch, G, N, lead


def ssm_scan_ckpt_shape(T, channels, d_state):
    """Shape of the forward's checkpoints: the states before every 8th token."""
    return ((T + 7) // 8, channels, d_state)


def ssm_scan_workspace_size(T, channels, d_state, groups=1) -> int:
    return int(load().gdn_ssm_scan_workspace_size(T, channels, d_state, groups))


def ssm_scan_bwd_workspace_size(T, channels, d_state, groups=1) -> int:
    return int(load().gdn_ssm_scan_bwd_workspace_size(T, channels, d_state, groups))


def gdn_ssm_scan_fwd(x, dt, A_log, B, C, cu_seqlens, D=None, z=None, dt_bias=None, h0=None, output_final_state=True,
                     checkpoints=False, out=None, workspace=None):
    """Selective state space scan over packed sequences.  x, dt, z [T, Ch]
    (row-strided views will do), B, C [T, G, N] (token stride free), A_log [Ch,
    N], D, dt_bias [Ch], h0 [num_seqs, Ch, N], the last four fp32.  Returns (y
    [T, Ch], h_final [num_seqs, Ch, N] or None, checkpoints for
    gdn_ssm_scan_bwd or None)."""
    T, ch, G, N, lead = _scan_args(x, dt, A_log, B, C, D, z, dt_bias)
    n = _lens(cu_seqlens)
    _need(h0, "h0", torch.float32)
    _shape(h0, "h0", n, ch, N)
    _same(x.dtype, out=out)
    _shape(out, "out", T, ch)
    _on_one_device(x, cu_seqlens, h0, out, workspace)
    dev, f32 = x.device, torch.float32
    y = _empty((T, ch), x.dtype, dev) if out is None else out
    hf = _empty((n, ch, N), f32, dev) if output_final_state else None
    ck = _empty(ssm_scan_ckpt_shape(T, ch, N), f32, dev) if checkpoints else None
    ws = _workspace(ssm_scan_workspace_size(T, ch, N, G), workspace, dev)
    A_log, D, dt_bias, h0 = A_log.contiguous(), _c(D), _c(dt_bias), _c(h0)
    _check(load().gdn_ssm_scan_fwd(*lead, _p(A_log), _p(D), _p(dt_bias), _p(h0), _p(cu_seqlens), n, T, ch, N, G, _p(y),
                                   _rows(y, "out"), _p(hf), _p(ck), _p(ws), ws.numel(), _stream()))
    return y, hf, ck


def gdn_ssm_scan_bwd(dy, x, dt, A_log, B, C, cu_seqlens, ckpt, D=None, z=None, dt_bias=None, h0=None, dh_final=None,
                     workspace=None):
    """Gradients of gdn_ssm_scan_fwd for dy [T, Ch] and dh_final [num_seqs, Ch,
    N] fp32 (None: zero), with the forward's inputs and checkpoints.  Returns a
    dict: dx, ddt, dz [T, Ch], dB, dC [T, G, N] in the inputs' dtype; dA_log
    [Ch, N], dD, ddt_bias [Ch], dh0 [num_seqs, Ch, N] fp32; dz, dD and ddt_bias
    None where the input is."""
    T, ch, G, N, lead = _scan_args(x, dt, A_log, B, C, D, z, dt_bias)
    n = _lens(cu_seqlens)
    _same(x.dtype, dy=dy)
    _same(torch.float32, ckpt=ckpt, h0=h0, dh_final=dh_final)
    _shape(dy, "dy", T, ch)
    _shape(ckpt, "ckpt", *ssm_scan_ckpt_shape(T, ch, N))
    _shape(h0, "h0", n, ch, N)
    _shape(dh_final, "dh_final", n, ch, N)
    _dense(ckpt, "ckpt")
    _on_one_device(x, dy, cu_seqlens, ckpt, h0, dh_final, workspace)
    e, dev, f32 = x.dtype, x.device, torch.float32
    r = dict(dx=_empty((T, ch), e, dev), ddt=_empty((T, ch), e, dev), dz=None if z is None else _empty((T, ch), e, dev),
             dA_log=_empty((ch, N), f32, dev), dB=_empty((T, G, N), e, dev), dC=_empty((T, G, N), e, dev),
             dD=None if D is None else _empty((ch,), f32, dev),
             ddt_bias=None if dt_bias is None else _empty((ch,), f32, dev), dh0=_empty((n, ch, N), f32, dev))
    ws = _workspace(ssm_scan_bwd_workspace_size(T, ch, N, G), workspace, dev)
    A_log, D, dt_bias, h0, dh_final = A_log.contiguous(), _c(D), _c(dt_bias), _c(h0), _c(dh_final)
    _check(load().gdn_ssm_scan_bwd(_p(dy), _rows(dy, "dy"), *lead, _p(A_log), _p(D), _p(dt_bias), _p(h0), _p(ckpt),
                                   _p(dh_final), _p(cu_seqlens), n, T, ch, N, G,
                                   *(_p(r[k]) for k in ("dx", "ddt", "dz", "dB", "dC", "dA_log", "dD", "ddt_bias",
                                                        "dh0")), _p(ws), ws.numel(), _stream()))
    return r


def gdn_ssm_scan_step(x, dt, A_log, B, C, states, D=None, z=None, dt_bias=None, src=None, dst=None, out=None):
    """One token of each request: x, dt, z [Bt, Ch], B, C [Bt, G, N]; states
    [slots, Ch, N] fp32, updated in place; src, dst as in gdn_ssm_conv_step.
    Returns y [Bt, Ch]."""
    Bt, ch, G, N, lead = _scan_args(x, dt, A_log, B, C, D, z, dt_bias)
    _need(states, "states", torch.float32)
    _shape(states, "states", states.shape[0], ch, N)
    _dense(states, "states")
    _same(x.dtype, out=out)
    _shape(out, "out", Bt, ch)
    _slots(src, dst, Bt)
    _on_one_device(x, states, src, dst, out)
    y = _empty((Bt, ch), x.dtype, x.device) if out is None else out
    A_log, D, dt_bias = A_log.contiguous(), _c(D), _c(dt_bias)
    _check(load().gdn_ssm_scan_step(*lead, _p(A_log), _p(D), _p(dt_bias), Bt, ch, N, G, _p(states), states.shape[0],
                                    _p(src), _p(dst), _p(y), _rows(y, "out"), _stream()))
    return y


# ----------------------------------------------------------------------------
# block norm
# ----------------------------------------------------------------------------

def _norm_args(o, res, w_pre, w_post, gate, scale, res_name):
    _same(o.dtype, o=o, w_pre=w_pre, w_post=w_post, gate=gate)
    _need(res, res_name)
    _need(scale, "scale", torch.float32)
    if res.dtype not in (torch.float32, o.dtype):
        raise TypeError(f"{res_name} must be float32 or {o.dtype}, got {res.dtype}")
    T, W = o.shape
    _shape(res, res_name, T, W)
    _shape(gate, "gate", T, W)
    for t, n in ((w_pre, "w_pre"), (w_post, "w_post"), (scale, "scale")):
        _shape(t, n, W)
    _on_one_device(o, res, w_pre, w_post, gate, scale)
    _dense(res, res_name)
    return T, W


def gdn_block_norm_fwd(o, res, w_pre, w_post=None, gate=None, scale=None, eps=1e-6, res_out=None, out=None):
    """Between two blocks: res_out = res + scale * sigmoid(gate) * rmsnorm(o) *
    w_post, y = rmsnorm(res_out) * w_pre.  o, gate [T, W] (row-strided views
    will do), res [T, W] in fp32 or o's dtype, weights [W], scale [W] fp32; a
    missing w_post leaves o as it is, a missing gate or scale is 1.  res_out may
    be res.  Returns (y, res_out)."""
    T, W = _norm_args(o, res, w_pre, w_post, gate, scale, "res")
    _same(o.dtype, out=out)
    _same(res.dtype, res_out=res_out)
    _shape(out, "out", T, W)
    _shape(res_out, "res_out", T, W)
    _on_one_device(o, out, res_out)
    y = torch.empty((T, W), dtype=o.dtype, device=o.device) if out is None else _dense(out, "out")
    r = torch.empty_like(res) if res_out is None else _dense(res_out, "res_out")
    w_pre, w_post, scale = w_pre.contiguous(), _c(w_post), _c(scale)
    _check(load().gdn_block_norm_fwd(_p(o), _rows(o, "o"), _p(gate), 0 if gate is None else _rows(gate, "gate"), _dt(o),
                                     _p(res), _dt(res), _p(w_post), _p(w_pre), _p(scale), float(eps), T, W, _p(r),
                                     _p(y), _stream()))
    return y, r


def gdn_block_norm_bwd(dy, dres_out, o, res_out, w_pre, w_post=None, gate=None, scale=None, eps=1e-6, workspace=None):
    """Gradients of gdn_block_norm_fwd for dy [T, W] and dres_out [T, W] (None:
    zero), at the stored res_out.  Returns a dict: do, dgate [T, W] (dtype of
    o), dres [T, W] (dtype of res_out), dw_pre, dw_post, dscale [W] fp32; dgate,
    dw_post and dscale None where the input is."""
    T, W = _norm_args(o, res_out, w_pre, w_post, gate, scale, "res_out")
    _same(o.dtype, dy=dy)
    _same(res_out.dtype, dres_out=dres_out)
    _shape(dy, "dy", T, W)
    _shape(dres_out, "dres_out", T, W)
    _on_one_device(o, dy, dres_out, workspace)
    e, dev, f32 = o.dtype, o.device, torch.float32
    lib = load()
    ws = _workspace(lib.gdn_block_norm_bwd_workspace_size(T, W), workspace, dev)
    r = dict(do=_empty((T, W), e, dev), dres=_empty((T, W), res_out.dtype, dev),
             dgate=None if gate is None else _empty((T, W), e, dev), dw_pre=_empty((W,), f32, dev),
             dw_post=None if w_post is None else _empty((W,), f32, dev),
             dscale=None if scale is None else _empty((W,), f32, dev))
    dy, dres_out, w_pre, w_post, scale = dy.contiguous(), _c(dres_out), w_pre.contiguous(), _c(w_post), _c(scale)
    _check(lib.gdn_block_norm_bwd(_p(dy), _p(dres_out), _p(o), _rows(o, "o"), _p(gate),
                                  0 if gate is None else _rows(gate, "gate"), _dt(o), _p(res_out), _dt(res_out),
                                  _p(w_post), _p(w_pre), _p(scale), float(eps), T, W, _p(r["do"]), _p(r["dgate"]),
                                  _p(r["dres"]), _p(r["dw_pre"]), _p(r["dw_post"]), _p(r["dscale"]), _p(ws),
                                  ws.numel(), _stream()))
    return r
