"""Front end of the selective scan layer and the block norm (see gdn_cp.h):
the short causal convolution with a state per sequence, the selective state
space scan and the norms between two blocks, each with its gradient, and the
single-token forms over a cache of states.

Argument marshalling only, on the current stream of the current device, which has
to be the tensors'; wrong arguments raise before anything is launched.  Results have
no autograd history: gradients are calls of their own, from which
examples/hybrid_lm.py makes autograd functions.  A single-token call's kernel takes a few microseconds, so
the checks look at each tensor once and hand plain integers to the library, and
results are made like an input (2.4 us between two launches; from a shape, a type
and a device 4.8).  Rows with a stride of their own give dense results: an array
like a view with gaps has none.
"""
from __future__ import annotations

import torch

from . import binding
from .binding import GDN_BF16, GDN_F32, GdnError, load

_F32, _I32, _U8 = torch.float32, torch.int32, torch.uint8
_CODE = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _lib():
    return binding._lib or load()


def _run(status):
    if status:
        raise GdnError(status, load().gdn_last_error().decode())


def _lead(t, name):
    """Device and dtype code of the tensor that the others have to match.  The
    library launches on the current device, whatever the stream."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != binding._current_device():
        raise ValueError(f"{name} is on CUDA device {dev}, which is not the current device "
                         f"({binding._current_device()}): make the call under torch.cuda.device({dev})")
    code = _CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return dev, code


def _wrong(t, name, dtype, dev, shape):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on CUDA device {dev}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _ptr(t, name, dtype, dev, shape):
    """Address of t (None: none), after its dtype, device and shape."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        _wrong(t, name, dtype, dev, shape)
    return t.data_ptr()


def _dense(t, name, dtype, dev, shape):
    """The same for an array that is read or written in place, which has to be contiguous."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        _wrong(t, name, dtype, dev, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name, dtype, dev, shape):
    """Address and row stride of a [T, C] view with unit column stride (None: none)."""
    if t is None:
        return None, 0
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        _wrong(t, name, dtype, dev, shape)
    s0, s1 = t.stride()
    if s1 != 1 and shape[1] > 1:
        raise ValueError(f"{name} must be a 2-d view with unit column stride")
    # a single row's stride is free: any valid one will do
    return t.data_ptr(), s0 if shape[0] > 1 else (shape[1] + 7) // 8 * 8


def _c(t):
    return t if t is None or t.is_contiguous() else t.contiguous()


def _new_like(t, shape, dtype, dev):
    """A new array, after t where it is given (whose shape and type are checked before the launch)."""
    return torch.empty(shape, dtype=dtype, device=dev) if t is None else torch.empty_like(t)


def _f32_like(t):
    """A new fp32 array of the shape of a contiguous t (None: none)."""
    return t if t is None else torch.empty_like(t) if t.dtype is _F32 else torch.empty_like(t, dtype=_F32)


def _lens(cu, dev):
    """Address of cu_seqlens and the number of sequences."""
    if cu.dim() != 1 or cu.shape[0] < 2:
        raise ValueError("cu_seqlens must be a vector of num_seqs + 1 offsets")
    return _dense(cu, "cu_seqlens", _I32, dev, cu.shape), cu.shape[0] - 1


def _workspace(need, given, dev):
    if given is None:
        return torch.empty(max(int(need), 256), dtype=_U8, device=dev)
    _dense(given, "workspace", _U8, dev, given.shape)
    return given


# ----------------------------------------------------------------------------
# short convolution
# ----------------------------------------------------------------------------

def gdn_ssm_conv_fwd(x, w, bias, cu_seqlens, state=None, output_state=True, out=None):
    """Causal depthwise conv1d + SiLU over packed sequences; x [T, C] (a
    row-strided view will do), w [C, K], bias [C] or None, state [N, K - 1, C]:
    the rows before each sequence (None: zeros).  out must not overlap x.
    Returns (y [T, C], the state after each sequence or None)."""
    dev, code = _lead(x, "x")
    dt, (T, C), K = x.dtype, x.shape, w.shape[-1]
    w, bias, state = _c(w), _c(bias), _c(state)
    cu, n = _lens(cu_seqlens, dev)
    y = torch.empty_like(x) if out is None else out
    st = _new_like(state, (n, K - 1, C), dt, dev) if output_state else None
    _run(_lib().gdn_ssm_conv_fwd(*_rows(x, "x", dt, dev, (T, C)), code, T, C, _ptr(w, "w", dt, dev, (C, K)),
                                 _ptr(bias, "bias", dt, dev, (C,)), K, cu, n,
                                 _ptr(state, "state", dt, dev, (n, K - 1, C)), None if st is None else st.data_ptr(),
                                 *_rows(y, "out", dt, dev, (T, C)), _raw_stream(dev)))
    return y, st


def gdn_ssm_conv_bwd(dy, x, w, bias, cu_seqlens, state=None, dstate_out=None, workspace=None):
    """Gradients of gdn_ssm_conv_fwd for dy [T, C] and dstate_out [N, K - 1, C]
    fp32 (None: zero).  Returns a dict: dx [T, C] (dtype of x), dw [C, K], dbias
    [C] (None without bias), dstate [N, K - 1, C], the last three fp32."""
    dev, code = _lead(x, "x")
    dt, (T, C), K = x.dtype, x.shape, w.shape[-1]
    w, bias, state, dstate_out = _c(w), _c(bias), _c(state), _c(dstate_out)
    cu, n = _lens(cu_seqlens, dev)
    lib = _lib()
    ws = _workspace(lib.gdn_ssm_conv_bwd_workspace_size(T, C, K), workspace, dev)
    r = dict(dx=torch.empty_like(x), dw=_f32_like(w), dbias=_f32_like(bias),
             dstate=_new_like(dstate_out, (n, K - 1, C), _F32, dev))
    _run(lib.gdn_ssm_conv_bwd(*_rows(dy, "dy", dt, dev, (T, C)), *_rows(x, "x", dt, dev, (T, C)), code, T, C,
                              _ptr(w, "w", dt, dev, (C, K)), _ptr(bias, "bias", dt, dev, (C,)), K, cu, n,
                              _ptr(state, "state", dt, dev, (n, K - 1, C)),
                              _ptr(dstate_out, "dstate_out", _F32, dev, (n, K - 1, C)),
                              *_rows(r["dx"], "dx", dt, dev, (T, C)), r["dw"].data_ptr(),
                              None if bias is None else r["dbias"].data_ptr(),
                              r["dstate"].data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(dev)))
    return r


def gdn_ssm_conv_step(x, w, bias, states, src=None, dst=None, out=None):
    """One token of each request: x [B, C]; states [slots, K - 1, C], updated in
    place; src, dst int32 [B]: the slot that request i reads and the one it
    writes (None: slot i; src < 0: a zero state; dst < 0: a padded row).
    Returns y [B, C]."""
    dev, code = _lead(x, "x")
    dt, (B, C), K, n = x.dtype, x.shape, w.shape[-1], states.shape[0]
    w, bias = _c(w), _c(bias)
    y = torch.empty_like(x) if out is None else out
    _run(_lib().gdn_ssm_conv_step(*_rows(x, "x", dt, dev, (B, C)), code, B, C, _ptr(w, "w", dt, dev, (C, K)),
                                  _ptr(bias, "bias", dt, dev, (C,)), K,
                                  _dense(states, "states", dt, dev, (n, K - 1, C)), n,
                                  _dense(src, "src", _I32, dev, (B,)), _dense(dst, "dst", _I32, dev, (B,)),
                                  *_rows(y, "out", dt, dev, (B, C)), _raw_stream(dev)))
    return y


# ----------------------------------------------------------------------------
# selective scan
# ----------------------------------------------------------------------------

def _scan_args(x, dt, A_log, B, C, D, z, dt_bias):
    """Sizes, device, the leading arguments of the scan's entry points and A_log, D, dt_bias."""
    dev, code = _lead(x, "x")
    e, (T, ch) = x.dtype, x.shape
    if B.dim() != 3 or A_log.dim() != 2:
        raise ValueError("B must be [T, groups, N] and A_log [channels, N]")
    G, N = B.shape[1], A_log.shape[1]
    ld = []
    for t, name in ((B, "B"), (C, "C")):
        s = t.stride()
        if (s[-1] != 1 and N > 1) or (G > 1 and s[-2] != N):
            raise ValueError(f"{name} must be a [T, groups, N] view with a dense (groups, N) part")
        ld.append(s[0] if T > 1 else G * N)
    tc, tgn = (T, ch), (T, G, N)
    lead = (*_rows(x, "x", e, dev, tc), *_rows(dt, "dt", e, dev, tc), *_rows(z, "z", e, dev, tc),
            _ptr(B, "B", e, dev, tgn), ld[0], _ptr(C, "C", e, dev, tgn), ld[1], code)
    par = [_c(A_log), _c(D), _c(dt_bias)]  # kept by the caller until its launch
    pp = (_ptr(par[0], "A_log", _F32, dev, (ch, N)), _ptr(par[1], "D", _F32, dev, (ch,)),
          _ptr(par[2], "dt_bias", _F32, dev, (ch,)))
    return T, ch, G, N, dev, lead, pp, par


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
    T, ch, G, N, dev, lead, pp, keep = _scan_args(x, dt, A_log, B, C, D, z, dt_bias)
    cu, n = _lens(cu_seqlens, dev)
    h0 = _c(h0)
    lib = _lib()
    y = torch.empty_like(x) if out is None else out
    hf = _new_like(h0, (n, ch, N), _F32, dev) if output_final_state else None
    ck = torch.empty(ssm_scan_ckpt_shape(T, ch, N), dtype=_F32, device=dev) if checkpoints else None
    ws = _workspace(lib.gdn_ssm_scan_workspace_size(T, ch, N, G), workspace, dev)
    _run(lib.gdn_ssm_scan_fwd(*lead, *pp, _ptr(h0, "h0", _F32, dev, (n, ch, N)), cu, n, T, ch, N, G,
                              *_rows(y, "out", x.dtype, dev, (T, ch)),
                              None if hf is None else hf.data_ptr(), None if ck is None else ck.data_ptr(),
                              ws.data_ptr(), ws.numel(), _raw_stream(dev)))
    return y, hf, ck


def gdn_ssm_scan_bwd(dy, x, dt, A_log, B, C, cu_seqlens, ckpt, D=None, z=None, dt_bias=None, h0=None, dh_final=None,
                     workspace=None):
    """Gradients of gdn_ssm_scan_fwd for dy [T, Ch] and dh_final [num_seqs, Ch,
    N] fp32 (None: zero), with the forward's inputs and checkpoints.  Returns a
    dict: dx, ddt, dz [T, Ch], dB, dC [T, G, N] in the inputs' dtype; dA_log
    [Ch, N], dD, ddt_bias [Ch], dh0 [num_seqs, Ch, N] fp32; dz, dD and ddt_bias
    None where the input is."""
    T, ch, G, N, dev, lead, pp, keep = _scan_args(x, dt, A_log, B, C, D, z, dt_bias)
    cu, n = _lens(cu_seqlens, dev)
    h0, dh_final = _c(h0), _c(dh_final)
    lib = _lib()
    e = x.dtype
    r = dict(dx=torch.empty_like(x), ddt=torch.empty_like(x), dz=None if z is None else torch.empty_like(x),
             dB=torch.empty_like(B, memory_format=torch.contiguous_format),
             dC=torch.empty_like(C, memory_format=torch.contiguous_format), dA_log=_f32_like(keep[0]),
             dD=_f32_like(keep[1]), ddt_bias=_f32_like(keep[2]), dh0=_new_like(h0, (n, ch, N), _F32, dev))
    ws = _workspace(lib.gdn_ssm_scan_bwd_workspace_size(T, ch, N, G), workspace, dev)
    _run(lib.gdn_ssm_scan_bwd(*_rows(dy, "dy", e, dev, (T, ch)), *lead, *pp,
                              _ptr(h0, "h0", _F32, dev, (n, ch, N)),
                              _dense(ckpt, "ckpt", _F32, dev, ssm_scan_ckpt_shape(T, ch, N)),
                              _ptr(dh_final, "dh_final", _F32, dev, (n, ch, N)), cu, n, T, ch, N, G,
                              *(None if t is None else t.data_ptr() for t in r.values()), ws.data_ptr(), ws.numel(),
                              _raw_stream(dev)))
    return r


def gdn_ssm_scan_step(x, dt, A_log, B, C, states, D=None, z=None, dt_bias=None, src=None, dst=None, out=None):
    """One token of each request: x, dt, z [Bt, Ch], B, C [Bt, G, N]; states
    [slots, Ch, N] fp32, updated in place; src, dst as in gdn_ssm_conv_step.
    Returns y [Bt, Ch]."""
    Bt, ch, G, N, dev, lead, pp, keep = _scan_args(x, dt, A_log, B, C, D, z, dt_bias)
    n = states.shape[0]
    y = torch.empty_like(x) if out is None else out
    _run(_lib().gdn_ssm_scan_step(*lead, *pp, Bt, ch, N, G, _dense(states, "states", _F32, dev, (n, ch, N)), n,
                                  _dense(src, "src", _I32, dev, (Bt,)), _dense(dst, "dst", _I32, dev, (Bt,)),
                                  *_rows(y, "out", x.dtype, dev, (Bt, ch)), _raw_stream(dev)))
    return y


# ----------------------------------------------------------------------------
# block norm
# ----------------------------------------------------------------------------

def gdn_block_norm_fwd(o, res, w_pre, w_post=None, gate=None, scale=None, eps=1e-6, res_out=None, out=None):
    """Between two blocks: res_out = res + scale * sigmoid(gate) * rmsnorm(o) *
    w_post, y = rmsnorm(res_out) * w_pre.  o, gate [T, W] (row-strided views
    will do), res [T, W] in fp32 or o's dtype, weights [W], scale [W] fp32; a
    missing w_post leaves o as it is, a missing gate or scale is 1.  res_out may
    be res.  Returns (y, res_out)."""
    dev, code = _lead(o, "o")
    e, rt, TW = o.dtype, res.dtype, o.shape
    if rt is not e and rt is not _F32:
        raise TypeError(f"res must be float32 or {e}, got {rt}")
    T, W = TW
    w_pre, w_post, scale = _c(w_pre), _c(w_post), _c(scale)
    y = torch.empty_like(o) if out is None else out
    r = torch.empty_like(res) if res_out is None else res_out
    _run(_lib().gdn_block_norm_fwd(*_rows(o, "o", e, dev, TW), *_rows(gate, "gate", e, dev, TW), code,
                                   _dense(res, "res", rt, dev, TW), _CODE[rt],
                                   _ptr(w_post, "w_post", e, dev, (W,)), _ptr(w_pre, "w_pre", e, dev, (W,)),
                                   _ptr(scale, "scale", _F32, dev, (W,)), eps, T, W,
                                   _dense(r, "res_out", rt, dev, TW), _dense(y, "out", e, dev, TW), _raw_stream(dev)))
    return y, r


def gdn_block_norm_bwd(dy, dres_out, o, res_out, w_pre, w_post=None, gate=None, scale=None, eps=1e-6, workspace=None):
    """Gradients of gdn_block_norm_fwd for dy [T, W] and dres_out [T, W] (None:
    zero), at the stored res_out.  Returns a dict: do, dgate [T, W] (dtype of
    o), dres [T, W] (dtype of res_out), dw_pre, dw_post, dscale [W] fp32; dgate,
    dw_post and dscale None where the input is."""
    dev, code = _lead(o, "o")
    e, rt, TW = o.dtype, res_out.dtype, o.shape
    if rt is not e and rt is not _F32:
        raise TypeError(f"res_out must be float32 or {e}, got {rt}")
    T, W = TW
    dy, dres_out, w_pre, w_post, scale = _c(dy), _c(dres_out), _c(w_pre), _c(w_post), _c(scale)
    lib = _lib()
    ws = _workspace(lib.gdn_block_norm_bwd_workspace_size(T, W), workspace, dev)
    r = dict(do=torch.empty_like(o), dgate=None if gate is None else torch.empty_like(o),
             dres=torch.empty_like(res_out), dw_pre=_f32_like(w_pre), dw_post=_f32_like(w_post), dscale=_f32_like(scale))
    _run(lib.gdn_block_norm_bwd(_ptr(dy, "dy", e, dev, TW), _ptr(dres_out, "dres_out", rt, dev, TW),
                                *_rows(o, "o", e, dev, TW), *_rows(gate, "gate", e, dev, TW), code,
                                _dense(res_out, "res_out", rt, dev, TW), _CODE[rt],
                                _ptr(w_post, "w_post", e, dev, (W,)), _ptr(w_pre, "w_pre", e, dev, (W,)),
                                _ptr(scale, "scale", _F32, dev, (W,)), eps, T, W,
                                *(None if t is None else t.data_ptr() for t in r.values()), ws.data_ptr(), ws.numel(),
                                _raw_stream(dev)))
    return r
