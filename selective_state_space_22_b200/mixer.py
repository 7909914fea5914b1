"""The rest of a mixer block around its matrix products: the short causal
convolution and the gated Mamba-1 scan on packed prompts and on single tokens,
their gradients, and the norms before and after the block.

The functions have the C entry points' names (``include/ssd.h`` says what each
argument means) and marshal arguments like the rest of the package.  Inputs that a
projection's output holds side by side may be passed as slices: rows may be
strided, the last dimension may not.  Outputs and scratch are allocated for each
call on the stream that the call runs on, so calls on several streams and captured
graphs never share scratch.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

_VP, _I, _LL, _SZ, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t, ctypes.c_float
_IO = {torch.float32: 0, torch.bfloat16: 1}
_f32 = torch.float32


class _SelArgs(ctypes.Structure):
    _fields_ = ([(k, _VP) for k in ("x", "dt", "z", "B", "C", "A", "D", "dt_bias")]
                + [(k, _LL) for k in ("x_stride", "dt_stride", "z_stride", "b_stride", "c_stride")]
                + [(k, _I) for k in ("io_dtype", "softplus", "channels", "ngroups", "dstate")])


def declare_mixer(lib):
    def sig(name, *args, res=_I):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, res

    sel = ctypes.POINTER(_SelArgs)
    sig("ssd_conv1d_varlen", _VP, _LL, *[_VP] * 9, *[_I] * 8, _VP)
    sig("ssd_conv1d_update", _VP, _VP, _VP, _LL, *[_VP] * 5, *[_I] * 7, _VP)
    sig("ssd_conv1d_bwd_workspace_size", _I, _I, _I, res=_SZ)
    sig("ssd_conv1d_bwd", _VP, _LL, *[_VP] * 9, *[_I] * 7, _VP, _SZ, _VP)
    sig("ssd_selective_scan_chunk_states", _I, _I, res=_SZ)
    sig("ssd_selective_scan_workspace_size", *[_I] * 4, res=_SZ)
    sig("ssd_selective_scan_varlen", sel, *[_VP] * 6, _I, _I, _I, _VP, _SZ, _VP)
    sig("ssd_selective_state_update", sel, _VP, _VP, _VP, _I, _I, _VP)
    sig("ssd_selective_scan_bwd_workspace_size", *[_I] * 5, res=_SZ)
    sig("ssd_selective_scan_bwd", sel, *[_VP] * 11, _I, _I, _VP, _SZ, _VP)
    sig("ssd_residual_rmsnorm", _VP, _LL, _VP, _LL, *[_VP] * 4, *[_I] * 4, _F, _VP)
    sig("ssd_gated_rmsnorm", _VP, _LL, _VP, _LL, _VP, _LL, *[_VP] * 3, *[_I] * 5, _F, _VP)
    sig("ssd_rmsnorm_bwd_workspace_size", _I, _I, res=_SZ)
    sig("ssd_residual_rmsnorm_bwd", _VP, _LL, *[_VP] * 4, _LL, *[_VP] * 5, *[_I] * 4, _F, _VP, _SZ, _VP)
    sig("ssd_gated_rmsnorm_bwd", _VP, _LL, _VP, _LL, *[_VP] * 7, *[_I] * 5, _F, _VP, _SZ, _VP)


_same = contextlib.nullcontext()
_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream  # without the lazy-init wrappers
_empty = torch.empty
_calls = {}


def _call(name):
    """The C function, and the function that turns its status into an exception."""
    f = _calls.get(name)
    if f is None:
        from . import _check, load_library
        f = _calls[name] = (getattr(load_library(), name), _check)
    return f


def _on(dev, stream):
    """Makes the call's device and stream current where they are not."""
    if stream is not None:
        return torch.cuda.stream(stream)
    return _same if _device() == dev.index else torch.cuda.device(dev)


def _device_of(t, name):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _io_of(t, name):
    io = _IO.get(t.dtype)
    if io is None:
        raise ValueError(f"{name} must be bfloat16 or float32")
    return io


def _whole(t, name, dtype, dev, shape):
    """Data pointer of a contiguous tensor."""
    if t is None or t.dtype != dtype or t.device != dev or t.shape != shape or not t.is_contiguous():
        _explain(t, name, dtype, dev, shape)
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _maybe(t, name, dtype, dev, shape):
    return None if t is None else _whole(t, name, dtype, dev, shape)


def _explain(t, name, dtype, dev, shape):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _rows(t, name, dtype, dev, shape):
    """(data pointer, row stride) of rows whose inner dimensions are contiguous."""
    if t is None or t.dtype != dtype or t.device != dev or t.shape != shape:
        _explain(t, name, dtype, dev, shape)
    width = shape[1] if len(shape) == 2 else shape[1] * shape[2]
    if t.is_contiguous():
        return t.data_ptr(), width
    step = t.stride()
    inner = step[-1] == 1 or shape[-1] == 1
    if len(shape) == 3:
        inner &= step[1] == shape[2] or shape[1] == 1
    if not inner or (shape[0] > 1 and step[0] < width):
        raise ValueError(f"{name}: the dimensions after the first must be contiguous and rows must not overlap")
    return t.data_ptr(), max(step[0], width)


def _need_dim(t, name, n):
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, got {t.dim()}")


def _sequences(cu_seqlens, dev):
    if cu_seqlens is None or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be a vector of the sequences' bounds")
    nseq = cu_seqlens.shape[0] - 1
    return _whole(cu_seqlens, "cu_seqlens", torch.int32, dev, (nseq + 1,)), nseq


def _scratch(nbytes, dev):
    return _empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None


def _size(name, *sizes):
    """What one of the C size functions answers."""
    n = _call(name)[0](*sizes)
    if n == (1 << 64) - 1:  # SSD_WORKSPACE_INVALID
        from . import SSDError
        raise SSDError(1, f"{name}: invalid sizes {sizes}")
    return n


def _fresh(out, name, shape, dtype, dev):
    """out[name] checked, or a new tensor put there."""
    t = out.get(name)
    if t is None:
        t = out[name] = _empty(shape, dtype=dtype, device=dev)
        return t.data_ptr()
    return _whole(t, name, dtype, dev, shape)


def _given_or_new(t, name, like, shape):
    """(tensor, data pointer) of an output: the given one checked, or a new one of like's dtype."""
    if t is None:
        t = like.new_empty(shape)
        return t, t.data_ptr()
    return t, _whole(t, name, like.dtype, like.device, shape)


# ------------------------------------------------------------------ convolution

def _conv_outputs(out, n, x_channels, bc_channels, like):
    sx, sb = (n, x_channels), (n, bc_channels)
    if out is None:
        out = (like.new_empty(sx), like.new_empty(sb), like.new_empty(sb))
        return out, (out[0].data_ptr(), out[1].data_ptr() or None, out[2].data_ptr() or None)
    io, dev = like.dtype, like.device
    return out, (_whole(out[0], "x", io, dev, sx), _whole(out[1], "B", io, dev, sb) or None, _whole(out[2], "C", io, dev, sb) or None)


def _conv_inputs(xbc, weight, bias, x_channels, bc_channels):
    dev = _device_of(xbc, "xbc")
    _device_of(weight, "weight")
    _need_dim(xbc, "xbc", 2)
    _need_dim(weight, "weight", 2)
    n, ct = xbc.shape
    if x_channels is None:
        x_channels = ct - 2 * bc_channels
    if ct != x_channels + 2 * bc_channels:
        raise ValueError("xbc width must be x_channels + 2 bc_channels")
    width = weight.shape[1]
    xp, ld = _rows(xbc, "xbc", xbc.dtype, dev, (n, ct))
    return (dev, _io_of(xbc, "xbc"), n, ct, x_channels, width, xp, ld, _whole(weight, "weight", _f32, dev, (ct, width)),
            _maybe(bias, "bias", _f32, dev, (ct,)))


def ssd_conv1d_varlen(xbc, weight, bias, cu_seqlens, *, x_channels=None, bc_channels=0, silu=True, conv_state=None,
                      slots=None, has_init=None, out=None, stream=None):
    """The causal depthwise conv over packed prompts, split into the scan's inputs.

    xbc [tokens, Cx+2Cb] bf16/float32 (rows may be strided), weight [Cx+2Cb, K] and
    bias [Cx+2Cb] (or None) float32, cu_seqlens [nseq+1] int32.  conv_state [nslots,
    Cx+2Cb, K-1] is read where has_init (bool [nseq]) says so and left holding each
    prompt's last inputs, in slot slots[i] (int32 [nseq]; None: i).  Returns (x
    [tokens, Cx], B, C [tokens, Cb]); rows of no sequence are left as they were."""
    f, check = _call("ssd_conv1d_varlen")
    dev, io, n, ct, x_channels, width, xp, ld, wp, bp = _conv_inputs(xbc, weight, bias, x_channels, bc_channels)
    cu, nseq = _sequences(cu_seqlens, dev)
    sp, nslots = None, 0
    if conv_state is not None:
        _need_dim(conv_state, "conv_state", 3)
        nslots = conv_state.shape[0]
        sp = _whole(conv_state, "conv_state", xbc.dtype, dev, (nslots, ct, width - 1)) or None
    slp = _maybe(slots, "slots", torch.int32, dev, (nseq,))
    hip = _maybe(has_init, "has_init", torch.bool, dev, (nseq,))
    with _on(dev, stream):
        out, (xo, bo, co) = _conv_outputs(out, n, x_channels, bc_channels, xbc)
        check(f(xp, ld, wp, bp, cu, sp, slp, hip, xo, bo, co, io, n, nseq, nslots, x_channels, bc_channels, width,
                bool(silu), _raw_stream(dev.index)))
    return out


def ssd_conv1d_update(conv_state, xbc, weight, bias=None, *, slots=None, x_channels=None, bc_channels=0, silu=True,
                      out=None, stream=None):
    """The conv of one new token per sequence; conv_state [nslots, Cx+2Cb, K-1] moves
    on in place.  xbc [b, Cx+2Cb] (rows may be strided); sequence i uses slot slots[i]
    (None: i), and a negative slot skips it.  Returns (x [b, Cx], B, C [b, Cb])."""
    f, check = _call("ssd_conv1d_update")
    dev, io, n, ct, x_channels, width, xp, ld, wp, bp = _conv_inputs(xbc, weight, bias, x_channels, bc_channels)
    _device_of(conv_state, "conv_state")
    _need_dim(conv_state, "conv_state", 3)
    nslots = conv_state.shape[0]
    sp = _whole(conv_state, "conv_state", xbc.dtype, dev, (nslots, ct, width - 1))
    slp = _maybe(slots, "slots", torch.int32, dev, (n,))
    with _on(dev, stream):
        out, (xo, bo, co) = _conv_outputs(out, n, x_channels, bc_channels, xbc)
        check(f(sp, slp, xp, ld, wp, bp, xo, bo, co, io, n, nslots, x_channels, bc_channels, width, bool(silu),
                _raw_stream(dev.index)))
    return out


def ssd_conv1d_bwd(xbc, weight, bias, cu_seqlens, dx, dB=None, dC=None, *, silu=True, out=None, stream=None):
    """Gradients of ssd_conv1d_varlen without states: dict of dxbc [tokens, Cx+2Cb],
    dweight and dbias (float32; dbias None when bias is); ``out`` may pass them
    preallocated."""
    f, check = _call("ssd_conv1d_bwd")
    _device_of(xbc, "xbc")
    _device_of(dx, "dx")
    _need_dim(dx, "dx", 2)
    cb = 0 if dB is None else dB.shape[-1]
    dev, io, n, ct, cx, width, xp, ld, wp, bp = _conv_inputs(xbc, weight, bias, dx.shape[1], cb)
    cu, nseq = _sequences(cu_seqlens, dev)
    gx = _whole(dx, "dx", xbc.dtype, dev, (n, cx))
    gb, gc = (_whole(t, k, xbc.dtype, dev, (n, cb)) if cb else None for t, k in ((dB, "dB"), (dC, "dC")))
    with _on(dev, stream):
        out = {} if out is None else out
        po = [_fresh(out, "dxbc", (n, ct), xbc.dtype, dev), _fresh(out, "dweight", (ct, width), _f32, dev),
              None if bias is None else _fresh(out, "dbias", (ct,), _f32, dev)]
        out.setdefault("dbias", None)
        nbytes = _size("ssd_conv1d_bwd_workspace_size", n, ct, width)
        ws = _scratch(nbytes, dev)
        check(f(xp, ld, wp, bp, cu, gx, gb, gc, *po, io, n, nseq, cx, cb, width, bool(silu),
                None if ws is None else ws.data_ptr(), nbytes, _raw_stream(dev.index)))
    return out


# --------------------------------------------------------------- selective scan

def _sel_args(x, dt, A, B, C, D, z, dt_bias, softplus):
    dev = _device_of(x, "x")
    _device_of(B, "B")
    _need_dim(x, "x", 2)
    _need_dim(B, "B", 3)
    rows, io = x.shape, x.dtype
    n, d = rows
    _, G, N = B.shape
    a = _SelArgs()
    a.io_dtype = _io_of(x, "x")
    a.x, a.x_stride = _rows(x, "x", io, dev, rows)
    a.dt, a.dt_stride = _rows(dt, "dt", io, dev, rows)
    if z is not None:
        a.z, a.z_stride = _rows(z, "z", io, dev, rows)
    a.B, a.b_stride = _rows(B, "B", io, dev, (n, G, N))
    a.C, a.c_stride = _rows(C, "C", io, dev, (n, G, N))
    a.A = _whole(A, "A", _f32, dev, (d, N))
    a.D = _maybe(D, "D", _f32, dev, (d,))
    a.dt_bias = _maybe(dt_bias, "dt_bias", _f32, dev, (d,))
    a.softplus, a.channels, a.ngroups, a.dstate = bool(softplus), d, G, N
    return a, dev, n, d, G, N


def _states(state, slots, rows, d, N, dev):
    _need_dim(state, "state", 3)
    nslots = state.shape[0]
    return _whole(state, "state", _f32, dev, (nslots, d, N)), _maybe(slots, "slots", torch.int32, dev, (rows,)), nslots


def ssd_selective_scan_varlen(x, dt, A, B, C, cu_seqlens, D=None, z=None, dt_bias=None, *, softplus=True, state=None,
                              slots=None, has_init=None, y=None, return_chunk_states=False, stream=None):
    """The gated Mamba-1 scan over packed prompts.  Returns (y, chunk_states or None).

    x, dt, z [tokens, channels] and B, C [tokens, G, N], one dtype (bf16/float32), rows
    may be strided; A [channels, N], D, dt_bias [channels] float32; cu_seqlens [nseq+1]
    int32.  dt is before the bias and the softplus.  state [nslots, channels, N]
    float32 is read where has_init (bool [nseq]) says so and left holding each
    prompt's end state, in slot slots[i] (int32; None: i).  return_chunk_states keeps
    what ssd_selective_scan_bwd needs."""
    f, check = _call("ssd_selective_scan_varlen")
    a, dev, n, d, _, N = _sel_args(x, dt, A, B, C, D, z, dt_bias, softplus)
    cu, nseq = _sequences(cu_seqlens, dev)
    sp = slp = None
    nslots = 0
    if state is not None:
        sp, slp, nslots = _states(state, slots, nseq, d, N, dev)
    hip = _maybe(has_init, "has_init", torch.bool, dev, (nseq,))
    with _on(dev, stream):
        y, yp = _given_or_new(y, "y", x, (n, d))
        kept = None
        if return_chunk_states:
            kept = torch.empty((_size("ssd_selective_scan_chunk_states", n, nseq), N, d), dtype=_f32, device=dev)
        nbytes = _size("ssd_selective_scan_workspace_size", n, nseq, d, N)
        ws = _scratch(nbytes, dev)
        check(f(a, cu, sp, slp, hip, None if kept is None else kept.data_ptr(), yp, n,
                nseq, nslots, None if ws is None else ws.data_ptr(), nbytes, _raw_stream(dev.index)))
    return y, kept


def ssd_selective_state_update(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, *, softplus=True, slots=None, y=None,
                               stream=None):
    """One token per sequence of the gated Mamba-1 scan; ``state`` [nslots, channels, N]
    float32 is updated in place.  x, dt, z [b, channels], B, C [b, G, N] (rows may be
    strided); sequence i uses slot slots[i] (None: i), and a negative slot skips it.
    Returns y [b, channels]."""
    f, check = _call("ssd_selective_state_update")
    a, dev, n, d, _, N = _sel_args(x, dt, A, B, C, D, z, dt_bias, softplus)
    _device_of(state, "state")
    sp, slp, nslots = _states(state, slots, n, d, N, dev)
    with _on(dev, stream):
        y, yp = _given_or_new(y, "y", x, (n, d))
        check(f(a, sp, slp, yp, n, nslots, _raw_stream(dev.index)))
    return y


def ssd_selective_scan_bwd(x, dt, A, B, C, cu_seqlens, dy, chunk_states, D=None, z=None, dt_bias=None, *, softplus=True,
                           out=None, stream=None):
    """Gradients of ssd_selective_scan_varlen without states, from dy and the forward's
    chunk_states: dict of dx, ddt, dz, dB, dC (io dtype) and dA, dD, ddt_bias (float32);
    those of absent inputs are None.  ``out`` may pass them preallocated."""
    f, check = _call("ssd_selective_scan_bwd")
    a, dev, n, d, G, N = _sel_args(x, dt, A, B, C, D, z, dt_bias, softplus)
    cu, nseq = _sequences(cu_seqlens, dev)
    gy = _whole(dy, "dy", x.dtype, dev, (n, d))
    kept = _whole(chunk_states, "chunk_states", _f32, dev, (_size("ssd_selective_scan_chunk_states", n, nseq), N, d))
    with _on(dev, stream):
        out = {} if out is None else out
        shapes = dict(dx=((n, d), x.dtype, x), ddt=((n, d), x.dtype, dt), dz=((n, d), x.dtype, z), dB=((n, G, N), x.dtype, B),
                      dC=((n, G, N), x.dtype, C), dA=((d, N), _f32, A), dD=((d,), _f32, D), ddt_bias=((d,), _f32, dt_bias))
        po = [None if of is None else _fresh(out, k, s, t, dev) for k, (s, t, of) in shapes.items()]
        for k in shapes:
            out.setdefault(k, None)
        nbytes = _size("ssd_selective_scan_bwd_workspace_size", n, nseq, d, G, N)
        ws = _scratch(nbytes, dev)
        check(f(a, cu, gy, kept, *po, n, nseq, None if ws is None else ws.data_ptr(), nbytes, _raw_stream(dev.index)))
    return out


# ------------------------------------------------------------------------ norms

def ssd_residual_rmsnorm(x, weight, residual=None, scale=None, *, eps=1e-5, out=None, residual_out=None, stream=None):
    """r = residual + scale * x and out = rmsnorm(r) * weight, before a block.

    x [rows, width] bf16/float32, residual of x's dtype or float32 (rows of both may
    be strided), scale and weight [width] float32.  Returns (out, r): r in the
    residual's dtype (x's when there is none; residual_out may be residual itself)."""
    f, check = _call("ssd_residual_rmsnorm")
    dev, t = _device_of(x, "x"), x.dtype
    _need_dim(x, "x", 2)
    shape = n, d = x.shape
    io, rt, rp, ldr = _io_of(x, "x"), t, None, 0
    if residual is not None:
        rt = residual.dtype
        if rt != t and rt != _f32:
            raise ValueError("residual must have x's dtype or float32")
        rp, ldr = _rows(residual, "residual", rt, dev, shape)
    xp, ldx = _rows(x, "x", t, dev, shape)
    wp, sp = _whole(weight, "weight", _f32, dev, (d,)), _maybe(scale, "scale", _f32, dev, (d,))
    with _on(dev, stream):
        out, op = _given_or_new(out, "out", x, shape)
        residual_out, rop = _given_or_new(residual_out, "residual_out", x if residual is None else residual, shape)
        check(f(xp, ldx, rp, ldr, sp, wp, op, rop, io, _IO[rt], n, d, eps, _raw_stream(dev.index)))
    return out, residual_out


def ssd_residual_rmsnorm_bwd(residual, weight, dout, dresidual=None, x=None, scale=None, *, eps=1e-5, out=None, stream=None):
    """Gradients of ssd_residual_rmsnorm from the r it returned: dict of dresidual (r's
    dtype), dx (dout's dtype; the same tensor where neither scale nor a wider dtype
    sets them apart), dweight, and dscale (None without scale, which needs x)."""
    f, check = _call("ssd_residual_rmsnorm_bwd")
    dev = _device_of(residual, "residual")
    _device_of(dout, "dout")
    _need_dim(residual, "residual", 2)
    shape, rt, t = residual.shape, residual.dtype, dout.dtype
    n, d = shape
    io = _io_of(dout, "dout")
    if rt != t and rt != _f32:
        raise ValueError("residual must have dout's dtype or float32")
    rp, ldr = _rows(residual, "residual", rt, dev, shape)
    xp, ldx = _rows(x, "x", t, dev, shape) if scale is not None else (None, 0)
    wp, sp = _whole(weight, "weight", _f32, dev, (d,)), _maybe(scale, "scale", _f32, dev, (d,))
    up, ur = _whole(dout, "dout", t, dev, shape), _maybe(dresidual, "dresidual", rt, dev, shape)
    with _on(dev, stream):
        out = {} if out is None else out
        gr, apart = _fresh(out, "dresidual", shape, rt, dev), scale is not None or rt != t
        gx = _fresh(out, "dx", shape, t, dev) if apart else None
        if not apart:
            out["dx"] = out["dresidual"]
        gw = _fresh(out, "dweight", (d,), _f32, dev)
        gs = None if scale is None else _fresh(out, "dscale", (d,), _f32, dev)
        out.setdefault("dscale", None)
        nbytes = _size("ssd_rmsnorm_bwd_workspace_size", n, d)
        ws = _scratch(nbytes, dev)
        check(f(rp, ldr, wp, up, ur, xp, ldx, sp, gx, gr, gw, gs, io, _IO[rt], n, d, eps, None if ws is None else ws.data_ptr(),
                nbytes, _raw_stream(dev.index)))
    return out


def _gated_inputs(y, z, weight, scale):
    dev, t = _device_of(y, "y"), y.dtype
    _need_dim(y, "y", 2)
    shape = y.shape
    yp, ldy = _rows(y, "y", t, dev, shape)
    zp, ldz = (None, 0) if z is None else _rows(z, "z", t, dev, shape)
    width = (shape[1],)
    return (dev, _io_of(y, "y"), shape, yp, ldy, zp, ldz, _whole(weight, "weight", _f32, dev, width),
            _maybe(scale, "scale", _f32, dev, width))


def ssd_gated_rmsnorm(y, z, weight, residual=None, scale=None, *, ngroups=1, norm_before_gate=False, eps=1e-5, out=None,
                      stream=None):
    """rmsnorm(y * silu(z)) * weight over each of ngroups groups of channels, or
    rmsnorm(y) * weight * silu(z) with norm_before_gate; times scale and plus residual
    where they are given.  y, z (None: no gate), residual [rows, width] of one dtype
    (bf16/float32; rows may be strided), weight, scale [width] float32."""
    f, check = _call("ssd_gated_rmsnorm")
    dev, io, shape, yp, ldy, zp, ldz, wp, sp = _gated_inputs(y, z, weight, scale)
    rp, ldr = (None, 0) if residual is None else _rows(residual, "residual", y.dtype, dev, shape)
    with _on(dev, stream):
        out, op = _given_or_new(out, "out", y, shape)
        check(f(yp, ldy, zp, ldz, rp, ldr, sp, wp, op, io, *shape, ngroups, bool(norm_before_gate), eps,
                _raw_stream(dev.index)))
    return out


def ssd_gated_rmsnorm_bwd(y, z, weight, dout, scale=None, *, ngroups=1, norm_before_gate=False, eps=1e-5, out=None,
                          stream=None):
    """Gradients of ssd_gated_rmsnorm: dict of dy, dz (None without z), dweight and
    dscale (None without scale); the residual's gradient is dout."""
    f, check = _call("ssd_gated_rmsnorm_bwd")
    dev, io, shape, yp, ldy, zp, ldz, wp, sp = _gated_inputs(y, z, weight, scale)
    t, width = y.dtype, (shape[1],)
    up = _whole(dout, "dout", t, dev, shape)
    with _on(dev, stream):
        out = {} if out is None else out
        gy, gz = _fresh(out, "dy", shape, t, dev), None if z is None else _fresh(out, "dz", shape, t, dev)
        gw = _fresh(out, "dweight", width, _f32, dev)
        gs = None if scale is None else _fresh(out, "dscale", width, _f32, dev)
        out.setdefault("dz", None)
        out.setdefault("dscale", None)
        nbytes = _size("ssd_rmsnorm_bwd_workspace_size", *shape)
        ws = _scratch(nbytes, dev)
        check(f(yp, ldy, zp, ldz, wp, up, sp, gy, gz, gw, gs, io, *shape, ngroups, bool(norm_before_gate), eps,
                None if ws is None else ws.data_ptr(), nbytes, _raw_stream(dev.index)))
    return out
