"""The rest of a mixer block around its matrix products: the short causal
convolution and the gated Mamba-1 scan on packed prompts and on single tokens,
their gradients, and the norms before and after the block.

The functions have the C entry points' names (``include/ssd.h`` says what each
argument means).  Their checks, outputs and scratch are in the native module _bind
(``csrc/bind.cpp``), which makes the C calls: from Python they cost more than the
launch of a small kernel itself.  Inputs that a
projection's output holds side by side may be passed as slices: rows may be
strided, the last dimension may not.  Outputs and scratch are allocated for each
call on the stream that the call runs on, so calls on several streams and captured
graphs never share scratch.

No call records an autograd graph: a result carries no gradient even where an input
requires one.  Training calls the ``_bwd`` functions, or wraps a pair in its own
torch.autograd.Function.  A dict given as ``out`` may be an earlier call's: what it
holds is written again, and gradients of absent inputs become None.
"""
from __future__ import annotations

import ctypes

import torch

_VP, _I, _LL, _SZ, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t, ctypes.c_float


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


_native = None


def _load():
    """The native module, bound to the loaded library's entry points."""
    global _native
    from . import load_library
    lib = load_library()
    try:
        from . import _bind
    except ImportError as e:
        raise RuntimeError("the native binding cannot be loaded: build it with "
                           f"`python -m selective_state_space_22_b200.build` ({e})") from e
    _bind.bind({n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _bind.names()})
    _native = _bind
    return _bind


def _run(name, stream, *args):
    if stream is not None:
        device = getattr(args[0], "device", stream.device)  # the first argument's is the call's
        if device.type == "cuda" and stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
        with torch.cuda.stream(stream):
            return _run(name, None, *args)
    r = getattr(_native or _load(), name)(*args)
    if type(r) is int:
        from . import _check
        _check(r)
    return r


# ------------------------------------------------------------------ convolution

def ssd_conv1d_varlen(xbc, weight, bias, cu_seqlens, *, x_channels=None, bc_channels=0, silu=True, conv_state=None,
                      slots=None, has_init=None, out=None, stream=None):
    """The causal depthwise conv over packed prompts, split into the scan's inputs.

    xbc [tokens, Cx+2Cb] bf16/float32 (rows may be strided), weight [Cx+2Cb, K] and
    bias [Cx+2Cb] (or None) float32, cu_seqlens [nseq+1] int32.  conv_state [nslots,
    Cx+2Cb, K-1] is read where has_init (bool [nseq]) says so and left holding each
    prompt's last inputs, in slot slots[i] (int32 [nseq]; None: i).  Returns (x
    [tokens, Cx], B, C [tokens, Cb]); rows of no sequence are left as they were."""
    return _run("conv1d_varlen", stream, xbc, weight, bias, cu_seqlens, x_channels, bc_channels, silu, conv_state,
                slots, has_init, out)


def ssd_conv1d_update(conv_state, xbc, weight, bias=None, *, slots=None, x_channels=None, bc_channels=0, silu=True,
                      out=None, stream=None):
    """The conv of one new token per sequence; conv_state [nslots, Cx+2Cb, K-1] moves
    on in place.  xbc [b, Cx+2Cb] (rows may be strided); sequence i uses slot slots[i]
    (None: i), and a negative slot skips it.  Returns (x [b, Cx], B, C [b, Cb])."""
    return _run("conv1d_update", stream, xbc, weight, bias, conv_state, x_channels, bc_channels, silu, slots, out)


def ssd_conv1d_bwd(xbc, weight, bias, cu_seqlens, dx, dB=None, dC=None, *, silu=True, out=None, stream=None):
    """Gradients of ssd_conv1d_varlen without states: dict of dxbc [tokens, Cx+2Cb],
    dweight and dbias (float32; dbias None when bias is); ``out`` may pass them
    preallocated."""
    return _run("conv1d_bwd", stream, xbc, weight, bias, cu_seqlens, dx, dB, dC, silu, out)


# --------------------------------------------------------------- selective scan

def ssd_selective_scan_varlen(x, dt, A, B, C, cu_seqlens, D=None, z=None, dt_bias=None, *, softplus=True, state=None,
                              slots=None, has_init=None, y=None, return_chunk_states=False, stream=None):
    """The gated Mamba-1 scan over packed prompts.  Returns (y, chunk_states or None).

    x, dt, z [tokens, channels] and B, C [tokens, G, N], one dtype (bf16/float32), rows
    may be strided; A [channels, N], D, dt_bias [channels] float32; cu_seqlens [nseq+1]
    int32.  dt is before the bias and the softplus.  state [nslots, channels, N]
    float32 is read where has_init (bool [nseq]) says so and left holding each
    prompt's end state, in slot slots[i] (int32; None: i).  return_chunk_states keeps
    what ssd_selective_scan_bwd needs: N / 2 bytes per token and channel (268 MB for
    32768 tokens of 1024 channels of 16 states)."""
    return _run("selective_scan_varlen", stream, x, dt, A, B, C, D, z, dt_bias, softplus, cu_seqlens, state, slots,
                has_init, y, return_chunk_states)


def ssd_selective_state_update(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, *, softplus=True, slots=None, y=None,
                               stream=None):
    """One token per sequence of the gated Mamba-1 scan; ``state`` [nslots, channels, N]
    float32 is updated in place.  x, dt, z [b, channels], B, C [b, G, N] (rows may be
    strided); sequence i uses slot slots[i] (None: i), and a negative slot skips it.
    Returns y [b, channels]."""
    return _run("selective_state_update", stream, x, dt, A, B, C, D, z, dt_bias, softplus, state, slots, y)


def ssd_selective_scan_bwd(x, dt, A, B, C, cu_seqlens, dy, chunk_states, D=None, z=None, dt_bias=None, *, softplus=True,
                           out=None, stream=None):
    """Gradients of ssd_selective_scan_varlen without states, from dy and the forward's
    chunk_states: dict of dx, ddt, dz, dB, dC (io dtype) and dA, dD, ddt_bias (float32);
    those of absent inputs are None.  ``out`` may pass them preallocated."""
    return _run("selective_scan_bwd", stream, x, dt, A, B, C, D, z, dt_bias, softplus, cu_seqlens, dy, chunk_states,
                out)


# ------------------------------------------------------------------------ norms

def ssd_residual_rmsnorm(x, weight, residual=None, scale=None, *, eps=1e-5, out=None, residual_out=None, stream=None):
    """r = residual + scale * x and out = rmsnorm(r) * weight, before a block.

    x [rows, width] bf16/float32, residual of x's dtype or float32 (rows of both may
    be strided), scale and weight [width] float32.  Returns (out, r): r in the
    residual's dtype (x's when there is none; residual_out may be residual itself)."""
    return _run("residual_rmsnorm", stream, x, weight, residual, scale, eps, out, residual_out)


def ssd_residual_rmsnorm_bwd(residual, weight, dout, dresidual=None, x=None, scale=None, *, eps=1e-5, out=None, stream=None):
    """Gradients of ssd_residual_rmsnorm from the r it returned: dict of dresidual (r's
    dtype), dx (dout's dtype; the same tensor where neither scale nor a wider dtype
    sets them apart and ``out`` holds no dx), dweight, and dscale (None without scale,
    which needs x).  ``out`` may pass them preallocated; where it holds one tensor as both
    and the call sets them apart, dx becomes a new one."""
    return _run("residual_rmsnorm_bwd", stream, residual, weight, dout, dresidual, x, scale, eps, out)


def ssd_gated_rmsnorm(y, z, weight, residual=None, scale=None, *, ngroups=1, norm_before_gate=False, eps=1e-5, out=None,
                      stream=None):
    """rmsnorm(y * silu(z)) * weight over each of ngroups groups of channels, or
    rmsnorm(y) * weight * silu(z) with norm_before_gate; times scale and plus residual
    where they are given.  y, z (None: no gate), residual [rows, width] of one dtype
    (bf16/float32; rows may be strided), weight, scale [width] float32."""
    return _run("gated_rmsnorm", stream, y, z, weight, residual, scale, ngroups, norm_before_gate, eps, out)


def ssd_gated_rmsnorm_bwd(y, z, weight, dout, scale=None, *, ngroups=1, norm_before_gate=False, eps=1e-5, out=None,
                          stream=None):
    """Gradients of ssd_gated_rmsnorm: dict of dy, dz (None without z), dweight and
    dscale (None without scale); the residual's gradient is dout.  ``out`` may pass them
    preallocated."""
    return _run("gated_rmsnorm_bwd", stream, y, z, weight, dout, scale, ngroups, norm_before_gate, eps, out)
