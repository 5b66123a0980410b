"""Python binding of the layer operators of libgdn.so: the short causal convolution,
the S6 scan and the RMS norm.

As in binding.py the functions carry the C ABI's names; the signatures are here, the checks,
allocations and calls in the extension module that csrc/layer_binding.cpp builds.  Row operands
may be slices of a wider projection (the last dimension dense, tokens a constant stride apart);
parameters, states and outputs are contiguous.  As everywhere in the library the outputs carry
no gradient.  ``stream`` (a torch stream, or a cudaStream_t as a number) runs a call, and makes
its allocations, on another stream than the current one.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _build
from .binding import _check, load_library

_E4M3 = torch.float8_e4m3fn
# entry points in the order that the extension's Library has them: bf16, fp32
_ENTRY_POINTS = ("gdn_short_conv_fwd", "gdn_short_conv_fwd_f32", "gdn_short_conv_step",
                 "gdn_short_conv_step_f32", "gdn_s6_chunk_fwd", "gdn_s6_chunk_fwd_f32",
                 "gdn_s6_recurrent_step", "gdn_s6_recurrent_step_f32",
                 "gdn_s6_chunk_fwd_workspace_size", "gdn_rms_norm_fwd", "gdn_rms_norm_fwd_f32",
                 "gdn_rms_norm_fwd_e4m3", "gdn_rms_norm_fwd_e4m3_f32")
_native = None


def _load():
    """The extension module, told the library's entry points (once)."""
    global _native
    lib = load_library()
    built_for, key = _build.binding_built_for(), _build.binding_key()
    if built_for is None or built_for != key:  # another torch's C++ ABI is not to be loaded
        raise RuntimeError(f"the layer operators' binding is built for {built_for or 'nothing'}, this is {key}: "
                           "python -m linear_attention_prefill_gb300._build")
    from . import _layer_native
    _layer_native.init(tuple(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _ENTRY_POINTS),
                       _check)
    _native = _layer_native
    return _native


def _on(stream, x):
    """``stream`` as the current one: the call's own allocations belong to it too."""
    if not isinstance(stream, torch.cuda.Stream):
        if not isinstance(x, torch.Tensor) or not x.is_cuda:
            raise ValueError("a stream needs operands on a CUDA device")
        stream = (torch.cuda.ExternalStream(int(stream), device=x.device) if int(stream) else
                  torch.cuda.default_stream(x.device))
    elif isinstance(x, torch.Tensor) and x.device != stream.device:
        raise ValueError(f"x is on {x.device}, the stream on {stream.device}")
    return torch.cuda.stream(stream)


def _act(activation) -> int:
    if activation == "silu":
        return 1
    if activation is None:
        return 0
    raise ValueError(f"activation must be 'silu' or None, got {activation!r}")


def gdn_short_conv_fwd(x, weight, bias=None, s0=None, y=None, sT=None, *,
                       activation: Optional[str] = "silu", cu_seqlens=None,
                       output_final_state=True, stream=None):
    """Short causal convolution of a prompt, one filter per channel; returns (y, sT).

    y_t = act(bias + sum_j weight[:, j] x_{t-W+1+j}).  x [B, T, D] (bf16 or fp32; may be a
    slice of a wider projection), weight [D, W] fp32 (W 2 to 4, the last tap meets x_t),
    bias [D] fp32 or None, s0 [N, W-1, D] (x's type: the inputs before each sequence, oldest
    first) or None for zeros.  With cu_seqlens (int32 [N+1] on the device) the batch is one
    packed row, B = 1; rows behind cu_seqlens[N] are left as they were.  sT [N, W-1, D] may
    be s0 (in place).
    """
    if stream is not None:
        with _on(stream, x):
            return gdn_short_conv_fwd(x, weight, bias, s0, y, sT, activation=activation,
                                      cu_seqlens=cu_seqlens, output_final_state=output_final_state)
    return (_native or _load()).conv_fwd(x, weight, bias, s0, y, sT, _act(activation), cu_seqlens,
                                         output_final_state)


def gdn_short_conv_step(x, weight, s, bias=None, y=None, *, activation: Optional[str] = "silu",
                        stream=None):
    """One token of the short convolution; shifts s [N, W-1, D] in place, returns y.

    x [N, D] (may be a slice of a wider projection); weight, bias and activation as in
    gdn_short_conv_fwd.
    """
    if stream is not None:
        with _on(stream, x):
            return gdn_short_conv_step(x, weight, s, bias, y, activation=activation)
    return (_native or _load()).conv_step(x, weight, s, bias, y, _act(activation))


def gdn_s6_chunk_fwd_workspace_size(N, T, dim, Ns, varlen=False) -> int:
    """Bytes of workspace the S6 scan needs (0: none, or rejected sizes)."""
    return int(load_library().gdn_s6_chunk_fwd_workspace_size(N, T, dim, Ns, int(bool(varlen))))


def gdn_s6_chunk_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, y=None, hT=None, *,
                     dt_softplus: bool = False, cu_seqlens=None, output_final_state=True,
                     stream=None, workspace=None):
    """Selective state space scan with a diagonal A (S6) over a prompt; returns (y, hT).

    With step = softplus(dt + dt_bias) (dt_softplus) or dt + dt_bias, per channel and state
    h_t = exp(step A) h_{t-1} + step x_t B_t, y_t = (C_t . h_t + D x_t) silu(z_t).
    x, dt [B, T, D] and z [B, T, D] or None, B, C [B, T, Ns] (bf16 or fp32, all the same; each
    may be a slice of a wider projection); A [D, Ns], D and dt_bias [D] fp32 or None; h0
    [N, D, Ns] fp32 or None.  With cu_seqlens (int32 [N+1] on the device) the batch is one
    packed row, B = 1; rows behind cu_seqlens[N] are left as they were.  hT may be h0 (in
    place).  ``workspace``: a uint8 device tensor of at least
    gdn_s6_chunk_fwd_workspace_size bytes, or None for a fresh one where the sizes need one.
    """
    if stream is not None:
        with _on(stream, x):
            return gdn_s6_chunk_fwd(x, dt, A, B, C, D, z, dt_bias, h0, y, hT, dt_softplus=dt_softplus,
                                    cu_seqlens=cu_seqlens, output_final_state=output_final_state,
                                    workspace=workspace)
    return (_native or _load()).s6_fwd(x, dt, A, B, C, D, z, dt_bias, h0, y, hT, dt_softplus, cu_seqlens,
                                       output_final_state, workspace)


def gdn_s6_recurrent_step(x, dt, A, B, C, h, D=None, z=None, dt_bias=None, y=None, *,
                          dt_softplus: bool = False, stream=None):
    """One token of the S6 recurrence; updates h [N, D, Ns] in place and returns y.

    x, dt, z [N, D]; B, C [N, Ns]; the rest as in gdn_s6_chunk_fwd.
    """
    if stream is not None:
        with _on(stream, x):
            return gdn_s6_recurrent_step(x, dt, A, B, C, h, D, z, dt_bias, y, dt_softplus=dt_softplus)
    return (_native or _load()).s6_step(x, dt, A, B, C, D, z, dt_bias, h, y, dt_softplus)


def gdn_rms_norm_fwd(x, weight, residual=None, gate=None, y=None, residual_out=None, scales=None, *,
                     eps: float = 1e-6, out_dtype=None, group: Optional[int] = None, stream=None):
    """RMS norm of the rows of x [..., D]; returns (y, scales, residual_out).

    r = x + residual; y = r / sqrt(mean(r^2) + eps) * weight * silu(gate) (the gate of a Gated
    DeltaNet layer; there is no sigmoid gate and none before the norm).  x, residual, gate
    are bf16 or fp32, all the same; weight [D] fp32.  x and gate may be slices, both in one of two
    forms: rows a constant stride apart, or [..., H, D] with dense H D and a constant stride before it.
    residual is contiguous and residual_out (a fresh tensor, or residual itself: in place) takes
    r in x's type.  out_dtype torch.float8_e4m3fn gives y in 8 bits with fp32
    scales [..., ceil(D / group)], one per ``group`` (32, 64, 128) columns or one a row (None):
    scale = max|y| / 448 (1 for zeros); a value is y times the scale's reciprocal, rounded to nearest
    (within a few fp32 roundings of a tie, either way).  scales and residual_out are None where there
    are none.
    """
    if stream is not None:
        with _on(stream, x):
            return gdn_rms_norm_fwd(x, weight, residual, gate, y, residual_out, scales, eps=eps,
                                    out_dtype=out_dtype, group=group)
    fp8 = out_dtype is _E4M3
    if not fp8 and out_dtype is not None and out_dtype != getattr(x, "dtype", None):
        raise TypeError(f"out_dtype must be the type of x or {_E4M3}, got {out_dtype}")
    if group is not None and (not fp8 or group not in (32, 64, 128)):
        raise ValueError(f"group (of the e4m3 output) must be 32, 64, 128 or None, got {group!r}")
    return (_native or _load()).norm_fwd(x, weight, residual, gate, y, residual_out, scales, eps, fp8,
                                         group or 0)
