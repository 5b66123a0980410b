"""Python binding of the layer operators of libgdn.so: the short causal convolution,
the S6 scan, the RMS norm, the gated linear recurrence, layer norm and rotary positions.

As in binding.py the functions carry the C ABI's names; the signatures are here, the checks,
allocations and calls in the extension module that csrc/layer_binding.cpp builds.  Row operands
may be slices of a wider projection (the last dimension dense, tokens a constant stride apart);
parameters, states and outputs are contiguous.  As everywhere in the library the outputs carry
no gradient; the recurrence, layer norm and rotary positions have theirs as calls of their own
(``_bwd``).  ``stream`` (a torch stream, or a cudaStream_t as a number) runs a call, and makes
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
                 "gdn_rms_norm_fwd_e4m3", "gdn_rms_norm_fwd_e4m3_f32",
                 "gdn_glr_chunk_fwd", "gdn_glr_chunk_fwd_f32", "gdn_glr_recurrent_step",
                 "gdn_glr_recurrent_step_f32", "gdn_glr_chunk_bwd", "gdn_glr_chunk_bwd_f32",
                 "gdn_glr_chunk_bwd_workspace_size", "gdn_layer_norm_fwd", "gdn_layer_norm_fwd_f32",
                 "gdn_layer_norm_bwd", "gdn_layer_norm_bwd_f32", "gdn_layer_norm_bwd_workspace_size",
                 "gdn_rotary_fwd", "gdn_rotary_fwd_f32", "gdn_rotary_bwd", "gdn_rotary_bwd_f32")
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


_GATES = {"log": 0, "sigmoid": 1, "rate": 2}
_INPUT_NORMS = {None: 0, "linear": 1, "sqrt": 2}


def _glr_form(gate, input_norm):
    if gate not in _GATES:
        raise ValueError(f"gate must be 'log', 'sigmoid' or 'rate', got {gate!r}")
    if input_norm not in _INPUT_NORMS:
        raise ValueError(f"input_norm must be None, 'linear' or 'sqrt', got {input_norm!r}")
    return _GATES[gate], _INPUT_NORMS[input_norm]


def gdn_glr_chunk_fwd(x, g, rate=None, h0=None, y=None, hT=None, states=None, *, gate: str = "log",
                      input_norm: Optional[str] = None, cu_seqlens=None, output_final_state=True,
                      output_states=False, stream=None):
    """Gated linear recurrence over a prompt; returns (y, hT, states).

    Per channel h_t = a_t h_{t-1} + s_t x_t, y_t = h_t, with the decay a = exp(g) (gate "log", g <= 0),
    sigmoid(g) ("sigmoid") or exp(rate sigmoid(g)) ("rate"; rate [D] fp32, <= 0), and the input's weight
    s = 1 (input_norm None), 1 - a ("linear") or sqrt(1 - a^2) ("sqrt").  x, g [B, T, D] (bf16 or
    fp32, both the same; each may be a slice of a wider projection); h0 [N, D] fp32 or None; hT may be
    h0 (in place).  With cu_seqlens (int32 [N+1] on the device) the batch is one packed row, B = 1;
    rows behind cu_seqlens[N] are left as they were.  output_states: ``states`` [B, ceil(T / 64), D]
    fp32, the state before every 64th token of a row, which gdn_glr_chunk_bwd takes.
    """
    if stream is not None:
        with _on(stream, x):
            return gdn_glr_chunk_fwd(x, g, rate, h0, y, hT, states, gate=gate, input_norm=input_norm,
                                     cu_seqlens=cu_seqlens, output_final_state=output_final_state,
                                     output_states=output_states)
    return (_native or _load()).glr_fwd(x, g, rate, h0, y, hT, states, *_glr_form(gate, input_norm), cu_seqlens,
                                        output_final_state, output_states)


def gdn_glr_recurrent_step(x, g, h, rate=None, y=None, *, gate: str = "log", input_norm: Optional[str] = None,
                           stream=None):
    """One token of the gated linear recurrence; updates h [N, D] in place and returns y.

    x, g [N, D]; the rest as in gdn_glr_chunk_fwd.
    """
    if stream is not None:
        with _on(stream, x):
            return gdn_glr_recurrent_step(x, g, h, rate, y, gate=gate, input_norm=input_norm)
    return (_native or _load()).glr_step(x, g, h, rate, y, *_glr_form(gate, input_norm))


def gdn_glr_chunk_bwd_workspace_size(N, T, D, gate="log", varlen=False) -> int:
    """Bytes of workspace the gated recurrence's gradient needs (0: none, or rejected sizes)."""
    return int(load_library().gdn_glr_chunk_bwd_workspace_size(N, T, D, _glr_form(gate, None)[0], int(bool(varlen))))


def gdn_glr_chunk_bwd(dy, x, g, states, rate=None, h0=None, dhT=None, dx=None, dg=None, drate=None, dh0=None, *,
                      gate: str = "log", input_norm: Optional[str] = None, cu_seqlens=None, stream=None,
                      workspace=None):
    """Gradient of the gated linear recurrence; returns (dx, dg, drate, dh0).

    dy [B, T, D] (x's type, may be a slice) and dhT [N, D] fp32 (or None for zeros) are the gradients of
    y and hT; ``states`` is the forward's, the other inputs and the form are the same as there.
    drate [D] fp32 is None without a rate, dh0 [N, D] fp32 None without h0 (unless given).  h0 is what it
    was before the forward: with cu_seqlens it is read, so that a forward in place needs a copy of it.
    ``workspace``: a uint8 device tensor of at least gdn_glr_chunk_bwd_workspace_size bytes, or None for
    a fresh one where one is needed.
    """
    if stream is not None:
        with _on(stream, x):
            return gdn_glr_chunk_bwd(dy, x, g, states, rate, h0, dhT, dx, dg, drate, dh0, gate=gate,
                                     input_norm=input_norm, cu_seqlens=cu_seqlens, workspace=workspace)
    return (_native or _load()).glr_bwd(dy, x, g, states, rate, h0, dhT, dx, dg, drate, dh0,
                                        *_glr_form(gate, input_norm), cu_seqlens, workspace)


def gdn_layer_norm_fwd(x, weight=None, bias=None, residual=None, y=None, residual_out=None, *, eps: float = 1e-5,
                       stream=None):
    """Layer norm of the rows of x [..., D]; returns (y, residual_out).

    r = x + residual; y = (r - mean(r)) / sqrt(var(r) + eps) * weight + bias (the variance over D).  x
    and residual are bf16 or fp32, both the same; weight and bias [D] fp32 or None.  x may be a slice
    (rows a constant stride apart); residual is contiguous and residual_out (a fresh tensor, or residual
    itself: in place) takes r in x's type, None without a residual.
    """
    if stream is not None:
        with _on(stream, x):
            return gdn_layer_norm_fwd(x, weight, bias, residual, y, residual_out, eps=eps)
    return (_native or _load()).ln_fwd(x, weight, bias, residual, y, residual_out, eps)


def gdn_layer_norm_bwd_workspace_size(rows, D) -> int:
    """Bytes of workspace the gradient of weight and bias needs (0: rejected sizes)."""
    return int(load_library().gdn_layer_norm_bwd_workspace_size(rows, D))


def gdn_layer_norm_bwd(dy, x, weight=None, dres=None, dx=None, dweight=None, dbias=None, *, eps: float = 1e-5,
                       param_grads: bool = True, stream=None, workspace=None):
    """Gradient of layer norm; returns (dx, dweight, dbias).

    dy and x [..., D] (each may be a slice); x is what was normed: with a residual the forward's
    residual_out, whose own gradient ``dres`` (contiguous, or None) is added to dx (which may be dres: in
    place); dx is then the gradient of x and residual alike.  dweight and dbias [D] fp32, or None without
    param_grads.  ``workspace``: a uint8 device tensor of at least gdn_layer_norm_bwd_workspace_size
    bytes, or None for a fresh one.
    """
    if stream is not None:
        with _on(stream, x):
            return gdn_layer_norm_bwd(dy, x, weight, dres, dx, dweight, dbias, eps=eps, param_grads=param_grads,
                                      workspace=workspace)
    return (_native or _load()).ln_bwd(dy, x, weight, dres, dx, dweight, dbias, eps, param_grads, workspace)


_SCALINGS = {None: 0, "linear": 1, "ntk": 2, "yarn": 3}


def gdn_rotary_turns(dim: int, base: float = 10000.0, *, scaling: Optional[str] = None, factor: float = 1.0,
                     original_length: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """The table of gdn_rotary_fwd for ``dim`` rotated columns; returns (turns, magnitude).

    turns [dim / 2] (int64 on ``device``): pair i turns by base^(-2 i / dim) radians a position, kept as
    2^64ths of a turn; magnitude scales the rotated columns.  For contexts ``factor`` times as long:
    scaling "linear" divides the frequencies by it, "ntk" raises the base, "yarn" divides those that
    make few turns within ``original_length`` (below beta_slow) and keeps those that make many (above
    beta_fast), with a magnitude of 0.1 ln(factor) + 1.
    """
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be None, 'linear', 'ntk' or 'yarn', got {scaling!r}")
    if not 0 < dim <= 1 << 20:
        raise ValueError(f"dim = {dim} is out of range")
    table = torch.empty(max(dim // 2, 1), dtype=torch.int64)
    magnitude = ctypes.c_float()
    s = load_library().gdn_rotary_turns(dim, base, _SCALINGS[scaling], factor, original_length, beta_fast, beta_slow,
                                        table.data_ptr(), ctypes.addressof(magnitude))
    if s != 0:
        _check(s)
    return table.to(device), magnitude.value


def gdn_rotary_fwd(q, k, turns, positions=None, q_out=None, k_out=None, *, magnitude: float = 1.0,
                   interleaved: bool = False, cu_seqlens=None, offsets=None, stream=None):
    """Rotary positions of q [..., Hq, D] and k [..., Hk, D] (or None); returns (q_out, k_out).

    The first 2 len(turns) columns of every head are turned in pairs (i, i + R/2), or (2i, 2i + 1) with
    ``interleaved``, by position times ``turns`` (gdn_rotary_turns), and scaled by ``magnitude``; the
    others are passed through.  q and k are bf16 or fp32, both the same; each may be a slice of a
    projection whose tokens are a constant stride apart, and its own output (in place).  positions: int32,
    q's shape without [H, D].  Without them q is [B, T, H, D] and a token's position is counted from
    its sequence's first (cu_seqlens: one packed row, B = 1; rows behind the last sequence are left as
    they were), plus offsets [N] int32 (or None).
    """
    if stream is not None:
        with _on(stream, q):
            return gdn_rotary_fwd(q, k, turns, positions, q_out, k_out, magnitude=magnitude,
                                  interleaved=interleaved, cu_seqlens=cu_seqlens, offsets=offsets)
    return (_native or _load()).rotary(q, k, turns, positions, q_out, k_out, magnitude, interleaved, cu_seqlens,
                                       offsets, False)


def gdn_rotary_bwd(dq, dk, turns, positions=None, dq_out=None, dk_out=None, *, magnitude: float = 1.0,
                   interleaved: bool = False, cu_seqlens=None, offsets=None, stream=None):
    """Gradient of gdn_rotary_fwd: from those of q_out and k_out to those of q and k; arguments as there."""
    if stream is not None:
        with _on(stream, dq):
            return gdn_rotary_bwd(dq, dk, turns, positions, dq_out, dk_out, magnitude=magnitude,
                                  interleaved=interleaved, cu_seqlens=cu_seqlens, offsets=offsets)
    return (_native or _load()).rotary(dq, dk, turns, positions, dq_out, dk_out, magnitude, interleaved, cu_seqlens,
                                       offsets, True)
