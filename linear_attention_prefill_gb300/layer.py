"""Python binding of the layer operators of libgdn.so: the short causal convolution,
the S6 scan and the RMS norm.

As in binding.py the functions carry the C ABI's names, check their tensors, pass raw
pointers, strides and sizes on and raise what the library reports.  Row operands may be
slices of a wider projection (the last dimension dense, tokens a constant stride apart);
parameters, states and outputs are contiguous.
"""
from __future__ import annotations

from typing import Optional

import torch

from .binding import _check, _need, _ptr, _stream_handle, load_library

_ACT = {None: 0, "silu": 1}
_SUFFIX = {torch.bfloat16: "", torch.float32: "_f32"}
_E4M3 = torch.float8_e4m3fn


def _call(name: str, dev: torch.device, stream, *args):
    """One library call with ``dev`` as the current device, on ``stream`` or dev's current one."""
    fn = getattr(load_library(), name)
    if torch.cuda.current_device() == dev.index:
        _check(fn(*args, _stream_handle(stream, dev)))
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, _stream_handle(stream, dev)))


def _kind(x, name: str) -> str:
    """The C name's suffix for x's type; x must live on a GPU."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.device.type != "cuda":
        raise ValueError(f"{name} must be on a CUDA device")
    try:
        return _SUFFIX[x.dtype]
    except KeyError:
        raise TypeError(f"{name} must be bf16 or fp32, got {x.dtype}") from None


def _typed(t, name: str, dtype, device, shape):
    """Checks type, device and shape of an operand that need not be contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _stride_of(t, inner: int = 1):
    """Elements from token to token of ``t``, whose last ``inner`` dimensions are one dense
    token and whose others lie a constant stride apart; None if they do not."""
    shape, strides, cols = t.shape, t.stride(), 1
    if t.numel() == 0:
        return max(1, shape[-inner:].numel())
    split = len(shape) - inner
    for i in range(len(shape) - 1, split - 1, -1):
        if shape[i] != 1 and strides[i] != cols:
            return None
        cols *= shape[i]
    stride, seen = cols, 1
    for i in range(split - 1, -1, -1):
        if shape[i] != 1:
            if seen == 1:
                stride = strides[i]
            elif strides[i] != stride * seen:
                return None
            seen *= shape[i]
    return stride if stride >= cols or seen <= 1 else None


def _rows(t, name: str, dtype, device, shape) -> int:
    """Checks a row operand [..., cols] and returns its elements from token to token."""
    _typed(t, name, dtype, device, shape)
    stride = _stride_of(t)
    if stride is None:
        raise ValueError(f"{name} with strides {t.stride()}: the last dimension must be dense and "
                         "tokens a constant stride apart")
    return stride


def _param(t, name: str, device, shape):
    if t is not None:
        _need(t, name, torch.float32, device, shape)


def _sequences(lead, cu_seqlens, device):
    """(N, T) of a batch whose tensors have the leading dimensions ``lead`` = (B, T)."""
    if cu_seqlens is None:
        return lead
    _need(cu_seqlens, "cu_seqlens", torch.int32, device)
    if lead[0] != 1:
        raise ValueError("with cu_seqlens the batch must be one packed row (B == 1)")
    if cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens needs at least one sequence")
    return cu_seqlens.numel() - 1, lead[1]


def _act(activation) -> int:
    try:
        return _ACT[activation]
    except (KeyError, TypeError):
        raise ValueError(f"activation must be 'silu' or None, got {activation!r}") from None


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
    suffix = _kind(x, "x")
    if x.dim() != 3 or weight.dim() != 2:
        raise ValueError("x must be [B, T, D] and weight [D, W]")
    dev, dt, D, W = x.device, x.dtype, x.shape[2], weight.shape[1]
    N, T = _sequences(x.shape[:2], cu_seqlens, dev)
    stride = _rows(x, "x", dt, dev, x.shape)
    _param(weight, "weight", dev, (D, W))
    _param(bias, "bias", dev, (D,))
    states = (N, W - 1, D)
    if s0 is not None:
        _need(s0, "s0", dt, dev, states)
    if y is None:
        y = torch.empty(x.shape, dtype=dt, device=dev)
    else:
        _need(y, "y", dt, dev, x.shape)
    if sT is not None:
        _need(sT, "sT", dt, dev, states)
    elif output_final_state and W > 1:
        sT = torch.empty(states, dtype=dt, device=dev)
    _call("gdn_short_conv_fwd" + suffix, dev, stream, _ptr(x), _ptr(weight), _ptr(bias), _ptr(s0),
          _ptr(y), _ptr(sT), N, T, D, W, stride, _act(activation), _ptr(cu_seqlens))
    return y, sT


def gdn_short_conv_step(x, weight, s, bias=None, y=None, *, activation: Optional[str] = "silu",
                        stream=None):
    """One token of the short convolution; shifts s [N, W-1, D] in place, returns y.

    x [N, D] (may be a slice of a wider projection); weight, bias and activation as in
    gdn_short_conv_fwd.
    """
    suffix = _kind(x, "x")
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x must be [N, D] and weight [D, W]")
    dev, dt = x.device, x.dtype
    N, D = x.shape
    W = weight.shape[1]
    stride = _rows(x, "x", dt, dev, x.shape)
    _param(weight, "weight", dev, (D, W))
    _param(bias, "bias", dev, (D,))
    _need(s, "s", dt, dev, (N, W - 1, D))
    if y is None:
        y = torch.empty((N, D), dtype=dt, device=dev)
    else:
        _need(y, "y", dt, dev, (N, D))
    _call("gdn_short_conv_step" + suffix, dev, stream, _ptr(x), _ptr(weight), _ptr(bias), _ptr(s),
          _ptr(y), N, D, W, stride, _act(activation))
    return y


def gdn_s6_chunk_fwd_workspace_size(N, T, dim, Ns, varlen=False) -> int:
    """Bytes of workspace the S6 scan needs (0: none, or rejected sizes)."""
    return int(load_library().gdn_s6_chunk_fwd_workspace_size(N, T, dim, Ns, int(bool(varlen))))


def _s6_rows(x, dt, A, B, C, D, z, dt_bias):
    """Checks what the scan and its step share; returns (suffix, dim, Ns, strides)."""
    suffix = _kind(x, "x")
    if A.dim() != 2:
        raise ValueError("A must be [D, Ns]")
    dev, ty = x.device, x.dtype
    dim, Ns = x.shape[-1], A.shape[1]
    lead = tuple(x.shape[:-1])
    xs = _rows(x, "x", ty, dev, x.shape)
    ds = _rows(dt, "dt", ty, dev, x.shape)
    bs = _rows(B, "B", ty, dev, lead + (Ns,))
    cs = _rows(C, "C", ty, dev, lead + (Ns,))
    zs = 0 if z is None else _rows(z, "z", ty, dev, x.shape)
    _param(A, "A", dev, (dim, Ns))
    _param(D, "D", dev, (dim,))
    _param(dt_bias, "dt_bias", dev, (dim,))
    return suffix, dim, Ns, (xs, ds, bs, cs, zs)


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
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D]")
    suffix, dim, Ns, strides = _s6_rows(x, dt, A, B, C, D, z, dt_bias)
    dev = x.device
    N, T = _sequences(x.shape[:2], cu_seqlens, dev)
    states = (N, dim, Ns)
    _param(h0, "h0", dev, states)
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    else:
        _need(y, "y", x.dtype, dev, x.shape)
    if hT is not None:
        _need(hT, "hT", torch.float32, dev, states)
    elif output_final_state:
        hT = torch.empty(states, dtype=torch.float32, device=dev)
    if workspace is None:
        need = gdn_s6_chunk_fwd_workspace_size(N, T, dim, Ns, cu_seqlens is not None)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _need(workspace, "workspace", torch.uint8, dev)
    _call("gdn_s6_chunk_fwd" + suffix, dev, stream, _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C),
          _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(h0), _ptr(y), _ptr(hT), N, T, dim, Ns, *strides,
          int(bool(dt_softplus)), _ptr(cu_seqlens), _ptr(workspace),
          0 if workspace is None else workspace.numel())
    return y, hT


def gdn_s6_recurrent_step(x, dt, A, B, C, h, D=None, z=None, dt_bias=None, y=None, *,
                          dt_softplus: bool = False, stream=None):
    """One token of the S6 recurrence; updates h [N, D, Ns] in place and returns y.

    x, dt, z [N, D]; B, C [N, Ns]; the rest as in gdn_s6_chunk_fwd.
    """
    if x.dim() != 2:
        raise ValueError("x must be [N, D]")
    suffix, dim, Ns, strides = _s6_rows(x, dt, A, B, C, D, z, dt_bias)
    dev, N = x.device, x.shape[0]
    _need(h, "h", torch.float32, dev, (N, dim, Ns))
    if y is None:
        y = torch.empty((N, dim), dtype=x.dtype, device=dev)
    else:
        _need(y, "y", x.dtype, dev, (N, dim))
    _call("gdn_s6_recurrent_step" + suffix, dev, stream, _ptr(x), _ptr(dt), _ptr(A), _ptr(B),
          _ptr(C), _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(h), _ptr(y), N, dim, Ns, *strides,
          int(bool(dt_softplus)))
    return y


def gdn_rms_norm_fwd(x, weight, residual=None, gate=None, y=None, residual_out=None, scales=None, *,
                     eps: float = 1e-6, out_dtype=None, group: Optional[int] = None, stream=None):
    """RMS norm of the rows of x [..., D]; returns (y, scales, residual_out).

    r = x + residual; y = r / sqrt(mean(r^2) + eps) * weight * silu(gate).  x, residual, gate
    are bf16 or fp32, all the same; weight [D] fp32.  x and gate may be slices: rows a
    constant stride apart, or [..., H, D] with dense H D and a constant stride before it.  residual is contiguous and residual_out (a fresh tensor, or residual itself:
    in place) takes r in x's type.  out_dtype torch.float8_e4m3fn gives y in 8 bits with fp32
    scales [..., ceil(D / group)], one per ``group`` (32, 64, 128) columns or one a row (None):
    scale = max|y| / 448 (1 for zeros).  scales and residual_out are None where there are none.
    """
    suffix = _kind(x, "x")
    if x.dim() < 1:
        raise ValueError("x must be [..., D]")
    dev, dt, D = x.device, x.dtype, x.shape[-1]
    fp8 = out_dtype == _E4M3
    if not fp8 and out_dtype not in (None, dt):
        raise TypeError(f"out_dtype must be {dt} or {_E4M3}, got {out_dtype}")
    if group is not None and not fp8:
        raise ValueError("group applies to the e4m3 output")
    if fp8 and group not in (None, 32, 64, 128):
        raise ValueError(f"group must be 32, 64, 128 or None, got {group!r}")
    _param(weight, "weight", dev, (D,))
    _typed(x, "x", dt, dev, x.shape)
    if gate is not None:
        _typed(gate, "gate", dt, dev, x.shape)
    # rows a constant stride apart, or [..., H, D] whose tokens (H D dense) are
    heads, inner = 1, 1
    xs, gs = _stride_of(x), 0 if gate is None else _stride_of(gate)
    if (xs is None or gs is None) and x.dim() > 1:
        heads, inner = x.shape[-2], 2
        xs, gs = _stride_of(x, 2), 0 if gate is None else _stride_of(gate, 2)
    for s, t, name in ((xs, x, "x"), (gs, gate, "gate")):
        if s is None:
            raise ValueError(f"{name} with strides {t.stride()}: tokens must be dense and a constant "
                             "stride apart")
    tokens = 1
    for n in x.shape[:-inner]:
        tokens *= n
    if x.numel() == 0:
        tokens, heads = 0, 1
    if y is None:
        y = torch.empty(x.shape, dtype=_E4M3 if fp8 else dt, device=dev)
    else:
        _need(y, "y", _E4M3 if fp8 else dt, dev, x.shape)
    if residual is not None:
        _need(residual, "residual", dt, dev, x.shape)
        if residual_out is None:
            residual_out = torch.empty(x.shape, dtype=dt, device=dev)
        else:
            _need(residual_out, "residual_out", dt, dev, x.shape)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    args = (_ptr(x), _ptr(weight), _ptr(residual), _ptr(gate), _ptr(y))
    if fp8:
        parts = x.shape[:-1] + (-(-D // group) if group else 1,)
        if scales is None:
            scales = torch.empty(parts, dtype=torch.float32, device=dev)
        else:
            _need(scales, "scales", torch.float32, dev, parts)
        _call("gdn_rms_norm_fwd_e4m3" + suffix, dev, stream, *args, _ptr(scales),
              _ptr(residual_out), tokens, heads, D, xs, gs, group or 0, float(eps))
    else:
        if scales is not None:
            raise ValueError("scales belong to the e4m3 output")
        _call("gdn_rms_norm_fwd" + suffix, dev, stream, *args, _ptr(residual_out), tokens, heads, D,
              xs, gs, float(eps))
    return y, scales, residual_out
