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

from .binding import _check, _need, load_library

# A decode step takes a few microseconds on the GPU, and so do its checks here: they are
# written for the call that passes, one expression a tensor, with the reasons in _refuse.
_Tensor = torch.Tensor
_BF16, _F32, _E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream
_FN = {}  # (C name, type of the rows) -> library function


def _function(name: str, dtype):
    fn = _FN[name, dtype] = getattr(load_library(), name + ("_f32" if dtype is _F32 else ""))
    return fn


def _call(name: str, dtype, index: int, args):
    """One library call on the current stream of device ``index``, with it as the current one."""
    fn = _FN.get((name, dtype)) or _function(name, dtype)
    if _current_device() == index:
        status = fn(*args, _current_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _current_stream(index))
    if status:
        _check(status)


def _on(stream, x):
    """``stream`` (a torch stream, or a cudaStream_t as a number) as the current one: the call's
    own allocations belong to the stream that it runs on."""
    if not isinstance(stream, torch.cuda.Stream):
        if not isinstance(x, _Tensor) or x.get_device() < 0:
            raise ValueError("a stream needs operands on a CUDA device")
        stream = (torch.cuda.ExternalStream(int(stream), device=x.device) if int(stream) else
                  torch.cuda.default_stream(x.device))
    return torch.cuda.stream(stream)


def _kind(x, name: str, dims: int):
    """(type, device index) of the operand that sets them: bf16 or fp32, on a GPU."""
    if not isinstance(x, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dtype, index = x.dtype, x.get_device()
    if index < 0:
        raise ValueError(f"{name} must be on a CUDA device")
    if dtype is not _BF16 and dtype is not _F32:
        raise TypeError(f"{name} must be bf16 or fp32, got {dtype}")
    if x.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {tuple(x.shape)}")
    return dtype, index


def _refuse(t, name: str, dtype, index: int, shape, dense: bool = True):
    """Raises what is wrong with ``t``."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous" if dense else
                     f"{name} with strides {t.stride()}: the last dimension must be dense and tokens "
                     "a constant stride apart")


def _dense(t, name: str, dtype, index: int, shape) -> int:
    """Address of a contiguous operand of that type, device and shape."""
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == index
            and t.shape == shape and t.is_contiguous()):
        _refuse(t, name, dtype, index, shape)
    return t.data_ptr()


def _output(t, name: str, like, dtype, index: int, shape):
    """(address, tensor) of an output: the caller's, or a fresh one on the device of ``like``."""
    if t is None:
        t = torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format)
        return t.data_ptr(), t
    return _dense(t, name, dtype, index, shape), t


def _maybe(t, name: str, dtype, index: int, shape):
    return None if t is None else _dense(t, name, dtype, index, shape)


def _rows(t, name: str, dtype, index: int, shape):
    """(address, elements from token to token) of a row operand [..., cols]."""
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == index
            and t.shape == shape):
        _refuse(t, name, dtype, index, shape)
    if t.is_contiguous():
        return t.data_ptr(), shape[-1]
    stride = _stride_of(t)
    if stride is None:
        _refuse(t, name, dtype, index, shape, dense=False)
    return t.data_ptr(), stride


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


def _sequences(shape, cu_seqlens, device):
    """(N, T, address of cu_seqlens) of a batch of shape [B, T, ...]."""
    if cu_seqlens is None:
        return shape[0], shape[1], None
    _need(cu_seqlens, "cu_seqlens", torch.int32, device)
    if shape[0] != 1:
        raise ValueError("with cu_seqlens the batch must be one packed row (B == 1)")
    n = cu_seqlens.numel() - 1
    if n < 1:
        raise ValueError("cu_seqlens needs at least one sequence")
    return n, shape[1], cu_seqlens.data_ptr()


def _act(activation) -> int:
    if activation == "silu":
        return 1
    if activation is None:
        return 0
    raise ValueError(f"activation must be 'silu' or None, got {activation!r}")


def _taps(weight, index: int, D: int):
    """(address, W) of the filters [D, W]."""
    if not isinstance(weight, _Tensor) or weight.dim() != 2:
        raise (ValueError if isinstance(weight, _Tensor) else TypeError)("weight must be a tensor [D, W]")
    W = weight.shape[1]
    return _dense(weight, "weight", _F32, index, (D, W)), W


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
    dtype, index = _kind(x, "x", 3)
    shape = x.shape
    D = shape[2]
    w, W = _taps(weight, index, D)
    N, T, cu = _sequences(shape, cu_seqlens, x.device)
    xp, stride = _rows(x, "x", dtype, index, shape)
    states = (N, W - 1, D)
    yp, y = _output(y, "y", x, dtype, index, shape)
    if sT is None and output_final_state and W > 1:
        sT = torch.empty(states, dtype=dtype, device=x.device)
    _call("gdn_short_conv_fwd", dtype, index,
          (xp, w, _maybe(bias, "bias", _F32, index, (D,)), _maybe(s0, "s0", dtype, index, states),
           yp, _maybe(sT, "sT", dtype, index, states), N, T, D, W, stride, _act(activation), cu))
    return y, sT


def gdn_short_conv_step(x, weight, s, bias=None, y=None, *, activation: Optional[str] = "silu",
                        stream=None):
    """One token of the short convolution; shifts s [N, W-1, D] in place, returns y.

    x [N, D] (may be a slice of a wider projection); weight, bias and activation as in
    gdn_short_conv_fwd.
    """
    if stream is not None:
        with _on(stream, x):
            return gdn_short_conv_step(x, weight, s, bias, y, activation=activation)
    dtype, index = _kind(x, "x", 2)
    shape = x.shape
    N, D = shape
    w, W = _taps(weight, index, D)
    xp, stride = _rows(x, "x", dtype, index, shape)
    sp = _dense(s, "s", dtype, index, (N, W - 1, D))
    yp, y = _output(y, "y", x, dtype, index, shape)
    _call("gdn_short_conv_step", dtype, index,
          (xp, w, _maybe(bias, "bias", _F32, index, (D,)), sp, yp, N, D, W, stride,
           _act(activation)))
    return y


def gdn_s6_chunk_fwd_workspace_size(N, T, dim, Ns, varlen=False) -> int:
    """Bytes of workspace the S6 scan needs (0: none, or rejected sizes)."""
    return int(load_library().gdn_s6_chunk_fwd_workspace_size(N, T, dim, Ns, int(bool(varlen))))


def _s6_rows(x, dt, A, B, C, D, z, dt_bias, dims: int):
    """Checks what the scan and its step share; returns (type, device, dim, Ns, addresses
    x, dt, A, B, C, D, z, dt_bias, strides x, dt, B, C, z)."""
    dtype, index = _kind(x, "x", dims)
    shape = x.shape
    dim = shape[-1]
    if not isinstance(A, _Tensor) or A.dim() != 2:
        raise (ValueError if isinstance(A, _Tensor) else TypeError)("A must be a tensor [D, Ns]")
    Ns = A.shape[1]
    states = shape[:-1] + (Ns,)
    xp, xs = _rows(x, "x", dtype, index, shape)
    dp, ds = _rows(dt, "dt", dtype, index, shape)
    bp, bs = _rows(B, "B", dtype, index, states)
    cp, cs = _rows(C, "C", dtype, index, states)
    zp, zs = (None, 0) if z is None else _rows(z, "z", dtype, index, shape)
    return dtype, index, dim, Ns, (
        xp, dp, _dense(A, "A", _F32, index, (dim, Ns)), bp, cp, _maybe(D, "D", _F32, index, (dim,)), zp,
        _maybe(dt_bias, "dt_bias", _F32, index, (dim,))), (xs, ds, bs, cs, zs)


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
    dtype, index, dim, Ns, ptrs, strides = _s6_rows(x, dt, A, B, C, D, z, dt_bias, 3)
    N, T, cu = _sequences(x.shape, cu_seqlens, x.device)
    states = (N, dim, Ns)
    yp, y = _output(y, "y", x, dtype, index, x.shape)
    if hT is None and output_final_state:
        hT = torch.empty(states, dtype=_F32, device=x.device)
    if workspace is None:
        need = gdn_s6_chunk_fwd_workspace_size(N, T, dim, Ns, cu is not None)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    else:
        _need(workspace, "workspace", torch.uint8, x.device)
    _call("gdn_s6_chunk_fwd", dtype, index,
          (*ptrs, _maybe(h0, "h0", _F32, index, states), yp, _maybe(hT, "hT", _F32, index, states), N, T, dim, Ns, *strides, int(bool(dt_softplus)), cu,
           None if workspace is None else workspace.data_ptr(),
           0 if workspace is None else workspace.numel()))
    return y, hT


def gdn_s6_recurrent_step(x, dt, A, B, C, h, D=None, z=None, dt_bias=None, y=None, *,
                          dt_softplus: bool = False, stream=None):
    """One token of the S6 recurrence; updates h [N, D, Ns] in place and returns y.

    x, dt, z [N, D]; B, C [N, Ns]; the rest as in gdn_s6_chunk_fwd.
    """
    if stream is not None:
        with _on(stream, x):
            return gdn_s6_recurrent_step(x, dt, A, B, C, h, D, z, dt_bias, y, dt_softplus=dt_softplus)
    dtype, index, dim, Ns, ptrs, strides = _s6_rows(x, dt, A, B, C, D, z, dt_bias, 2)
    shape = x.shape
    N = shape[0]
    hp = _dense(h, "h", _F32, index, (N, dim, Ns))
    yp, y = _output(y, "y", x, dtype, index, shape)
    _call("gdn_s6_recurrent_step", dtype, index,
          (*ptrs, hp, yp, N, dim, Ns, *strides,
           int(bool(dt_softplus))))
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
    if stream is not None:
        with _on(stream, x):
            return gdn_rms_norm_fwd(x, weight, residual, gate, y, residual_out, scales, eps=eps,
                                    out_dtype=out_dtype, group=group)
    dtype, index = _kind(x, "x", x.dim() if isinstance(x, _Tensor) and x.dim() else 1)
    shape = x.shape
    D = shape[-1]
    fp8 = out_dtype is _E4M3
    if fp8:
        if group not in (None, 32, 64, 128):
            raise ValueError(f"group must be 32, 64, 128 or None, got {group!r}")
    else:
        if out_dtype is not None and out_dtype != dtype:
            raise TypeError(f"out_dtype must be {dtype} or {_E4M3}, got {out_dtype}")
        if group is not None or scales is not None:
            raise ValueError("group and scales belong to the e4m3 output")
    wp = _dense(weight, "weight", _F32, index, (D,))
    # rows a constant stride apart, or [..., H, D] whose tokens (H D dense) are
    heads, xs, gs, gp = 1, D, D, None
    strided = not x.is_contiguous()
    if gate is not None:
        if not (isinstance(gate, _Tensor) and gate.dtype is dtype and gate.get_device() == index
                and gate.shape == shape):
            _refuse(gate, "gate", dtype, index, shape)
        gp = gate.data_ptr()
        strided = strided or not gate.is_contiguous()
    rows = x.numel() // D if D else 0
    if strided and rows:
        xs, gs = _stride_of(x), 0 if gate is None else _stride_of(gate)
        if (xs is None or gs is None) and x.dim() > 1:
            heads = shape[-2]
            xs, gs = _stride_of(x, 2), 0 if gate is None else _stride_of(gate, 2)
        if xs is None:
            _refuse(x, "x", dtype, index, shape, dense=False)
        if gs is None:
            _refuse(gate, "gate", dtype, index, shape, dense=False)
    yp, y = _output(y, "y", x, _E4M3 if fp8 else dtype, index, shape)
    rp = op = None
    if residual is not None:
        rp = _dense(residual, "residual", dtype, index, shape)
        op, residual_out = _output(residual_out, "residual_out", residual, dtype, index, shape)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if fp8:
        parts = shape[:-1] + (-(-D // group) if group else 1,)
        if scales is None:
            scales = torch.empty(parts, dtype=_F32, device=x.device)
        _call("gdn_rms_norm_fwd_e4m3", dtype, index,
              (x.data_ptr(), wp, rp, gp, yp, _dense(scales, "scales", _F32, index, parts), op,
               rows // heads, heads, D, xs, gs, group or 0, eps))
    else:
        _call("gdn_rms_norm_fwd", dtype, index,
              (x.data_ptr(), wp, rp, gp, yp, op, rows // heads, heads, D, xs, gs, eps))
    return y, scales, residual_out
