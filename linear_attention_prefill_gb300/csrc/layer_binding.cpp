// layer_binding.cpp - the PyTorch binding of the layer operators as a Python extension
// (_layer_native), behind the functions of layer.py.
//
// A decode step takes a few microseconds on the GPU.  Checking its tensors and allocating its
// outputs from Python took the S6 step 17 us a call on the host, here it takes 3.5.  Argument
// marshalling only: types, devices, shapes and strides are checked, outputs allocated, the
// library's entry points called on the current stream.  The entry points' addresses and the
// raiser of their errors come from Python (init).
#include <Python.h>

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <sstream>
#include <string>

#include "../../include/gdn.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;
constexpr ScalarType kBf16 = ScalarType::BFloat16, kF32 = ScalarType::Float,
                     kE4m3 = ScalarType::Float8_e4m3fn;

// The library's entry points, bf16 and fp32 (the same arguments by address).
struct Library {
  decltype(&gdn_short_conv_fwd) conv[2];
  decltype(&gdn_short_conv_step) conv_step[2];
  decltype(&gdn_s6_chunk_fwd) s6[2];
  decltype(&gdn_s6_recurrent_step) s6_step[2];
  decltype(&gdn_s6_chunk_fwd_workspace_size) s6_workspace;
  decltype(&gdn_rms_norm_fwd) norm[2];
  decltype(&gdn_rms_norm_fwd_e4m3) norm8[2];
  decltype(&gdn_glr_chunk_fwd) glr[2];
  decltype(&gdn_glr_recurrent_step) glr_step[2];
  decltype(&gdn_glr_chunk_bwd) glr_bwd[2];
  decltype(&gdn_glr_chunk_bwd_workspace_size) glr_workspace;
  decltype(&gdn_layer_norm_fwd) ln[2];
  decltype(&gdn_layer_norm_bwd) ln_bwd[2];
  decltype(&gdn_layer_norm_bwd_workspace_size) ln_workspace;
  decltype(&gdn_rotary_fwd) rotary[2][2];  // forward, backward
} lib;
PyObject* raise_status = nullptr;  // called with a status that is not GDN_OK

// ---- refusals ------------------------------------------------------------------------
template <typename... Parts>
std::string text(const Parts&... parts) {
  std::ostringstream s;
  (s << ... << parts);
  return s.str();
}
struct Refusal {  // a Python error to raise
  PyObject* type;
  std::string what;
};
template <typename... Parts>
[[noreturn]] void type_error(const Parts&... parts) {
  throw Refusal{PyExc_TypeError, text(parts...)};
}
template <typename... Parts>
[[noreturn]] void value_error(const Parts&... parts) {
  throw Refusal{PyExc_ValueError, text(parts...)};
}

// ---- operands ------------------------------------------------------------------------
const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(name, " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

// The operand that sets type and device: bf16 or fp32, on a GPU.
struct Kind {
  ScalarType type;
  int device;
  int f32;
};
Kind kind_of(const Tensor& x, const char* name, int64_t dims) {
  if (!x.is_cuda()) value_error(name, " must be on a CUDA device");
  const ScalarType t = x.scalar_type();
  if (t != kBf16 && t != kF32) type_error(name, " must be bf16 or fp32, got ", t);
  if (dims >= 0 ? x.dim() != dims : x.dim() < 1)
    value_error(name, " must have ", dims >= 0 ? dims : 1, " dimensions, got ", x.sizes());
  return {t, x.get_device(), t == kF32};
}

void typed(const Tensor& t, const char* name, ScalarType type, int device, IntArrayRef shape) {
  if (t.scalar_type() != type) type_error(name, " must be ", type, ", got ", t.scalar_type());
  if (!t.is_cuda() || t.get_device() != device)
    value_error(name, " is on ", t.device(), ", expected cuda:", device);
  if (t.sizes() != shape) value_error(name, " has shape ", t.sizes(), ", expected ", shape);
}
void* dense(const Tensor& t, const char* name, ScalarType type, int device, IntArrayRef shape) {
  typed(t, name, type, device, shape);
  if (!t.is_contiguous()) value_error(name, " must be contiguous");
  return t.data_ptr();
}
void* dense(PyObject* o, const char* name, ScalarType type, int device, IntArrayRef shape) {
  return dense(tensor(o, name), name, type, device, shape);
}
void* maybe(PyObject* o, const char* name, ScalarType type, int device, IntArrayRef shape) {
  return o == Py_None ? nullptr : dense(o, name, type, device, shape);
}
const float* param(PyObject* o, const char* name, int device, IntArrayRef shape) {
  return static_cast<const float*>(maybe(o, name, kF32, device, shape));
}

// Elements from token to token of t, whose last `inner` dimensions are one dense token and
// whose others lie a constant stride apart; -1 if they do not.
int64_t stride_of(const Tensor& t, int64_t inner) {
  const IntArrayRef shape = t.sizes(), strides = t.strides();
  const int64_t split = t.dim() - inner;
  int64_t cols = 1;
  if (t.numel() == 0) {
    for (int64_t i = split; i < t.dim(); ++i) cols *= shape[i];
    return cols < 1 ? 1 : cols;
  }
  for (int64_t i = t.dim() - 1; i >= split; --i) {
    if (shape[i] != 1 && strides[i] != cols) return -1;
    cols *= shape[i];
  }
  int64_t stride = cols, seen = 1;
  for (int64_t i = split - 1; i >= 0; --i) {
    if (shape[i] == 1) continue;
    if (seen == 1) stride = strides[i];
    else if (strides[i] != stride * seen) return -1;
    seen *= shape[i];
  }
  return stride >= cols || seen <= 1 ? stride : -1;
}
[[noreturn]] void bad_strides(const Tensor& t, const char* name) {
  value_error(name, " with strides ", t.strides(),
              ": the last dimension must be dense and tokens a constant stride apart");
}
struct Rows {
  const void* p = nullptr;
  int64_t stride = 0;
};
Rows rows(PyObject* o, const char* name, ScalarType type, int device, IntArrayRef shape) {
  const Tensor& t = tensor(o, name);
  typed(t, name, type, device, shape);
  const int64_t stride = stride_of(t, 1);
  if (stride < 0) bad_strides(t, name);
  return {t.data_ptr(), stride};
}

// A tensor from torch's allocator, on the device's current stream.
Tensor fresh(IntArrayRef shape, ScalarType type, int device) {
  return Tensor(at::detail::empty_cuda(
      shape, type, c10::Device(c10::DeviceType::CUDA, (c10::DeviceIndex)device), std::nullopt));
}

// An output: the caller's, or a fresh one.  `object` is a new reference.
struct Output {
  void* p;
  PyObject* object;
};
PyObject* wrap(Tensor t) {
  PyObject* o = THPVariable_Wrap(std::move(t));
  if (!o) throw python_error();
  return o;
}
Output output(PyObject* o, const char* name, ScalarType type, int device, IntArrayRef shape) {
  if (o != Py_None) {
    void* p = dense(o, name, type, device, shape);
    Py_INCREF(o);
    return {p, o};
  }
  Tensor t = fresh(shape, type, device);
  void* p = t.data_ptr();
  return {p, wrap(std::move(t))};
}
// A reference that is dropped when a refusal passes it.
struct Held {
  PyObject* o;
  explicit Held(PyObject* o) : o(o) {}
  Held(const Held&) = delete;
  ~Held() { Py_XDECREF(o); }
  PyObject* take() {
    PyObject* r = o;
    o = nullptr;
    return r;
  }
};

// (N, T, cu_seqlens) of a batch of shape [B, T, ...].
struct Batch {
  int n, t;
  const int32_t* cu;
};
int small(int64_t v, const char* what) {
  if (v < 0 || v > 0x7fffffff) value_error(what, " = ", v, " is out of range");
  return (int)v;
}
Batch batch_of(IntArrayRef shape, PyObject* cu, int device) {
  if (cu == Py_None) return {small(shape[0], "the batch"), small(shape[1], "T"), nullptr};
  const Tensor& t = tensor(cu, "cu_seqlens");
  typed(t, "cu_seqlens", ScalarType::Int, device, t.sizes());
  if (t.dim() != 1 || !t.is_contiguous()) value_error("cu_seqlens must be one contiguous row");
  if (shape[0] != 1) value_error("with cu_seqlens the batch must be one packed row (B == 1)");
  if (t.numel() < 2) value_error("cu_seqlens needs at least one sequence");
  return {small(t.numel() - 1, "the batch"), small(shape[1], "T"),
          static_cast<const int32_t*>(t.data_ptr())};
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

gdn_stream_t stream_of(int device) {
  return reinterpret_cast<gdn_stream_t>(c10::cuda::getCurrentCUDAStream(device).stream());
}
// Runs `call` with the interpreter released; raises what the library reports.
template <typename Call>
void run(int device, Call call) {
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
  const gdn_stream_t stream = stream_of(device);
  gdn_status s;
  Py_BEGIN_ALLOW_THREADS s = call(stream);
  Py_END_ALLOW_THREADS
  if (s == GDN_OK) return;
  PyObject* r = PyObject_CallFunction(raise_status, "i", (int)s);
  Py_XDECREF(r);
  if (r) PyErr_Format(PyExc_RuntimeError, "status %d", (int)s);
  throw python_error();
}

// ---- short convolution -----------------------------------------------------------------
// filters [D, W]
const float* taps(PyObject* o, int device, int64_t D, int* W) {
  const Tensor& t = tensor(o, "weight");
  if (t.dim() != 2) value_error("weight must be [D, W], got ", t.sizes());
  *W = small(t.size(1), "W");
  return static_cast<const float*>(dense(t, "weight", kF32, device, {D, t.size(1)}));
}

// x, weight, bias, s0, y, sT, activation, cu_seqlens, output_final_state
PyObject* conv_fwd(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  const Kind k = kind_of(x, "x", 3);
  const IntArrayRef shape = x.sizes();
  const int D = small(shape[2], "D");
  int W;
  const float* w = taps(a[1], k.device, D, &W);
  const Batch b = batch_of(shape, a[7], k.device);
  const Rows xr = rows(a[0], "x", k.type, k.device, shape);
  const int64_t states[3] = {b.n, W - 1, D};
  const float* bias = param(a[2], "bias", k.device, {D});
  const void* s0 = maybe(a[3], "s0", k.type, k.device, states);
  const int act = (int)PyLong_AsLong(a[6]);
  const Output y = output(a[4], "y", k.type, k.device, shape);
  Held hy(y.object);
  const bool state = W > 1 && (a[5] != Py_None || truth(a[8]));
  const Output sT = state ? output(a[5], "sT", k.type, k.device, states)
                          : Output{nullptr, (Py_INCREF(Py_None), Py_None)};
  Held hs(sT.object);
  run(k.device, [&](gdn_stream_t st) {
    return lib.conv[k.f32](xr.p, w, bias, s0, y.p, sT.p, b.n, b.t, D, W, xr.stride, act, b.cu, st);
  });
  PyObject* r = PyTuple_New(2);
  if (!r) throw python_error();
  PyTuple_SET_ITEM(r, 0, hy.take());
  PyTuple_SET_ITEM(r, 1, hs.take());
  return r;
}

// x, weight, s, bias, y, activation
PyObject* conv_step(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  const Kind k = kind_of(x, "x", 2);
  const IntArrayRef shape = x.sizes();
  const int64_t N = shape[0];
  const int D = small(shape[1], "D");
  int W;
  const float* w = taps(a[1], k.device, D, &W);
  const Rows xr = rows(a[0], "x", k.type, k.device, shape);
  void* s = dense(a[2], "s", k.type, k.device, {N, W - 1, D});
  const float* bias = param(a[3], "bias", k.device, {D});
  const int act = (int)PyLong_AsLong(a[5]), n = small(N, "the batch");
  const Output y = output(a[4], "y", k.type, k.device, shape);
  Held hy(y.object);
  run(k.device, [&](gdn_stream_t st) {
    return lib.conv_step[k.f32](xr.p, w, bias, s, y.p, n, D, W, xr.stride, act, st);
  });
  return hy.take();
}

// ---- S6 --------------------------------------------------------------------------------
// What the scan and its step share: x, dt, A, B, C, D, z, dt_bias at a[0..7].
struct S6 {
  Kind k;
  int64_t dim, Ns;
  Rows x, dt, B, C, z;
  const float *A, *D, *bias;
};
S6 s6_operands(PyObject* const* a, int64_t dims) {
  S6 s;
  const Tensor& x = tensor(a[0], "x");
  s.k = kind_of(x, "x", dims);
  const IntArrayRef shape = x.sizes();
  s.dim = shape[dims - 1];
  const Tensor& A = tensor(a[2], "A");
  if (A.dim() != 2) value_error("A must be [D, Ns], got ", A.sizes());
  s.Ns = A.size(1);
  const int dev = s.k.device;
  s.A = static_cast<const float*>(dense(A, "A", kF32, dev, {s.dim, s.Ns}));
  int64_t states[3] = {shape[0], dims == 3 ? shape[1] : s.Ns, s.Ns};
  const IntArrayRef bc(states, dims);
  s.x = rows(a[0], "x", s.k.type, dev, shape);
  s.dt = rows(a[1], "dt", s.k.type, dev, shape);
  s.B = rows(a[3], "B", s.k.type, dev, bc);
  s.C = rows(a[4], "C", s.k.type, dev, bc);
  if (a[6] != Py_None) s.z = rows(a[6], "z", s.k.type, dev, shape);
  s.D = param(a[5], "D", dev, {s.dim});
  s.bias = param(a[7], "dt_bias", dev, {s.dim});
  return s;
}

// x, dt, A, B, C, D, z, dt_bias, h0, y, hT, dt_softplus, cu_seqlens, output_final_state, workspace
PyObject* s6_fwd(PyObject* const* a) {
  const S6 s = s6_operands(a, 3);
  const int dev = s.k.device;
  const IntArrayRef shape = tensor(a[0], "x").sizes();
  const Batch b = batch_of(shape, a[12], dev);
  const int64_t states[3] = {b.n, s.dim, s.Ns};
  const float* h0 = param(a[8], "h0", dev, states);
  const int softplus = truth(a[11]), dim = small(s.dim, "D"), Ns = small(s.Ns, "Ns");
  const Output y = output(a[9], "y", s.k.type, dev, shape);
  Held hy(y.object);
  const Output hT = a[10] != Py_None || truth(a[13]) ? output(a[10], "hT", kF32, dev, states)
                                                     : Output{nullptr, (Py_INCREF(Py_None), Py_None)};
  Held hh(hT.object);
  Tensor scratch;  // given back to the allocator of this stream when the call is enqueued
  void* ws = nullptr;
  size_t bytes = 0;
  if (a[14] != Py_None) {
    const Tensor& t = tensor(a[14], "workspace");
    ws = dense(t, "workspace", ScalarType::Byte, dev, t.sizes());
    bytes = (size_t)t.numel();
  } else if ((bytes = lib.s6_workspace(b.n, b.t, dim, Ns, b.cu != nullptr)) != 0) {
    scratch = fresh({(int64_t)bytes}, ScalarType::Byte, dev);
    ws = scratch.data_ptr();
  }
  run(dev, [&](gdn_stream_t st) {
    return lib.s6[s.k.f32](s.x.p, s.dt.p, s.A, s.B.p, s.C.p, s.D, s.z.p, s.bias, h0, y.p,
                           static_cast<float*>(hT.p), b.n, b.t, dim, Ns, s.x.stride, s.dt.stride,
                           s.B.stride, s.C.stride, s.z.stride, softplus, b.cu, ws, bytes, st);
  });
  PyObject* r = PyTuple_New(2);
  if (!r) throw python_error();
  PyTuple_SET_ITEM(r, 0, hy.take());
  PyTuple_SET_ITEM(r, 1, hh.take());
  return r;
}

// x, dt, A, B, C, D, z, dt_bias, h, y, dt_softplus
PyObject* s6_step(PyObject* const* a) {
  const S6 s = s6_operands(a, 2);
  const int dev = s.k.device;
  const IntArrayRef shape = tensor(a[0], "x").sizes();
  float* h = static_cast<float*>(dense(a[8], "h", kF32, dev, {shape[0], s.dim, s.Ns}));
  const int softplus = truth(a[10]), n = small(shape[0], "the batch");
  const int dim = small(s.dim, "D"), Ns = small(s.Ns, "Ns");
  const Output y = output(a[9], "y", s.k.type, dev, shape);
  Held hy(y.object);
  run(dev, [&](gdn_stream_t st) {
    return lib.s6_step[s.k.f32](s.x.p, s.dt.p, s.A, s.B.p, s.C.p, s.D, s.z.p, s.bias, h, y.p, n, dim,
                                Ns, s.x.stride, s.dt.stride, s.B.stride, s.C.stride, s.z.stride,
                                softplus, st);
  });
  return hy.take();
}

// ---- RMS norm ----------------------------------------------------------------------------
// x, weight, residual, gate, y, residual_out, scales, eps, e4m3, group
PyObject* norm_fwd(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  const Kind k = kind_of(x, "x", -1);
  const int dev = k.device;
  const IntArrayRef shape = x.sizes();
  const int64_t D = shape[x.dim() - 1];
  const float* w = static_cast<const float*>(dense(a[1], "weight", kF32, dev, {D}));
  const bool e4m3 = truth(a[8]);
  const int group = (int)PyLong_AsLong(a[9]);
  const double eps = PyFloat_AsDouble(a[7]);
  if (eps == -1.0 && PyErr_Occurred()) throw python_error();
  const Tensor* gate = nullptr;
  if (a[3] != Py_None) {
    gate = &tensor(a[3], "gate");
    typed(*gate, "gate", k.type, dev, shape);
  }
  // rows a constant stride apart, or [..., H, D] whose tokens (H D dense) are
  int64_t heads = 1, xs = stride_of(x, 1), gs = gate ? stride_of(*gate, 1) : 0;
  if ((xs < 0 || gs < 0) && x.dim() > 1) {
    heads = shape[x.dim() - 2];
    xs = stride_of(x, 2);
    gs = gate ? stride_of(*gate, 2) : 0;
  }
  if (xs < 0) bad_strides(x, "x");
  if (gs < 0) bad_strides(*gate, "gate");
  const int64_t n = D ? x.numel() / D : 0, tokens = heads ? n / heads : 0;
  if (heads < 1) heads = 1;
  const Output y = output(a[4], "y", e4m3 ? kE4m3 : k.type, dev, shape);
  Held hy(y.object);
  const void* res = nullptr;
  Output out{nullptr, nullptr};
  if (a[2] != Py_None) {
    res = dense(a[2], "residual", k.type, dev, shape);
    out = output(a[5], "residual_out", k.type, dev, shape);
  } else {
    if (a[5] != Py_None) value_error("residual_out needs a residual");
    out.object = (Py_INCREF(Py_None), Py_None);
  }
  Held ho(out.object);
  Output sc{nullptr, nullptr};
  if (e4m3) {
    std::vector<int64_t> parts(shape.begin(), shape.end());
    parts.back() = group ? (D + group - 1) / group : 1;
    sc = output(a[6], "scales", kF32, dev, parts);
  } else {
    if (a[6] != Py_None) value_error("scales belong to the e4m3 output");
    sc.object = (Py_INCREF(Py_None), Py_None);
  }
  Held hs(sc.object);
  const void* g = gate ? gate->data_ptr() : nullptr;
  const int h = small(heads, "the heads"), d = small(D, "D");
  run(dev, [&](gdn_stream_t st) {
    return e4m3 ? lib.norm8[k.f32](x.data_ptr(), w, res, g, y.p, static_cast<float*>(sc.p), out.p,
                                   tokens, h, d, xs, gs, group, (float)eps, st)
                : lib.norm[k.f32](x.data_ptr(), w, res, g, y.p, out.p, tokens, h, d, xs, gs,
                                  (float)eps, st);
  });
  PyObject* r = PyTuple_New(3);
  if (!r) throw python_error();
  PyTuple_SET_ITEM(r, 0, hy.take());
  PyTuple_SET_ITEM(r, 1, hs.take());
  PyTuple_SET_ITEM(r, 2, ho.take());
  return r;
}

// ---- gated linear recurrence ---------------------------------------------------------------
PyObject* none() { return Py_INCREF(Py_None), Py_None; }
// The caller's output, or a fresh one where `wanted`, or None.
Output maybe_output(PyObject* o, bool wanted, const char* name, ScalarType type, int device, IntArrayRef shape) {
  return o != Py_None || wanted ? output(o, name, type, device, shape) : Output{nullptr, none()};
}
// A call's scratch: the caller's workspace, or one from the allocator of the current stream, to
// which it goes back when the call is enqueued.
struct Scratch {
  Tensor own;
  void* p = nullptr;
  size_t bytes = 0;
  Scratch(PyObject* o, size_t need, int device) {
    if (o != Py_None) {
      const Tensor& t = tensor(o, "workspace");
      p = dense(t, "workspace", ScalarType::Byte, device, t.sizes());
      bytes = (size_t)t.numel();
    } else if (need) {
      own = fresh({(int64_t)need}, ScalarType::Byte, device);
      p = own.data_ptr();
      bytes = need;
    }
  }
};
template <size_t n>
PyObject* tuple_of(Held* (&&held)[n]) {
  PyObject* r = PyTuple_New((Py_ssize_t)n);
  if (!r) throw python_error();
  for (size_t i = 0; i < n; ++i) PyTuple_SET_ITEM(r, (Py_ssize_t)i, held[i]->take());
  return r;
}

// x, g, rate, h0, y, hT, states, gate, input_norm, cu_seqlens, output_final_state, output_states
PyObject* glr_fwd(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  const Kind k = kind_of(x, "x", 3);
  const int dev = k.device;
  const IntArrayRef shape = x.sizes();
  const int D = small(shape[2], "D"), gate = (int)PyLong_AsLong(a[7]), norm = (int)PyLong_AsLong(a[8]);
  const Batch b = batch_of(shape, a[9], dev);
  const Rows xr = rows(a[0], "x", k.type, dev, shape), gr = rows(a[1], "g", k.type, dev, shape);
  const float* rate = param(a[2], "rate", dev, {D});
  const int64_t states[2] = {b.n, D}, kept[3] = {shape[0], (shape[1] + 63) / 64, D};
  const float* h0 = param(a[3], "h0", dev, states);
  const Output y = output(a[4], "y", k.type, dev, shape);
  Held hy(y.object);
  const Output hT = maybe_output(a[5], truth(a[10]), "hT", kF32, dev, states);
  Held hh(hT.object);
  const Output st = maybe_output(a[6], truth(a[11]), "states", kF32, dev, kept);
  Held hs(st.object);
  run(dev, [&](gdn_stream_t s) {
    return lib.glr[k.f32](xr.p, gr.p, rate, h0, y.p, static_cast<float*>(hT.p), static_cast<float*>(st.p), b.n, b.t, D,
                          xr.stride, gr.stride, gate, norm, b.cu, s);
  });
  return tuple_of({&hy, &hh, &hs});
}

// x, g, h, rate, y, gate, input_norm
PyObject* glr_step(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  const Kind k = kind_of(x, "x", 2);
  const int dev = k.device;
  const IntArrayRef shape = x.sizes();
  const int n = small(shape[0], "the batch"), D = small(shape[1], "D");
  const int gate = (int)PyLong_AsLong(a[5]), norm = (int)PyLong_AsLong(a[6]);
  const Rows xr = rows(a[0], "x", k.type, dev, shape), gr = rows(a[1], "g", k.type, dev, shape);
  float* h = static_cast<float*>(dense(a[2], "h", kF32, dev, shape));
  const float* rate = param(a[3], "rate", dev, {D});
  const Output y = output(a[4], "y", k.type, dev, shape);
  Held hy(y.object);
  run(dev, [&](gdn_stream_t s) {
    return lib.glr_step[k.f32](xr.p, gr.p, rate, h, y.p, n, D, xr.stride, gr.stride, gate, norm, s);
  });
  return hy.take();
}

// dy, x, g, states, rate, h0, dhT, dx, dg, drate, dh0, gate, input_norm, cu_seqlens, workspace
PyObject* glr_bwd(PyObject* const* a) {
  const Tensor& x = tensor(a[1], "x");
  const Kind k = kind_of(x, "x", 3);
  const int dev = k.device;
  const IntArrayRef shape = x.sizes();
  const int D = small(shape[2], "D"), gate = (int)PyLong_AsLong(a[11]), norm = (int)PyLong_AsLong(a[12]);
  const Batch b = batch_of(shape, a[13], dev);
  const Rows dr = rows(a[0], "dy", k.type, dev, shape), xr = rows(a[1], "x", k.type, dev, shape),
             gr = rows(a[2], "g", k.type, dev, shape);
  const int64_t states[2] = {b.n, D}, kept[3] = {shape[0], (shape[1] + 63) / 64, D};
  const float* st = static_cast<const float*>(dense(a[3], "states", kF32, dev, kept));
  const float *rate = param(a[4], "rate", dev, {D}), *h0 = param(a[5], "h0", dev, states),
              *dhT = param(a[6], "dhT", dev, states);
  if (a[4] == Py_None && a[9] != Py_None) value_error("drate needs a rate");
  const Output dx = output(a[7], "dx", k.type, dev, shape);
  Held hx(dx.object);
  const Output dg = output(a[8], "dg", k.type, dev, shape);
  Held hg(dg.object);
  const Output drate = maybe_output(a[9], a[4] != Py_None, "drate", kF32, dev, {D});
  Held hr(drate.object);
  const Output dh0 = maybe_output(a[10], a[5] != Py_None, "dh0", kF32, dev, states);
  Held hh(dh0.object);
  const Scratch ws(a[14], lib.glr_workspace(b.n, b.t, D, gate, b.cu != nullptr), dev);
  run(dev, [&](gdn_stream_t s) {
    return lib.glr_bwd[k.f32](dr.p, xr.p, gr.p, rate, h0, st, dhT, dx.p, dg.p, static_cast<float*>(drate.p),
                              static_cast<float*>(dh0.p), b.n, b.t, D, dr.stride, xr.stride, gr.stride, gate, norm,
                              b.cu, ws.p, ws.bytes, s);
  });
  return tuple_of({&hx, &hg, &hr, &hh});
}

// ---- layer norm ------------------------------------------------------------------------------
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

// x, weight, bias, residual, y, residual_out, eps
PyObject* ln_fwd(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  const Kind k = kind_of(x, "x", -1);
  const int dev = k.device;
  const IntArrayRef shape = x.sizes();
  const int D = small(shape[x.dim() - 1], "D");
  const Rows xr = rows(a[0], "x", k.type, dev, shape);
  const float *w = param(a[1], "weight", dev, {D}), *b = param(a[2], "bias", dev, {D});
  const float eps = (float)number(a[6]);
  const void* res = maybe(a[3], "residual", k.type, dev, shape);
  if (a[3] == Py_None && a[5] != Py_None) value_error("residual_out needs a residual");
  const Output y = output(a[4], "y", k.type, dev, shape);
  Held hy(y.object);
  const Output out = maybe_output(a[5], a[3] != Py_None, "residual_out", k.type, dev, shape);
  Held ho(out.object);
  const int64_t n = D ? x.numel() / D : 0;
  run(dev, [&](gdn_stream_t s) {
    return lib.ln[k.f32](xr.p, w, b, res, y.p, out.p, n, D, xr.stride, eps, s);
  });
  return tuple_of({&hy, &ho});
}

// dy, x, weight, dres, dx, dweight, dbias, eps, param_grads, workspace
PyObject* ln_bwd(PyObject* const* a) {
  const Tensor& x = tensor(a[1], "x");
  const Kind k = kind_of(x, "x", -1);
  const int dev = k.device;
  const IntArrayRef shape = x.sizes();
  const int D = small(shape[x.dim() - 1], "D");
  const Rows dr = rows(a[0], "dy", k.type, dev, shape), xr = rows(a[1], "x", k.type, dev, shape);
  const float* w = param(a[2], "weight", dev, {D});
  const void* res = maybe(a[3], "dres", k.type, dev, shape);
  const float eps = (float)number(a[7]);
  const bool grads = truth(a[8]);
  if (!grads && (a[5] != Py_None || a[6] != Py_None)) value_error("dweight and dbias belong to param_grads");
  const Output dx = output(a[4], "dx", k.type, dev, shape);
  Held hx(dx.object);
  const Output dw = maybe_output(a[5], grads, "dweight", kF32, dev, {D});
  Held hw(dw.object);
  const Output db = maybe_output(a[6], grads, "dbias", kF32, dev, {D});
  Held hb(db.object);
  const int64_t n = D ? x.numel() / D : 0;
  const Scratch ws(a[9], grads ? lib.ln_workspace(n, D) : 0, dev);
  run(dev, [&](gdn_stream_t s) {
    return lib.ln_bwd[k.f32](dr.p, xr.p, w, res, dx.p, static_cast<float*>(dw.p), static_cast<float*>(db.p), n, D,
                             dr.stride, xr.stride, eps, ws.p, ws.bytes, s);
  });
  return tuple_of({&hx, &hw, &hb});
}

// ---- rotary positions ------------------------------------------------------------------------
// A tensor of tokens of [H, D], tokens a constant stride apart.
Rows token_rows(const Tensor& t, const char* name) {
  const int64_t stride = stride_of(t, 2);
  if (stride < 0) value_error(name, " with strides ", t.strides(), ": a token's heads must be dense and tokens a "
                              "constant stride apart");
  return {t.data_ptr(), stride};
}
// q, k, turns, positions, q_out, k_out, magnitude, interleaved, cu_seqlens, offsets, backward
PyObject* rotary(PyObject* const* a) {
  const Tensor& q = tensor(a[0], "q");
  const Kind kind = kind_of(q, "q", -1);
  const int dev = kind.device;
  const IntArrayRef shape = q.sizes();
  if (q.dim() < 3) value_error("q must be [..., H, D] with tokens before, got ", shape);
  const int64_t lead = q.dim() - 2;
  const int Hq = small(shape[lead], "the heads"), D = small(shape[lead + 1], "D");
  int64_t tokens = 1;
  for (int64_t i = 0; i < lead; ++i) tokens *= shape[i];
  const Tensor& turns = tensor(a[2], "turns");
  if (turns.dim() != 1) value_error("turns must be one row, got ", turns.sizes());
  const auto* table = static_cast<const unsigned long long*>(
      dense(turns, "turns", ScalarType::Long, dev, turns.sizes()));
  const int R = small(2 * turns.numel(), "the rotated columns");
  const float magnitude = (float)number(a[6]);
  const int interleaved = truth(a[7]), backward = truth(a[10]);
  Batch b{1, small(tokens, "the tokens"), nullptr};
  const int32_t *positions = nullptr, *offsets = nullptr;
  if (a[3] != Py_None) {
    if (a[8] != Py_None || a[9] != Py_None)
      value_error("positions stand for themselves: neither cu_seqlens nor offsets with them");
    positions = static_cast<const int32_t*>(dense(a[3], "positions", ScalarType::Int, dev, shape.slice(0, lead)));
  } else {
    if (q.dim() != 4) value_error("without positions q must be [B, T, H, D], got ", shape);
    b = batch_of(shape, a[8], dev);
    offsets = static_cast<const int32_t*>(maybe(a[9], "offsets", ScalarType::Int, dev, {b.n}));
  }
  const Rows qr = token_rows(q, "q");
  Rows kr;
  int Hk = 0;
  std::vector<int64_t> kshape(shape.begin(), shape.end());
  if (a[1] != Py_None) {
    const Tensor& k = tensor(a[1], "k");
    if (k.dim() == q.dim()) kshape[lead] = k.size(lead);
    typed(k, "k", kind.type, dev, kshape);
    Hk = small(kshape[lead], "the heads of k");
    if (Hk < 1) value_error("k has no heads: give None");
    kr = token_rows(k, "k");
  } else if (a[5] != Py_None) {
    value_error("k_out needs a k");
  }
  // the caller's outputs may be strided, as q and k (in place: q and k themselves)
  const auto out = [&](PyObject* o, const char* name, IntArrayRef sizes, Rows* r) {
    if (o == Py_None) {
      Tensor t = fresh(sizes, kind.type, dev);
      *r = token_rows(t, name);
      return wrap(std::move(t));
    }
    typed(tensor(o, name), name, kind.type, dev, sizes);
    *r = token_rows(tensor(o, name), name);
    Py_INCREF(o);
    return o;
  };
  Rows qo, ko;
  Held hq(out(a[4], "q_out", shape, &qo));
  Held hk(Hk ? out(a[5], "k_out", kshape, &ko) : none());
  run(dev, [&](gdn_stream_t s) {
    return lib.rotary[backward][kind.f32](qr.p, kr.p, table, positions, offsets, b.cu, const_cast<void*>(qo.p),
                                          const_cast<void*>(ko.p), b.n, b.t, Hq, Hk, D, R, qr.stride, kr.stride,
                                          qo.stride, ko.stride, interleaved, magnitude, s);
  });
  return tuple_of({&hq, &hk});
}

// ---- the module ----------------------------------------------------------------------------
// Positional arguments only: layer.py has the signatures.
template <PyObject* (*kCall)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != kArgs || !raise_status) {
    PyErr_Format(PyExc_RuntimeError, "_layer_native: %d arguments of %d, or no init", (int)n, kArgs);
    return nullptr;
  }
  try {
    return kCall(args);
  } catch (const Refusal& r) {
    PyErr_SetString(r.type, r.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// init(addresses in Library's order, raiser)
PyObject* init(PyObject*, PyObject* args) {
  PyObject *addresses, *raiser;
  if (!PyArg_ParseTuple(args, "O!O", &PyTuple_Type, &addresses, &raiser)) return nullptr;
  constexpr size_t kCount = sizeof(Library) / sizeof(void*);
  if ((size_t)PyTuple_GET_SIZE(addresses) != kCount) {
    PyErr_Format(PyExc_ValueError, "%zu addresses expected", kCount);
    return nullptr;
  }
  void** to = reinterpret_cast<void**>(&lib);
  for (size_t i = 0; i < kCount; ++i) {
    to[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(addresses, (Py_ssize_t)i));
    if (!to[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "NULL entry point");
      return nullptr;
    }
  }
  Py_INCREF(raiser);
  Py_XDECREF(raise_status);
  raise_status = raiser;
  Py_RETURN_NONE;
}

#define ENTRY(name, call, count) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<call, count>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"init", init, METH_VARARGS, nullptr},
                         ENTRY("conv_fwd", conv_fwd, 9),
                         ENTRY("conv_step", conv_step, 6),
                         ENTRY("s6_fwd", s6_fwd, 15),
                         ENTRY("s6_step", s6_step, 11),
                         ENTRY("norm_fwd", norm_fwd, 10),
                         ENTRY("glr_fwd", glr_fwd, 12),
                         ENTRY("glr_step", glr_step, 7),
                         ENTRY("glr_bwd", glr_bwd, 15),
                         ENTRY("ln_fwd", ln_fwd, 7),
                         ENTRY("ln_bwd", ln_bwd, 10),
                         ENTRY("rotary", rotary, 11),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_native", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__layer_native(void) { return PyModule_Create(&module); }
