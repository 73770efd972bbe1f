// The Python binding of libcr's model operators: checks of the arguments,
// outputs, workspace and stream, then one C call (include/cr.h).
//
// A single-token call is a few microseconds on the device; taking the
// tensors apart in Python took three times that. Functions here take
// positional arguments only: model.py names, defaults and documents them.
// Nothing is computed here, and libcr is not linked: bind() gets the addresses
// of the functions that model.py has loaded.
#include <Python.h>

#include <array>
#include <cmath>
#include <cstdint>
#include <exception>
#include <initializer_list>
#include <optional>
#include <sstream>
#include <string>
#include <vector>

#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "cr.h"

namespace {

// ---------------------------------------------------------------- errors
struct Error {
  PyObject* type;  // nullptr: the Python error is set already
  std::string what;
};

template <class... A>
std::string join(const A&... a) {
  std::ostringstream s;
  (s << ... << a);
  return s.str();
}

[[noreturn]] void bad_value(const std::string& s) { throw Error{PyExc_ValueError, s}; }
[[noreturn]] void bad_type(const std::string& s) { throw Error{PyExc_TypeError, s}; }

PyObject* g_check = nullptr;      // model._check(code, name): raises CrError

// ------------------------------------------------------------ libcr calls
decltype(&cr_embedding) f_embedding;
decltype(&cr_embedding_backward_workspace_bytes) f_embedding_backward_workspace_bytes;
decltype(&cr_embedding_backward) f_embedding_backward;
decltype(&cr_causal_conv) f_causal_conv;
decltype(&cr_causal_conv_backward_workspace_bytes) f_causal_conv_backward_workspace_bytes;
decltype(&cr_causal_conv_backward) f_causal_conv_backward;
decltype(&cr_causal_conv_step) f_causal_conv_step;
decltype(&cr_selective_scan_checkpoints) f_selective_scan_checkpoints;
decltype(&cr_selective_scan_workspace_bytes) f_selective_scan_workspace_bytes;
decltype(&cr_selective_scan) f_selective_scan;
decltype(&cr_selective_scan_backward_workspace_bytes) f_selective_scan_backward_workspace_bytes;
decltype(&cr_selective_scan_backward) f_selective_scan_backward;
decltype(&cr_selective_scan_step) f_selective_scan_step;
decltype(&cr_layer_norm) f_layer_norm;
decltype(&cr_layer_norm_backward_workspace_bytes) f_layer_norm_backward_workspace_bytes;
decltype(&cr_layer_norm_backward) f_layer_norm_backward;
decltype(&cr_gated_scan_checkpoints) f_gated_scan_checkpoints;
decltype(&cr_gated_scan) f_gated_scan;
decltype(&cr_gated_scan_backward) f_gated_scan_backward;
decltype(&cr_gated_scan_step) f_gated_scan_step;
decltype(&cr_sample) f_sample;

void check(cr_status code, const char* name) {
  if (code == CR_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "is", (int)code, name);
  Py_XDECREF(r);
  if (r != nullptr) throw Error{PyExc_RuntimeError, join(name, " failed")};
  throw Error{nullptr, ""};
}

// ------------------------------------------------------------- arguments
const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad_type(join(name, " must be a tensor"));
  return THPVariable_Unpack(o);
}

bool flag(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Error{nullptr, ""};
  return v != 0;
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Error{nullptr, ""};
  return v;
}

float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Error{nullptr, ""};
  return (float)v;
}

int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda())
    bad_value(join(name, " must be a CUDA tensor (the model operators have no host form)"));
  return t.get_device();
}

cr_dtype type_code(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return CR_F32;
    case at::kBFloat16: return CR_BF16;
    case at::kHalf: return CR_F16;
    default:
      bad_type(join("the model operators take float32, bfloat16 or float16, got ",
                    t.scalar_type()));
  }
}

// Raises unless t has this shape and type and is on CUDA device `index`.
void need(const at::Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType dtype,
          int index) {
  if (t.scalar_type() != dtype)
    bad_type(join(name, " must be ", dtype, ", got ", t.scalar_type()));
  if (t.sizes() != shape) bad_value(join(name, " must have shape ", shape, ", got ", t.sizes()));
  if (!t.is_cuda() || t.get_device() != index)
    bad_value(join(name, " must be on cuda:", index, ", got ", t.device()));
}

int32_t activation(PyObject* o) {
  if (o == Py_None) return CR_ACT_NONE;
  if (PyUnicode_Check(o) && PyUnicode_CompareWithASCIIString(o, "silu") == 0) return CR_ACT_SILU;
  PyObject* r = PyObject_Repr(o);
  const char* s = r != nullptr ? PyUnicode_AsUTF8(r) : nullptr;
  const std::string got = s != nullptr ? s : "?";
  Py_XDECREF(r);
  PyErr_Clear();
  bad_value("activation must be None or 'silu', got " + got);
}

// Where a call runs. With a stream other than the current one, copies and
// outputs are made on it, and the allocator is told what it uses.
struct On {
  int index;
  cudaStream_t ptr;
  std::optional<c10::cuda::CUDAStream> other;
  c10::cuda::OptionalCUDAGuard device;
  c10::cuda::OptionalCUDAStreamGuard guard;

  On(int index_, PyObject* stream) : index(index_) {
    device.set_index((c10::DeviceIndex)index);
    ptr = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
    if (stream == Py_None) return;
    PyObject* id = PyObject_GetAttrString(stream, "stream_id");
    PyObject* dev = PyObject_GetAttrString(stream, "device_index");
    PyObject* kind = PyObject_GetAttrString(stream, "device_type");
    int64_t v[3] = {0, 0, 0};
    if (id != nullptr && dev != nullptr && kind != nullptr) {
      v[0] = PyLong_AsLongLong(id);
      v[1] = PyLong_AsLongLong(dev);
      v[2] = PyLong_AsLongLong(kind);
    }
    Py_XDECREF(id);
    Py_XDECREF(dev);
    Py_XDECREF(kind);
    if (PyErr_Occurred()) throw Error{nullptr, ""};
    if (v[1] != index) bad_value(join("stream must be of cuda:", index));
    const auto s = c10::cuda::CUDAStream::unpack3(v[0], (c10::DeviceIndex)v[1],
                                                  (c10::DeviceType)v[2]);
    if (s.stream() == ptr) return;
    other = s;
    ptr = s.stream();
    guard.reset_stream(s);
  }

  at::Tensor empty(at::IntArrayRef shape, at::ScalarType dtype) const {
    return at::empty(shape, at::TensorOptions().dtype(dtype).device(at::kCUDA, index));
  }
  at::Tensor output(PyObject* out, at::IntArrayRef shape, at::ScalarType dtype) const {
    if (out == Py_None) return empty(shape, dtype);
    const at::Tensor& t = tensor(out, "out");
    need(t, "out", shape, dtype, index);
    if (t.size(-1) > 1 && t.stride(-1) != 1) bad_value("out must have a contiguous last axis");
    writes(t);
    return t;
  }
  void uses(const at::Tensor& t) const {
    if (other) t.record_stream(*other);
  }

  // t is written: autograd sees that it is no longer what a call may have saved.
  void writes(const at::Tensor& t) const {
    uses(t);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  }

  // A call's workspace: its own, from the stream's allocator, which may have
  // it back when the call has been enqueued. (Held from call to call it would
  // be replaced by a larger call's while a captured graph still writes to it,
  // or shared by two graphs of one stream that are replayed on two.)
  at::Tensor workspace(size_t bytes, const char* name) const {
    if (bytes == 0) bad_value(join("invalid ", name, " arguments"));
    return empty({(int64_t)bytes}, at::kByte);
  }
};

// An argument as the calls take it, copied where its layout asks for it. The
// copy is made on the call's stream, so it is the caller's tensor that the
// allocator is told about: the copy is of that stream's own memory.
// With a contiguous last axis:
at::Tensor rows(const On& on, const at::Tensor& t) {
  on.uses(t);
  return t.size(-1) <= 1 || t.stride(-1) == 1 ? t : t.contiguous();
}

at::Tensor dense(const On& on, const at::Tensor& t) {
  on.uses(t);
  return t.is_contiguous() ? t : t.contiguous();
}

// An int32 or int64 tensor of indices, contiguous.
struct Indices {
  at::Tensor t;
  const void* p = nullptr;
  int32_t bytes = 4;
};

Indices indices(const On& on, PyObject* o, const char* name,
                std::optional<at::IntArrayRef> shape) {
  Indices r;
  if (o == Py_None) return r;
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kInt && t.scalar_type() != at::kLong)
    bad_type(join(name, " must be int32 or int64, got ", t.scalar_type()));
  need(t, name, shape ? *shape : t.sizes(), t.scalar_type(), on.index);
  r.t = dense(on, t);
  r.p = r.t.data_ptr();
  r.bytes = (int32_t)r.t.element_size();
  return r;
}

// An optional float32 vector or array, contiguous.
struct Floats {
  at::Tensor t;
  float* p = nullptr;
};

Floats floats(const On& on, PyObject* o, const char* name, at::IntArrayRef shape) {
  Floats r;
  if (o == Py_None) return r;
  const at::Tensor& t = tensor(o, name);
  need(t, name, shape, at::kFloat, on.index);
  r.t = dense(on, t);
  r.p = static_cast<float*>(r.t.data_ptr());
  return r;
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

void put(PyObject* dict, const char* name, const at::Tensor& t) {
  PyObject* v = wrap(t);
  if (v == nullptr || PyDict_SetItemString(dict, name, v) != 0) {
    Py_XDECREF(v);
    Py_DECREF(dict);
    throw Error{nullptr, ""};
  }
  Py_DECREF(v);
}

// Whether autograd has to know of a call: it records, and one of these
// arguments requires a gradient; or one has a tangent. The call then returns
// NotImplemented and model.py makes it part of the graph.
bool recorded(PyObject* const* a, std::initializer_list<int> which) {
  const bool records = c10::GradMode::is_enabled();
  for (int i : which) {
    if (!THPVariable_Check(a[i])) continue;
    const at::Tensor& t = THPVariable_Unpack(a[i]);
    if ((records && t.requires_grad()) || t._fw_grad(0).defined()) return true;
  }
  return false;
}

PyObject* not_implemented() {
  Py_INCREF(Py_NotImplemented);
  return Py_NotImplemented;
}

// ------------------------------------------------------------- embedding
// (tokens, table, scale, out, stream)
PyObject* embedding(PyObject* const* a) {
  if (recorded(a, {1})) return not_implemented();
  const at::Tensor& table0 = tensor(a[1], "table");
  const int index = device_of(table0, "table");
  if (table0.dim() != 2) bad_value("table must be 2-D (vocab, dim)");
  const cr_dtype code = type_code(table0);
  const float scale = real(a[2]);
  const On on(index, a[4]);
  if (a[0] == Py_None) bad_type("tokens must be a tensor");
  const Indices tok = indices(on, a[0], "tokens", std::nullopt);
  const int64_t n = tok.t.numel(), vocab = table0.size(0), dim = table0.size(1);
  at::Tensor table = rows(on, table0);
  if (vocab > 1 && table.stride(0) < dim) table = table.contiguous();  // rows that overlap
  std::vector<int64_t> shape = tok.t.sizes().vec();
  shape.push_back(dim);
  const at::Tensor o = on.output(a[3], shape, table.scalar_type());
  const at::Tensor flat = o.dim() == 2 ? o : o.view({n, dim});
  // a single row's stride means nothing; those of several are the tensors' own
  check(f_embedding(tok.p, tok.bytes, n, table.data_ptr(), vocab, dim,
                    vocab > 1 ? table.stride(0) : dim, scale, code, flat.data_ptr(),
                    n > 1 ? flat.stride(0) : dim, on.ptr),
        "cr_embedding");
  return wrap(o);
}

// (tokens, grad, vocab, scale, out, accumulate, stream)
PyObject* embedding_backward(PyObject* const* a) {
  const at::Tensor& grad0 = tensor(a[1], "grad");
  const int index = device_of(grad0, "grad");
  const at::Tensor& tokens = tensor(a[0], "tokens");
  if (grad0.dim() != tokens.dim() + 1 || grad0.sizes().slice(0, tokens.dim()) != tokens.sizes())
    bad_value("grad must have the shape of tokens and a channel axis");
  const bool accumulate = flag(a[5]);
  if (accumulate && a[4] == Py_None) bad_value("accumulate needs out");
  const int64_t vocab = integer(a[2]);
  if (vocab < 0) bad_value("vocab must be >= 0");
  const float scale = real(a[3]);
  const cr_dtype code = type_code(grad0);
  const On on(index, a[6]);
  const Indices tok = indices(on, a[0], "tokens", std::nullopt);
  const int64_t n = tok.t.numel(), dim = grad0.size(-1);
  on.uses(grad0);  // which reshape may copy
  at::Tensor grad = rows(on, grad0.dim() == 2 ? grad0 : grad0.reshape({n, dim}));
  if (n > 1 && grad.stride(0) < dim) grad = grad.contiguous();  // a zero stride
  const at::Tensor o = on.output(a[4], {vocab, dim}, at::kFloat);
  const at::Tensor ws = on.workspace(f_embedding_backward_workspace_bytes(n, vocab, dim),
                                     "embedding_backward");
  check(f_embedding_backward(tok.p, tok.bytes, n, grad.data_ptr(), n > 1 ? grad.stride(0) : dim,
                             vocab, dim, scale, code, accumulate,
                             static_cast<float*>(o.data_ptr()), vocab > 1 ? o.stride(0) : dim,
                             ws.data_ptr(), ws.numel(), on.ptr),
        "cr_embedding_backward");
  return wrap(o);
}

// ----------------------------------------------------------- convolution
// What the forward and the backward call share: (x, weight, bias, activation,
// state, lengths) and the stream.
struct Conv {
  const at::Tensor& x0;
  int index;
  On on;
  at::Tensor x, state;
  Floats weight, bias;
  Indices lengths;
  cr_causal_conv_args args;

  static const at::Tensor& checked(PyObject* o) {
    const at::Tensor& t = tensor(o, "x");
    device_of(t, "x");
    if (t.dim() != 3) bad_value("x must be (batch, time, channel)");
    return t;
  }

  Conv(PyObject* const* a, PyObject* stream)
      : x0(checked(a[0])), index(x0.get_device()), on(index, stream) {
    const cr_dtype code = type_code(x0);
    const int64_t batch = x0.size(0), len = x0.size(1), dim = x0.size(2);
    const at::Tensor& w = tensor(a[1], "weight");
    if (w.dim() != 2) bad_value("weight must be (channel, width)");
    const int64_t K = w.size(1);
    weight = floats(on, a[1], "weight", {dim, K});
    bias = floats(on, a[2], "bias", {dim});
    const int32_t act = activation(a[3]);
    if (a[4] != Py_None) {
      const at::Tensor& s = tensor(a[4], "state");
      need(s, "state", {batch, K - 1, dim}, x0.scalar_type(), index);
      state = dense(on, s);
    }
    lengths = indices(on, a[5], "lengths", at::IntArrayRef({batch}));
    x = rows(on, x0);
    args = {batch, len, dim, (int32_t)K, act, code, lengths.bytes, x.data_ptr(), x.stride(0),
            x.stride(1), weight.p, bias.p, state.defined() ? state.data_ptr() : nullptr,
            lengths.p};
  }
};

// (x, weight, bias, activation, state, lengths, return_state, out, stream)
PyObject* causal_conv(PyObject* const* a) {
  if (recorded(a, {0, 1, 2, 4})) return not_implemented();
  const Conv c(a, a[8]);
  const bool return_state = flag(a[6]);
  const at::Tensor y = c.on.output(a[7], c.x0.sizes(), c.x0.scalar_type());
  at::Tensor final;
  if (return_state)
    final = c.on.empty({c.args.batch, c.args.width - 1, c.args.dim}, c.x0.scalar_type());
  check(f_causal_conv(&c.args, y.data_ptr(), y.stride(0), y.stride(1),
                      return_state ? final.data_ptr() : nullptr, c.on.ptr),
        "cr_causal_conv");
  return return_state ? Py_BuildValue("(NN)", wrap(y), wrap(final)) : wrap(y);
}

// (x, weight, bias, activation, state, lengths, dy, dfinal, stream)
PyObject* causal_conv_backward(PyObject* const* a) {
  const Conv c(a, a[8]);
  const at::ScalarType type = c.x0.scalar_type();
  const at::Tensor& dy0 = tensor(a[6], "dy");
  need(dy0, "dy", c.x0.sizes(), type, c.index);
  const at::Tensor dy = rows(c.on, dy0);
  const int64_t K = c.args.width;
  at::Tensor dfinal, db, ds;
  if (a[7] != Py_None) {
    const at::Tensor& t = tensor(a[7], "dfinal");
    need(t, "dfinal", {c.args.batch, K - 1, c.args.dim}, type, c.index);
    dfinal = dense(c.on, t);
  }
  const at::Tensor dx = c.on.empty(c.x0.sizes(), type);
  const at::Tensor dw = c.on.empty({c.args.dim, K}, at::kFloat);
  if (c.bias.p != nullptr || c.bias.t.defined()) db = c.on.empty({c.args.dim}, at::kFloat);
  if (c.state.defined()) ds = c.on.empty(c.state.sizes(), type);
  const at::Tensor ws = c.on.workspace(
      f_causal_conv_backward_workspace_bytes(c.args.batch, c.args.len, c.args.dim, (int32_t)K),
      "causal_conv_backward");
  const cr_causal_conv_grads g = {dy.data_ptr(),
                                  dy.stride(0),
                                  dy.stride(1),
                                  dfinal.defined() ? dfinal.data_ptr() : nullptr,
                                  dx.data_ptr(),
                                  dx.stride(0),
                                  dx.stride(1),
                                  static_cast<float*>(dw.data_ptr()),
                                  db.defined() ? static_cast<float*>(db.data_ptr()) : nullptr,
                                  ds.defined() ? ds.data_ptr() : nullptr};
  check(f_causal_conv_backward(&c.args, &g, ws.data_ptr(), ws.numel(), c.on.ptr),
        "cr_causal_conv_backward");
  PyObject* r = PyDict_New();
  if (r == nullptr) throw Error{nullptr, ""};
  put(r, "x", dx);
  put(r, "weight", dw);
  if (db.defined()) put(r, "bias", db);
  if (ds.defined()) put(r, "state", ds);
  return r;
}

// A state that a step updates in place: (rows, ...), contiguous.
const at::Tensor& step_state(const On& on, PyObject* o, at::IntArrayRef row, at::ScalarType dtype,
                             int64_t batch, bool slots) {
  const at::Tensor& t = tensor(o, "state");
  if (t.dim() != 3) bad_value("state must be 3-D (rows, then what a row holds)");
  need(t, "state", {t.size(0), row[0], row[1]}, dtype, on.index);
  if (!t.is_contiguous()) bad_value("state must be contiguous (it is updated in place)");
  if (!slots && t.size(0) < batch)
    bad_value(join("state must have a row for each of the ", batch, " streams"));
  on.writes(t);
  return t;
}

// (x, state, weight, bias, activation, slots, out, stream)
PyObject* causal_conv_step(PyObject* const* a) {
  const at::Tensor& x0 = tensor(a[0], "x");
  const int index = device_of(x0, "x");
  const at::Tensor& w = tensor(a[2], "weight");
  if (x0.dim() != 2 || w.dim() != 2) bad_value("x must be (batch, dim), weight (dim, K)");
  const cr_dtype code = type_code(x0);
  const On on(index, a[7]);
  const int64_t batch = x0.size(0), dim = x0.size(1), K = w.size(1);
  const Floats weight = floats(on, a[2], "weight", {dim, K});
  const Floats bias = floats(on, a[3], "bias", {dim});
  const Indices slots = indices(on, a[5], "slots", at::IntArrayRef({batch}));
  const at::Tensor& state =
      step_state(on, a[1], {K - 1, dim}, x0.scalar_type(), batch, a[5] != Py_None);
  const at::Tensor x = rows(on, x0);
  const at::Tensor y = on.output(a[6], x0.sizes(), x0.scalar_type());
  check(f_causal_conv_step(x.data_ptr(), x.stride(0), state.data_ptr(), state.size(0), slots.p,
                           slots.bytes, weight.p, bias.p, activation(a[4]), batch, dim,
                           (int32_t)K, code, y.data_ptr(), y.stride(0), on.ptr),
        "cr_causal_conv_step");
  return wrap(y);
}

// -------------------------------------------------------- selective scan
// What the calls share: (u, dt, A, B, C, D, z, dt_bias, softplus), a state
// (None for a step), lengths or slots, and the stream.
struct Scan {
  const at::Tensor& u0;
  int index;
  On on;
  at::Tensor u, dt, z, B, C;
  Floats A, D, dt_bias, state;
  Indices lengths;
  cr_selective_scan_args args;

  static const at::Tensor& checked(PyObject* o, bool step) {
    const at::Tensor& t = tensor(o, "u");
    device_of(t, "u");
    if (t.dim() != (step ? 2 : 3))
      bad_value(step ? "u must be (batch, dim)" : "u must be (batch, time, dim)");
    return t;
  }

  // B or C as (..., groups, N) with the last two axes contiguous
  at::Tensor states(PyObject* o, const char* name, int64_t N) {
    at::Tensor t = tensor(o, name);
    const int64_t lead = u0.dim() - 1;
    if (t.dim() == lead + 1) t = t.unsqueeze(-2);  // one group
    if (t.dim() != lead + 2)
      bad_value(join(name, " must be (..., groups, dstate) or (..., dstate)"));
    std::vector<int64_t> shape = u0.sizes().slice(0, lead).vec();
    shape.push_back(t.size(-2));
    shape.push_back(N);
    need(t, name, shape, u0.scalar_type(), index);
    on.uses(t);
    if ((N > 1 && t.stride(-1) != 1) || (t.size(-2) > 1 && t.stride(-2) != N)) t = t.contiguous();
    return t;
  }

  at::Tensor like_u(PyObject* o, const char* name) {
    const at::Tensor& t = tensor(o, name);
    need(t, name, u0.sizes(), u0.scalar_type(), index);
    return rows(on, t);
  }

  Scan(PyObject* const* a, PyObject* state0, PyObject* lengths0, PyObject* stream, bool step)
      : u0(checked(a[0], step)), index(u0.get_device()), on(index, stream) {
    const cr_dtype code = type_code(u0);
    const int64_t batch = u0.size(0), len = step ? 1 : u0.size(1), dim = u0.size(-1);
    const at::Tensor& A0 = tensor(a[2], "A");
    if (A0.dim() != 2) bad_value("A must be (dim, dstate)");
    const int64_t N = A0.size(1);
    A = floats(on, a[2], "A", {dim, N});
    u = rows(on, u0);
    dt = like_u(a[1], "dt");
    B = states(a[3], "B", N);
    C = states(a[4], "C", N);
    const int64_t groups = B.size(-2);
    if (groups < 1 || dim % groups != 0 || C.size(-2) != groups)
      bad_value("B and C must be (..., groups, dstate) with groups dividing dim");
    D = floats(on, a[5], "D", {dim});
    if (a[6] != Py_None) z = like_u(a[6], "z");
    dt_bias = floats(on, a[7], "dt_bias", {dim});
    const bool softplus = flag(a[8]);
    if (state0 != Py_None) state = floats(on, state0, "state", {batch, dim, N});
    lengths = indices(on, lengths0, step ? "slots" : "lengths", at::IntArrayRef({batch}));
    const int64_t t = step ? 0 : 1;
    args = {batch,
            len,
            dim,
            (int32_t)N,
            (int32_t)groups,
            softplus ? 1 : 0,
            code,
            lengths.bytes,
            0,
            u.data_ptr(),
            u.stride(0),
            u.stride(t),
            dt.data_ptr(),
            dt.stride(0),
            dt.stride(t),
            z.defined() ? z.data_ptr() : nullptr,
            z.defined() ? z.stride(0) : 0,
            z.defined() ? z.stride(t) : 0,
            B.data_ptr(),
            B.stride(0),
            B.stride(t),
            C.data_ptr(),
            C.stride(0),
            C.stride(t),
            A.p,
            D.p,
            dt_bias.p,
            state.p,
            step ? nullptr : lengths.p};
  }
};

// (u, dt, A, B, C, D, z, dt_bias, softplus, state, lengths, return_state,
//  return_checkpoints, out, stream)
PyObject* selective_scan(PyObject* const* a) {
  if (recorded(a, {0, 1, 2, 3, 4, 5, 6, 7, 9})) return not_implemented();
  const Scan s(a, a[9], a[10], a[14], false);
  const bool return_state = flag(a[11]), return_checkpoints = flag(a[12]);
  const int64_t batch = s.args.batch, dim = s.args.dim, N = s.args.dstate;
  const at::Tensor y = s.on.output(a[13], s.u0.sizes(), s.u0.scalar_type());
  at::Tensor final, kept;
  if (return_state) final = s.on.empty({batch, dim, N}, at::kFloat);
  if (return_checkpoints)
    kept = s.on.empty({batch, f_selective_scan_checkpoints(s.args.len), dim, N}, at::kFloat);
  const at::Tensor ws =
      s.on.workspace(f_selective_scan_workspace_bytes(batch, s.args.len, dim, (int32_t)N),
                     "selective_scan");
  check(f_selective_scan(&s.args, y.data_ptr(), y.stride(0), y.stride(1),
                         return_state ? static_cast<float*>(final.data_ptr()) : nullptr,
                         return_checkpoints ? static_cast<float*>(kept.data_ptr()) : nullptr,
                         ws.data_ptr(), ws.numel(), s.on.ptr),
        "cr_selective_scan");
  if (return_state && return_checkpoints)
    return Py_BuildValue("(NNN)", wrap(y), wrap(final), wrap(kept));
  if (return_state) return Py_BuildValue("(NN)", wrap(y), wrap(final));
  if (return_checkpoints) return Py_BuildValue("(NN)", wrap(y), wrap(kept));
  return wrap(y);
}

// (u, dt, A, B, C, D, z, dt_bias, softplus, state, lengths, dy, dfinal,
//  checkpoints, stream)
PyObject* selective_scan_backward(PyObject* const* a) {
  const Scan s(a, a[9], a[10], a[14], false);
  const int64_t batch = s.args.batch, dim = s.args.dim, N = s.args.dstate;
  const at::ScalarType type = s.u0.scalar_type();
  const at::Tensor& dy0 = tensor(a[11], "dy");
  need(dy0, "dy", s.u0.sizes(), type, s.index);
  const at::Tensor dy = rows(s.on, dy0);
  const Floats dfinal = floats(s.on, a[12], "dfinal", {batch, dim, N});
  const at::Tensor& kept = tensor(a[13], "checkpoints");
  need(kept, "checkpoints", {batch, f_selective_scan_checkpoints(s.args.len), dim, N}, at::kFloat,
       s.index);
  if (!kept.is_contiguous())
    bad_value("checkpoints must be contiguous, as the forward call returns them");
  struct Out {
    const char* name;
    at::Tensor t;
    void* p() const { return t.defined() ? t.data_ptr() : nullptr; }
    float* f() const { return static_cast<float*>(p()); }
  };
  Out du{"u"}, ddt{"dt"}, dz{"z"}, dB{"B"}, dC{"C"}, dA{"A"}, dD{"D"}, db{"dt_bias"},
      ds{"state"};
  du.t = s.on.empty(s.u0.sizes(), type);
  ddt.t = s.on.empty(s.u0.sizes(), type);
  dA.t = s.on.empty({dim, N}, at::kFloat);
  dB.t = s.on.empty(tensor(a[3], "B").sizes(), type);
  dC.t = s.on.empty(tensor(a[4], "C").sizes(), type);
  if (s.D.t.defined()) dD.t = s.on.empty({dim}, at::kFloat);
  if (s.z.defined()) dz.t = s.on.empty(s.u0.sizes(), type);
  if (s.dt_bias.t.defined()) db.t = s.on.empty({dim}, at::kFloat);
  if (s.state.t.defined()) ds.t = s.on.empty({batch, dim, N}, at::kFloat);
  const at::Tensor ws = s.on.workspace(
      f_selective_scan_backward_workspace_bytes(batch, s.args.len, dim, (int32_t)N,
                                                s.args.groups),
      "selective_scan_backward");
  s.on.uses(kept);
  const cr_selective_scan_grads g = {dy.data_ptr(), dy.stride(0), dy.stride(1), dfinal.p,
                                     static_cast<const float*>(kept.data_ptr()),
                                     du.p(), ddt.p(), dz.p(), dB.p(), dC.p(), dA.f(), dD.f(),
                                     db.f(), ds.f()};
  check(f_selective_scan_backward(&s.args, &g, ws.data_ptr(), ws.numel(), s.on.ptr),
        "cr_selective_scan_backward");
  PyObject* r = PyDict_New();
  if (r == nullptr) throw Error{nullptr, ""};
  for (const Out* o : {&du, &ddt, &dA, &dB, &dC, &dD, &dz, &db, &ds})
    if (o->t.defined()) put(r, o->name, o->t);
  return r;
}

// (u, dt, A, B, C, D, z, dt_bias, softplus, state, slots, out, stream)
PyObject* selective_scan_step(PyObject* const* a) {
  const Scan s(a, Py_None, a[10], a[12], true);
  const int64_t batch = s.args.batch, dim = s.args.dim;
  const at::Tensor& state =
      step_state(s.on, a[9], {dim, s.args.dstate}, at::kFloat, batch, a[10] != Py_None);
  const at::Tensor y = s.on.output(a[11], s.u0.sizes(), s.u0.scalar_type());
  check(f_selective_scan_step(&s.args, static_cast<float*>(state.data_ptr()), state.size(0),
                              s.lengths.p, y.data_ptr(), y.stride(0), s.on.ptr),
        "cr_selective_scan_step");
  return wrap(y);
}

// ------------------------------------------------------------ layer norm
// A tensor's rows (all axes but the last) as two axes with a stride each: up to
// three axes as they are, more of them as one, copied where their strides ask
// for it.
struct RowAxes {
  at::Tensor t;
  int64_t batch, len, bs, ts;

  explicit RowAxes(const at::Tensor& x) : t(x) {
    if (x.dim() > 3) {
      int64_t n = 1;
      for (const int64_t v : x.sizes().slice(0, x.dim() - 1)) n *= v;
      t = x.reshape({n, x.size(-1)});
    }
    batch = t.dim() == 3 ? t.size(0) : 1;
    len = t.dim() >= 2 ? t.size(-2) : 1;
    bs = t.dim() == 3 ? t.stride(0) : 0;
    ts = t.dim() >= 2 ? t.stride(-2) : 0;
  }
};

// What the forward and the backward call share: (x, weight, bias, eps) and the
// stream.
struct Norm {
  const at::Tensor& x0;
  int index;
  On on;
  RowAxes x;
  Floats weight, bias;
  std::vector<int64_t> stats_shape;
  cr_layer_norm_args args;

  static const at::Tensor& checked(PyObject* o) {
    const at::Tensor& t = tensor(o, "x");
    device_of(t, "x");
    if (t.dim() < 1) bad_value("x must have a channel axis");
    return t;
  }

  Norm(PyObject* const* a, PyObject* stream)
      : x0(checked(a[0])), index(x0.get_device()), on(index, stream), x(rows(on, x0)) {
    const cr_dtype code = type_code(x0);
    const int64_t dim = x0.size(-1);
    weight = floats(on, a[1], "weight", {dim});
    bias = floats(on, a[2], "bias", {dim});
    const float eps = real(a[3]);
    if (!(eps >= 0.0f)) bad_value("eps must be >= 0");
    stats_shape = x0.sizes().vec();
    stats_shape.back() = 3;
    args = {x.batch, x.len, dim, code, eps, x.t.data_ptr(), x.bs, x.ts, weight.p, bias.p};
  }
};

// (x, weight, bias, eps, return_stats, out, stream)
PyObject* layer_norm(PyObject* const* a) {
  if (recorded(a, {0, 1, 2})) return not_implemented();
  const Norm c(a, a[6]);
  const bool return_stats = flag(a[4]);
  const at::Tensor y = c.on.output(a[5], c.x0.sizes(), c.x0.scalar_type());
  if (y.dim() > 3 && !y.is_contiguous()) bad_value("out with more than 3 axes must be contiguous");
  const RowAxes o(y);
  at::Tensor stats;
  if (return_stats) stats = c.on.empty(c.stats_shape, at::kFloat);
  if (return_stats && c.args.dim == 0) stats.fill_(NAN);  // of nothing, by no kernel
  check(f_layer_norm(&c.args, o.t.data_ptr(), o.bs, o.ts,
                     return_stats ? static_cast<float*>(stats.data_ptr()) : nullptr, c.on.ptr),
        "cr_layer_norm");
  return return_stats ? Py_BuildValue("(NN)", wrap(y), wrap(stats)) : wrap(y);
}

// (x, weight, bias, eps, dy, stats, stream)
PyObject* layer_norm_backward(PyObject* const* a) {
  const Norm c(a, a[6]);
  const at::ScalarType type = c.x0.scalar_type();
  const at::Tensor& dy0 = tensor(a[4], "dy");
  need(dy0, "dy", c.x0.sizes(), type, c.index);
  const RowAxes dy(rows(c.on, dy0));
  const Floats stats = floats(c.on, a[5], "stats", c.stats_shape);
  const at::Tensor dx = c.on.empty(c.x0.sizes(), type);
  const RowAxes o(dx);
  at::Tensor dw, db;
  if (c.weight.t.defined()) dw = c.on.empty({c.args.dim}, at::kFloat);
  if (c.bias.t.defined()) db = c.on.empty({c.args.dim}, at::kFloat);
  const at::Tensor ws = c.on.workspace(
      f_layer_norm_backward_workspace_bytes(c.args.batch, c.args.len, c.args.dim),
      "layer_norm_backward");
  const cr_layer_norm_grads g = {dy.t.data_ptr(),
                                 dy.bs,
                                 dy.ts,
                                 stats.p,
                                 o.t.data_ptr(),
                                 o.bs,
                                 o.ts,
                                 dw.defined() ? static_cast<float*>(dw.data_ptr()) : nullptr,
                                 db.defined() ? static_cast<float*>(db.data_ptr()) : nullptr};
  check(f_layer_norm_backward(&c.args, &g, ws.data_ptr(), ws.numel(), c.on.ptr),
        "cr_layer_norm_backward");
  PyObject* r = PyDict_New();
  if (r == nullptr) throw Error{nullptr, ""};
  put(r, "x", dx);
  if (dw.defined()) put(r, "weight", dw);
  if (db.defined()) put(r, "bias", db);
  return r;
}

// ------------------------------------------------------------ gated scan
// What the calls share: (x, gate, z), a state (None for a step), lengths or
// slots, and the stream.
struct Gated {
  const at::Tensor& x0;
  int index;
  On on;
  at::Tensor x, gate, z;
  Floats state;
  Indices lengths;
  cr_gated_scan_args args;

  static const at::Tensor& checked(PyObject* o, bool step) {
    const at::Tensor& t = tensor(o, "x");
    device_of(t, "x");
    if (t.dim() != (step ? 2 : 3))
      bad_value(step ? "x must be (batch, dim)" : "x must be (batch, time, dim)");
    return t;
  }

  Gated(PyObject* const* a, PyObject* state0, PyObject* lengths0, PyObject* stream, bool step)
      : x0(checked(a[0], step)), index(x0.get_device()), on(index, stream) {
    const cr_dtype code = type_code(x0);
    const int64_t batch = x0.size(0), len = step ? 1 : x0.size(1), dim = x0.size(-1);
    auto like_x = [&](PyObject* o, const char* name) {
      const at::Tensor& t = tensor(o, name);
      need(t, name, x0.sizes(), x0.scalar_type(), index);
      return rows(on, t);
    };
    x = rows(on, x0);
    gate = like_x(a[1], "gate");
    if (a[2] != Py_None) z = like_x(a[2], "z");
    if (state0 != Py_None) state = floats(on, state0, "state", {batch, dim});
    lengths = indices(on, lengths0, step ? "slots" : "lengths", at::IntArrayRef({batch}));
    const int64_t t = step ? 0 : 1;
    args = {batch,
            len,
            dim,
            code,
            lengths.bytes,
            x.data_ptr(),
            x.stride(0),
            x.stride(t),
            gate.data_ptr(),
            gate.stride(0),
            gate.stride(t),
            z.defined() ? z.data_ptr() : nullptr,
            z.defined() ? z.stride(0) : 0,
            z.defined() ? z.stride(t) : 0,
            state.p,
            step ? nullptr : lengths.p};
  }
};

// (x, gate, z, state, lengths, return_state, return_checkpoints, out, stream)
PyObject* gated_scan(PyObject* const* a) {
  if (recorded(a, {0, 1, 2, 3})) return not_implemented();
  const Gated s(a, a[3], a[4], a[8], false);
  const bool return_state = flag(a[5]), return_checkpoints = flag(a[6]);
  const int64_t batch = s.args.batch, dim = s.args.dim;
  const at::Tensor y = s.on.output(a[7], s.x0.sizes(), s.x0.scalar_type());
  at::Tensor final, kept;
  if (return_state) final = s.on.empty({batch, dim}, at::kFloat);
  if (return_checkpoints)
    kept = s.on.empty({batch, f_gated_scan_checkpoints(s.args.len), dim}, at::kFloat);
  check(f_gated_scan(&s.args, y.data_ptr(), y.stride(0), y.stride(1),
                     return_state ? static_cast<float*>(final.data_ptr()) : nullptr,
                     return_checkpoints ? static_cast<float*>(kept.data_ptr()) : nullptr,
                     s.on.ptr),
        "cr_gated_scan");
  if (return_state && return_checkpoints)
    return Py_BuildValue("(NNN)", wrap(y), wrap(final), wrap(kept));
  if (return_state) return Py_BuildValue("(NN)", wrap(y), wrap(final));
  if (return_checkpoints) return Py_BuildValue("(NN)", wrap(y), wrap(kept));
  return wrap(y);
}

// (x, gate, z, state, lengths, dy, dfinal, checkpoints, stream)
PyObject* gated_scan_backward(PyObject* const* a) {
  const Gated s(a, a[3], a[4], a[8], false);
  const int64_t batch = s.args.batch, dim = s.args.dim;
  const at::ScalarType type = s.x0.scalar_type();
  const at::Tensor& dy0 = tensor(a[5], "dy");
  need(dy0, "dy", s.x0.sizes(), type, s.index);
  const at::Tensor dy = rows(s.on, dy0);
  const Floats dfinal = floats(s.on, a[6], "dfinal", {batch, dim});
  const at::Tensor& kept = tensor(a[7], "checkpoints");
  need(kept, "checkpoints", {batch, f_gated_scan_checkpoints(s.args.len), dim}, at::kFloat,
       s.index);
  if (!kept.is_contiguous())
    bad_value("checkpoints must be contiguous, as the forward call returns them");
  at::Tensor dz, ds;
  const at::Tensor dx = s.on.empty(s.x0.sizes(), type), dgate = s.on.empty(s.x0.sizes(), type);
  if (s.z.defined()) dz = s.on.empty(s.x0.sizes(), type);
  if (s.state.t.defined()) ds = s.on.empty({batch, dim}, at::kFloat);
  s.on.uses(kept);
  const cr_gated_scan_grads g = {dy.data_ptr(),
                                 dy.stride(0),
                                 dy.stride(1),
                                 dfinal.p,
                                 static_cast<const float*>(kept.data_ptr()),
                                 dx.data_ptr(),
                                 dgate.data_ptr(),
                                 dz.defined() ? dz.data_ptr() : nullptr,
                                 ds.defined() ? static_cast<float*>(ds.data_ptr()) : nullptr};
  check(f_gated_scan_backward(&s.args, &g, s.on.ptr), "cr_gated_scan_backward");
  PyObject* r = PyDict_New();
  if (r == nullptr) throw Error{nullptr, ""};
  put(r, "x", dx);
  put(r, "gate", dgate);
  if (dz.defined()) put(r, "z", dz);
  if (ds.defined()) put(r, "state", ds);
  return r;
}

// (x, gate, state, z, slots, out, stream)
PyObject* gated_scan_step(PyObject* const* a) {
  PyObject* const main[] = {a[0], a[1], a[3]};
  const Gated s(main, Py_None, a[4], a[6], true);
  const at::Tensor& state = tensor(a[2], "state");
  if (state.dim() != 2) bad_value("state must be (rows, dim)");
  need(state, "state", {state.size(0), s.args.dim}, at::kFloat, s.index);
  if (!state.is_contiguous()) bad_value("state must be contiguous (it is updated in place)");
  if (a[4] == Py_None && state.size(0) < s.args.batch)
    bad_value(join("state must have a row for each of the ", s.args.batch, " streams"));
  s.on.writes(state);
  const at::Tensor y = s.on.output(a[5], s.x0.sizes(), s.x0.scalar_type());
  check(f_gated_scan_step(&s.args, static_cast<float*>(state.data_ptr()), state.size(0),
                          s.lengths.p, y.data_ptr(), y.stride(0), s.on.ptr),
        "cr_gated_scan_step");
  return wrap(y);
}

// -------------------------------------------------------------- sampling
// A setting: a number for every row, or a tensor with one a row.
struct Setting {
  double value;
  Floats each;
};

Setting setting(const On& on, PyObject* o, const char* name, at::IntArrayRef shape, double none) {
  Setting r{none, {}};
  if (o == Py_None) return r;
  if (THPVariable_Check(o)) {
    r.each = floats(on, o, name, shape);
    return r;
  }
  r.value = PyFloat_AsDouble(o);
  if (r.value == -1.0 && PyErr_Occurred()) throw Error{nullptr, ""};
  return r;
}

// (logits, u, temperature, top_k, top_p, min_p, out, stream)
PyObject* sample(PyObject* const* a) {
  const at::Tensor& x0 = tensor(a[0], "logits");
  const int index = device_of(x0, "logits");
  if (x0.dim() < 1) bad_value("logits must be (..., vocab)");
  const cr_dtype code = type_code(x0);
  const On on(index, a[7]);
  const at::IntArrayRef shape = x0.sizes().slice(0, x0.dim() - 1);
  if (a[1] == Py_None) bad_type("u must be a tensor");
  const Floats u = floats(on, a[1], "u", shape);
  const Setting temperature = setting(on, a[2], "temperature", shape, 1.0);
  const Setting top_p = setting(on, a[4], "top_p", shape, 1.0);
  const Setting min_p = setting(on, a[5], "min_p", shape, 0.0);
  if (!(temperature.value >= 0.0)) bad_value("temperature must be >= 0");
  if (!(top_p.value >= 0.0)) bad_value("top_p must be >= 0");
  if (!(min_p.value >= 0.0 && min_p.value <= 1.0)) bad_value("min_p must be in [0, 1]");
  Indices ks;
  int64_t top_k = 0;
  if (a[3] != Py_None) {
    if (THPVariable_Check(a[3])) ks = indices(on, a[3], "top_k", shape);
    else top_k = integer(a[3]);
  }
  if (top_k < 0) bad_value("top_k must be >= 0");
  at::Tensor x = rows(on, x0);
  if (x.dim() != 2) x = x.reshape({u.t.numel(), x0.size(-1)});
  at::Tensor out;
  if (a[6] == Py_None) {
    out = on.empty(shape, at::kLong);
  } else {
    out = tensor(a[6], "out");
    need(out, "out", shape, at::kLong, index);
    if (!out.is_contiguous()) bad_value("out must be contiguous");
    on.writes(out);
  }
  const int64_t n = x.size(0), vocab = x.size(1);
  const cr_sample_args args = {n,
                               vocab,
                               code,
                               ks.bytes,
                               x.data_ptr(),
                               n > 1 ? x.stride(0) : vocab,
                               u.p,
                               temperature.value,
                               top_p.value,
                               min_p.value,
                               top_k,
                               temperature.each.p,
                               top_p.each.p,
                               min_p.each.p,
                               ks.p};
  check(f_sample(&args, static_cast<int64_t*>(out.data_ptr()), on.ptr), "cr_sample");
  return wrap(out);
}

// ---------------------------------------------------------------- module
// One entry: the number of arguments, and every C++ exception turned into a
// Python one.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments are needed, got %zd", N, n);
    return nullptr;
  }
  if (g_check == nullptr) {
    PyErr_SetString(PyExc_RuntimeError, "bind() comes first");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Error& e) {
    if (e.type != nullptr) PyErr_SetString(e.type, e.what.c_str());
    return nullptr;
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    PyErr_Clear();
    PyErr_SetString(type != nullptr ? type : PyExc_RuntimeError, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
    return nullptr;
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    return nullptr;
  }
}

// bind(addresses by name, check)
PyObject* bind(PyObject*, PyObject* args) {
  PyObject *names = nullptr, *chk = nullptr;
  if (!PyArg_ParseTuple(args, "O!O", &PyDict_Type, &names, &chk)) return nullptr;
  bool ok = true;
  auto get = [&](const char* name, auto& f) {
    PyObject* v = PyDict_GetItemString(names, name);
    void* p = v != nullptr ? PyLong_AsVoidPtr(v) : nullptr;
    if (p == nullptr) ok = false;
    f = reinterpret_cast<std::decay_t<decltype(f)>>(p);
  };
#define CR_BIND(NAME) get("cr_" #NAME, f_##NAME)
  CR_BIND(embedding);
  CR_BIND(embedding_backward_workspace_bytes);
  CR_BIND(embedding_backward);
  CR_BIND(causal_conv);
  CR_BIND(causal_conv_backward_workspace_bytes);
  CR_BIND(causal_conv_backward);
  CR_BIND(causal_conv_step);
  CR_BIND(selective_scan_checkpoints);
  CR_BIND(selective_scan_workspace_bytes);
  CR_BIND(selective_scan);
  CR_BIND(selective_scan_backward_workspace_bytes);
  CR_BIND(selective_scan_backward);
  CR_BIND(selective_scan_step);
  CR_BIND(layer_norm);
  CR_BIND(layer_norm_backward_workspace_bytes);
  CR_BIND(layer_norm_backward);
  CR_BIND(gated_scan_checkpoints);
  CR_BIND(gated_scan);
  CR_BIND(gated_scan_backward);
  CR_BIND(gated_scan_step);
  CR_BIND(sample);
#undef CR_BIND
  if (!ok) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "a libcr function is missing");
    return nullptr;
  }
  Py_INCREF(chk);
  Py_XSETREF(g_check, chk);
  Py_RETURN_NONE;
}

#define CR_ENTRY(NAME, N) \
  {#NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<NAME, N>)), METH_FASTCALL, \
   nullptr}

PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr},
                         CR_ENTRY(embedding, 5),
                         CR_ENTRY(embedding_backward, 7),
                         CR_ENTRY(causal_conv, 9),
                         CR_ENTRY(causal_conv_backward, 9),
                         CR_ENTRY(causal_conv_step, 8),
                         CR_ENTRY(selective_scan, 15),
                         CR_ENTRY(selective_scan_backward, 15),
                         CR_ENTRY(selective_scan_step, 13),
                         CR_ENTRY(layer_norm, 7),
                         CR_ENTRY(layer_norm_backward, 7),
                         CR_ENTRY(gated_scan, 9),
                         CR_ENTRY(gated_scan_backward, 9),
                         CR_ENTRY(gated_scan_step, 7),
                         CR_ENTRY(sample, 8),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "cr_model_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_cr_model_binding(void) { return PyModule_Create(&module); }
