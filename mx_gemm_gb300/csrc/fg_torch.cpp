// Python binding of the operators around the GEMM (mx_gemm_gb300/moe.py) and of
// the GEMM's ordinary call: the checks of their tensors, their outputs'
// allocation, and the call of the C ABI.  A call of theirs on one token keeps the GPU busy for 2 to 5 us, while
// allocating each output from Python takes 1.5 us and a ctypes call of fifteen
// arguments as much again (routing: 17 us a call that way); from here the same
// steps cost a third of it.
//
// Errors: ValueError for tensors that the library would misread, the package's
// FgError for a status of the C ABI, and torch's own for the allocations.
#include <Python.h>
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <string>

#include "../../include/fg.h"

namespace {

PyObject* g_error = nullptr;  // the package's FgError

struct Refused : std::exception {  // a ValueError with this text
  std::string text;
  explicit Refused(std::string t) : text(std::move(t)) {}
  const char* what() const noexcept override { return text.c_str(); }
};

[[noreturn]] void refuse(const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  throw Refused(buf);
}

struct Status : std::exception {  // a status of the C ABI and its message
  int status;
  std::string text;
  explicit Status(int s) : status(s), text(fg_last_error_message()) {}
};

void check(fg_status s) {
  if (s != FG_OK) throw Status(s);
}

// The interpreter's lock is free while memory is allocated and kernels are
// launched, as in a ctypes call.
struct Unlocked {
  PyThreadState* s = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(s); }
};

template <typename F>
PyObject* guarded(F&& body) {
  HANDLE_TH_ERRORS
  try {
    return body();
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const Status& e) {
    PyObject* x = PyObject_CallFunction(g_error, "is", e.status, e.text.c_str());
    if (x) {
      PyErr_SetObject(g_error, x);
      Py_DECREF(x);
    }
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------- arguments

std::string shape_of(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse("%s must be an integer", name);
  }
  return v;
}

// ... that fits the C ABI's int, or its 32 bits of flags: cut down to them, 2^32
// + 1 would pass for 1.
int small(PyObject* o, const char* name) {
  const int64_t v = integer(o, name);
  if (v < INT32_MIN || v > INT32_MAX) refuse("%s=%lld is out of range", name, (long long)v);
  return static_cast<int>(v);
}

uint32_t flag_bits(PyObject* o, const char* name) {
  const int64_t v = integer(o, name);
  if (v < 0 || v > UINT32_MAX) refuse("%s=%lld is out of range", name, (long long)v);
  return static_cast<uint32_t>(v);
}

bool truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    refuse("%s must be true or false", name);
  }
  return v == 1;
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse("%s must be a torch.Tensor, got %s", name, Py_TYPE(o)->tp_name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) refuse("%s must be a CUDA tensor (it is on %s)", name, t.device().str().c_str());
  return t;
}

void on(const at::Tensor& t, const char* name, const at::Device& device) {
  if (t.device() != device)
    refuse("%s is on %s, the other operands on %s", name, t.device().str().c_str(), device.str().c_str());
}

struct Rows {
  int64_t m, k, ld;
};

// A 2-D tensor whose rows are contiguous, any distance apart.
Rows rows_of(const at::Tensor& t, const char* name) {
  if (t.dim() != 2) refuse("%s must be 2-D, got shape %s", name, shape_of(t).c_str());
  Rows r{t.size(0), t.size(1), t.stride(0)};
  if (t.stride(1) != 1 && r.k > 1)
    refuse("%s must have contiguous rows (shape %s, strides (%lld, %lld))", name, shape_of(t).c_str(), (long long)t.stride(0),
           (long long)t.stride(1));
  if (r.m <= 1)
    r.ld = r.k > 1 ? r.k : 1;  // the distance of a single row says nothing
  else if (r.ld < r.k)
    refuse("%s has overlapping rows (shape %s, strides (%lld, %lld))", name, shape_of(t).c_str(), (long long)t.stride(0),
           (long long)t.stride(1));
  return r;
}

void contiguous(const at::Tensor& t, const char* name) {
  if (!t.is_contiguous())
    refuse("%s must be contiguous row-major memory (shape %s)", name, shape_of(t).c_str());
}

bool is_bytes(at::ScalarType d) { return d == at::kByte || d == at::kChar; }

void typed(const at::Tensor& t, const char* name, bool ok, const char* expected) {
  if (!ok) refuse("%s has dtype %s; expected %s", name, c10::toString(t.scalar_type()), expected);
}

int type_of(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kFloat) return FG_TYPE_F32;
  typed(t, name, t.scalar_type() == at::kBFloat16, "torch.float32 or torch.bfloat16");
  return FG_TYPE_BF16;
}

// ------------------------------------------------- outputs and the stream

// What torch.empty ends in for a CUDA device, without the dispatch before it.
at::Tensor make(at::IntArrayRef sizes, at::ScalarType type, const at::Device& device) {
  return at::detail::empty_cuda(sizes, type, device, std::nullopt);
}

PyObject* wrap(const at::Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}

// The stream of a call: the current one of the operands' device, or the caller's.
struct Launch {
  c10::cuda::CUDAStream current;
  cudaStream_t stream;
  bool other() const { return stream != current.stream(); }
};

Launch launch_of(PyObject* handle, const at::Device& device) {
  if (device.index() != c10::cuda::current_device())
    refuse("the operands are on %s, the current device is cuda:%d", device.str().c_str(), (int)c10::cuda::current_device());
  const auto current = c10::cuda::getCurrentCUDAStream(device.index());
  if (handle == Py_None) return {current, current.stream()};
  auto stream = reinterpret_cast<cudaStream_t>(static_cast<intptr_t>(integer(handle, "stream")));
  if (stream == cudaStreamLegacy) stream = nullptr;  // the default stream by its other name
  return {current, stream};
}

// While it lives, memory is allocated for the call's stream: a block that was
// freed on the caller's current stream may still be in use there by work that
// the call's stream does not wait for.
struct Pool {
  const Launch& launch;
  explicit Pool(const Launch& l) : launch(l) {
    if (l.other()) c10::cuda::setCurrentCUDAStream(c10::cuda::getStreamFromExternal(l.stream, l.current.device_index()));
  }
  ~Pool() {
    if (launch.other()) c10::cuda::setCurrentCUDAStream(launch.current);
  }
};

// On another stream than the current one: the memory of what was made here is
// not reused before the current stream, on which the caller uses it (after a
// wait of its own), is done with it, and that of the caller's tensors not before
// the call's stream is.
void keep(const Launch& launch, std::initializer_list<const at::Tensor*> made,
          std::initializer_list<const at::Tensor*> given) {
  if (!launch.other()) return;
  for (const at::Tensor* t : made)
    if (t->defined()) t->record_stream(launch.current.unwrap());
  const auto other = c10::cuda::getStreamFromExternal(launch.stream, launch.current.device_index());
  for (const at::Tensor* t : given)
    if (t && t->defined()) t->record_stream(other.unwrap());
}

struct Codes {
  at::Tensor codes, scales;
};

Codes make_codes(int mode, int64_t m, int64_t k, const at::Device& device) {
  Codes c;
  c.codes = mode == FG_MXFP4 ? make({m, k / 2}, at::kByte, device) : make({m, k}, at::kFloat8_e4m3fn, device);
  c.scales = mode == FG_FP8_BLOCK128 ? make({m, k / 128}, at::kFloat, device)
                                     : make({m, k / (mode == FG_MXFP8 ? 128 : 32)}, at::kFloat8_e8m0fnu, device);
  return c;
}

void* data(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

void arity(Py_ssize_t n, Py_ssize_t want, const char* name) {
  if (n != want) refuse("%s takes %d arguments, got %d", name, (int)want, (int)n);
}

// -------------------------------------------------------------- operators

// (mode, act, x, stream) -> (codes, scales)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 4, "quantize");
    const int mode = small(a[0], "mode"), act = small(a[1], "act");
    const at::Tensor& x = tensor(a[2], "x");
    Rows r = rows_of(x, "x");
    const int type = type_of(x, "x");
    if (act == FG_ACT_SWIGLU) {
      if (r.k % 2) refuse("x must have rows (g, u) of two equal halves, got %lld columns", (long long)r.k);
      r.k /= 2;
    }
    const at::Device device = x.device();
    const Launch launch = launch_of(a[3], device);
    Codes c;
    {
      Unlocked u;
      Pool pool(launch);
      c = make_codes(mode, r.m, r.k, device);
      check(fg_quantize(mode, act, x.data_ptr(), type, r.m, r.k, r.ld, c.codes.data_ptr(), c.scales.data_ptr(),
                        launch.stream));
      keep(launch, {&c.codes, &c.scales}, {&x});
    }
    return Py_BuildValue("(NN)", wrap(c.codes), wrap(c.scales));
  });
}

// (mode, x, weight, residual or None, eps, normed, stream) -> (codes, scales, h, y)
PyObject* rmsnorm_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 7, "rmsnorm_quantize");
    const int mode = small(a[0], "mode");
    const at::Tensor& x = tensor(a[1], "x");
    const Rows r = rows_of(x, "x");
    const int type = type_of(x, "x");
    const at::Device device = x.device();
    const at::Tensor& w = tensor(a[2], "weight");
    on(w, "weight", device);
    contiguous(w, "weight");
    typed(w, "weight", w.scalar_type() == x.scalar_type(), "that of x");
    if (w.dim() != 1 || w.size(0) != r.k) refuse("weight has shape %s, expected (%lld,)", shape_of(w).c_str(), (long long)r.k);
    const at::Tensor* res = a[3] == Py_None ? nullptr : &tensor(a[3], "residual");
    Rows rr{r.m, r.k, r.k};
    if (res) {
      on(*res, "residual", device);
      rr = rows_of(*res, "residual");
      typed(*res, "residual", res->scalar_type() == x.scalar_type(), "that of x");
      if (rr.m != r.m || rr.k != r.k)
        refuse("residual has shape %s, expected %s", shape_of(*res).c_str(), shape_of(x).c_str());
    }
    const double eps = PyFloat_AsDouble(a[4]);
    if (eps == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      refuse("eps must be a number");
    }
    const bool plain = mode == FG_BF16, normed = truth(a[5], "normed") || plain;
    const Launch launch = launch_of(a[6], device);
    Codes c;
    at::Tensor h, y;
    {
      Unlocked u;
      Pool pool(launch);
      if (!plain) c = make_codes(mode, r.m, r.k, device);
      if (res) h = make({r.m, r.k}, x.scalar_type(), device);
      if (normed) y = make({r.m, r.k}, x.scalar_type(), device);
      check(fg_rmsnorm_quantize(mode, x.data_ptr(), r.ld, res ? res->data_ptr() : nullptr, rr.ld, w.data_ptr(), (float)eps,
                                type, r.m, r.k, data(h), data(y), data(c.codes), data(c.scales), launch.stream));
      keep(launch, {&c.codes, &c.scales, &h, &y}, {&x, &w, res});
    }
    return Py_BuildValue("(NNNN)", wrap(c.codes), wrap(c.scales), wrap(h), wrap(y));
  });
}

// (logits, top_k, renormalize, stream) -> (weights, experts, offsets, rows, slots)
PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 4, "moe_route");
    const at::Tensor& x = tensor(a[0], "logits");
    const Rows r = rows_of(x, "logits");
    const int type = type_of(x, "logits");
    const int64_t k = integer(a[1], "top_k");
    if (k < 1 || k > (r.k > 1 ? r.k : 1)) refuse("top_k=%lld outside 1..%lld", (long long)k, (long long)r.k);
    const bool renormalize = truth(a[2], "renormalize");
    const at::Device device = x.device();
    const Launch launch = launch_of(a[3], device);
    at::Tensor weights, experts, offsets, rows, slots, ws;
    {
      Unlocked u;
      Pool pool(launch);
      uint64_t need = 0;
      check(fg_moe_route_workspace_size(r.m, (int)(r.k < (1 << 30) ? r.k : 1 << 30), &need));
      weights = make({r.m, k}, at::kFloat, device);
      experts = make({r.m, k}, at::kInt, device);
      offsets = make({r.k + 1}, at::kInt, device);
      rows = make({r.m * k}, at::kInt, device);
      slots = make({r.m, k}, at::kInt, device);
      if (need) ws = make({static_cast<int64_t>(need)}, at::kByte, device);
      check(fg_moe_route(x.data_ptr(), type, r.m, (int)r.k, r.ld, (int)(k < 1024 ? k : 1024),
                         renormalize ? FG_FLAG_RENORMALIZE : 0, weights.data_ptr<float>(), experts.data_ptr<int32_t>(),
                         offsets.data_ptr<int32_t>(), rows.data_ptr<int32_t>(), slots.data_ptr<int32_t>(), data(ws), need,
                         launch.stream));
      keep(launch, {&weights, &experts, &offsets, &rows, &slots}, {&x});
    }
    return Py_BuildValue("(NNNNN)", wrap(weights), wrap(experts), wrap(offsets), wrap(rows), wrap(slots));
  });
}

// (A, weight data, descriptor's address, offsets, a_scales or None, rows or None,
//  Y or None, workspace or None, flags, stream) -> Y
PyObject* grouped_gemm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 10, "grouped_gemm");
    const at::Tensor& weight = tensor(v[1], "the weight");
    const at::Device device = weight.device();
    const fg_bshuf* b = reinterpret_cast<const fg_bshuf*>(static_cast<intptr_t>(integer(v[2], "the descriptor's address")));
    const int mode = b->mode;
    const int64_t K = b->K;
    const at::Tensor& A = tensor(v[0], "A");
    on(A, "A", device);
    contiguous(A, "A");
    const at::ScalarType at_ = A.scalar_type();
    if (mode == FG_BF16)
      typed(A, "A", at_ == at::kBFloat16 || at_ == at::kShort || at_ == at::kUInt16, "torch.bfloat16");
    else if (mode == FG_MXFP4)
      typed(A, "A", is_bytes(at_) || at_ == at::kFloat4_e2m1fn_x2, "packed e2m1 bytes");
    else
      typed(A, "A", is_bytes(at_) || at_ == at::kFloat8_e4m3fn, "torch.float8_e4m3fn or bytes");
    const int64_t row = mode == FG_BF16 ? 2 * K : (mode == FG_MXFP4 ? K / 2 : K);
    if (A.dim() != 2 || A.size(1) * (int64_t)A.element_size() != row)
      refuse("A must be [T][K] codes of the mode (%lld bytes per row for K=%lld), got shape %s dtype %s", (long long)row,
             (long long)K, shape_of(A).c_str(), c10::toString(at_));
    const int64_t T = A.size(0);
    const at::Tensor& offsets = tensor(v[3], "offsets");
    on(offsets, "offsets", device);
    contiguous(offsets, "offsets");
    typed(offsets, "offsets", offsets.scalar_type() == at::kInt, "torch.int32");
    const int64_t E = offsets.numel() - 1;
    if (E < 1 || b->N % E)
      refuse("offsets must hold E + 1 values, E a divisor of the stacked weight's %lld rows", (long long)b->N);
    const int64_t N = b->N / E;
    const at::Tensor* scales = v[4] == Py_None ? nullptr : &tensor(v[4], "a_scales");
    if (scales && mode != FG_BF16) {
      on(*scales, "a_scales", device);
      contiguous(*scales, "a_scales");
      const at::ScalarType s = scales->scalar_type();
      const bool fp32 = mode == FG_FP8_TENSOR || mode == FG_FP8_BLOCK128;
      if (fp32) typed(*scales, "a_scales", s == at::kFloat, "torch.float32");
      else typed(*scales, "a_scales", is_bytes(s) || s == at::kFloat8_e8m0fnu, "torch.float8_e8m0fnu or bytes");
      const int64_t want = mode == FG_FP8_TENSOR ? 1 : T * (K / (mode == FG_MXFP8 || mode == FG_FP8_BLOCK128 ? 128 : 32));
      if (scales->numel() != want)
        refuse("a_scales has %lld elements, expected %lld", (long long)scales->numel(), (long long)want);
    }
    const at::Tensor* rows = v[5] == Py_None ? nullptr : &tensor(v[5], "rows");
    if (rows) {
      on(*rows, "rows", device);
      contiguous(*rows, "rows");
      typed(*rows, "rows", rows->scalar_type() == at::kInt, "torch.int32");
    }
    const int64_t R = rows ? rows->numel() : T;
    at::Tensor Y, ws;
    if (v[6] != Py_None) {
      Y = tensor(v[6], "Y");
      on(Y, "Y", device);
      contiguous(Y, "Y");
      typed(Y, "Y", Y.scalar_type() == at::kBFloat16 || Y.scalar_type() == at::kShort, "torch.bfloat16");
      if (Y.dim() != 2 || Y.size(0) != R || Y.size(1) != N)
        refuse("Y has shape %s, expected (%lld, %lld)", shape_of(Y).c_str(), (long long)R, (long long)N);
    }
    if (v[7] != Py_None) {
      ws = tensor(v[7], "workspace");
      on(ws, "workspace", device);
      contiguous(ws, "workspace");
    }
    const uint32_t flags = flag_bits(v[8], "flags");
    const Launch launch = launch_of(v[9], device);
    {
      Unlocked u;
      Pool pool(launch);
      uint64_t bytes = 0;
      if (!ws.defined()) {
        check(fg_grouped_gemm_workspace_size(mode, R, (int)E, N, K, rows != nullptr, &bytes));
        if (bytes) ws = make({static_cast<int64_t>(bytes)}, at::kByte, device);
      } else {
        bytes = ws.numel() * ws.element_size();
      }
      if (!Y.defined()) Y = make({R, N}, at::kBFloat16, device);
      check(fg_grouped_gemm(A.data_ptr(), scales ? scales->data_ptr() : nullptr, T, rows ? rows->data_ptr<int32_t>() : nullptr, R,
                            offsets.data_ptr<int32_t>(), (int)E, b, mode, Y.data_ptr(), data(ws), bytes, flags,
                            launch.stream));
      keep(launch, {&Y}, {&A, &weight, &offsets, scales, rows, &Y, &ws});
    }
    return wrap(Y);
  });
}

// (Y, slots, weights, residual or None, stream) -> out
PyObject* moe_combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 5, "moe_combine");
    const at::Tensor& Y = tensor(a[0], "Y");
    const at::Device device = Y.device();
    contiguous(Y, "Y");
    typed(Y, "Y", Y.scalar_type() == at::kBFloat16, "torch.bfloat16");
    const at::Tensor& slots = tensor(a[1], "slots");
    on(slots, "slots", device);
    contiguous(slots, "slots");
    typed(slots, "slots", slots.scalar_type() == at::kInt, "torch.int32");
    if (Y.dim() != 2 || slots.dim() != 2)
      refuse("Y and slots must be 2-D, got shapes %s and %s", shape_of(Y).c_str(), shape_of(slots).c_str());
    const int64_t t = slots.size(0), k = slots.size(1), cols = Y.size(1);
    const at::Tensor& w = tensor(a[2], "weights");
    on(w, "weights", device);
    contiguous(w, "weights");
    typed(w, "weights", w.scalar_type() == at::kFloat, "torch.float32");
    if (w.sizes() != slots.sizes())
      refuse("weights has shape %s, expected %s", shape_of(w).c_str(), shape_of(slots).c_str());
    const at::Tensor* r = a[3] == Py_None ? nullptr : &tensor(a[3], "residual");
    if (r) {
      on(*r, "residual", device);
      contiguous(*r, "residual");
      typed(*r, "residual", r->scalar_type() == at::kBFloat16, "torch.bfloat16");
      if (r->dim() != 2 || r->size(0) != t || r->size(1) != cols)
        refuse("residual has shape %s, expected (%lld, %lld)", shape_of(*r).c_str(), (long long)t, (long long)cols);
    }
    const Launch launch = launch_of(a[4], device);
    at::Tensor out;
    {
      Unlocked u;
      Pool pool(launch);
      out = make({t, cols}, at::kBFloat16, device);
      check(fg_moe_combine(Y.data_ptr(), Y.size(0), slots.data_ptr<int32_t>(), w.data_ptr<float>(), r ? r->data_ptr() : nullptr, t,
                           (int)(k < 1024 ? k : 1024), cols, out.data_ptr(), launch.stream));
      keep(launch, {&out}, {&Y, &slots, &w, r});
    }
    return wrap(out);
  });
}

// fg_gemm's ordinary call, (A, weight data, descriptor's address, a_scales or
// None, split_k, stream) -> Y; None where an argument is not as it should be or needs
// more than this, which the caller's own checks then name.
PyObject* gemm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 6, "gemm");
    if (!THPVariable_Check(v[0]) || !THPVariable_Check(v[1]) || !PyLong_Check(v[4])) Py_RETURN_NONE;
    const at::Tensor &A = THPVariable_Unpack(v[0]), &weight = THPVariable_Unpack(v[1]);
    const fg_bshuf* b = reinterpret_cast<const fg_bshuf*>(static_cast<intptr_t>(integer(v[2], "the descriptor's address")));
    const int mode = b->mode;
    const int64_t K = b->K;
    const at::Device device = weight.device();
    const at::ScalarType type = A.scalar_type();
    const int64_t row = mode == FG_BF16 ? 2 * K : (mode == FG_MXFP4 ? K / 2 : K);
    const bool codes = mode == FG_BF16 ? type == at::kBFloat16 || type == at::kShort || type == at::kUInt16
                                       : is_bytes(type) || type == (mode == FG_MXFP4 ? at::kFloat4_e2m1fn_x2 : at::kFloat8_e4m3fn);
    if (!weight.is_cuda() || device.index() != c10::cuda::current_device() || A.device() != device || !A.is_contiguous() ||
        A.dim() != 2 || A.size(0) == 0 || !codes || A.size(1) * (int64_t)A.element_size() != row)
      Py_RETURN_NONE;
    const int64_t M = A.size(0);
    const void* scales = nullptr;
    const at::Tensor* a_scales = nullptr;
    if (mode != FG_BF16) {
      if (!THPVariable_Check(v[3])) Py_RETURN_NONE;
      const at::Tensor& s = THPVariable_Unpack(v[3]);
      a_scales = &s;
      const bool fp32 = mode == FG_FP8_TENSOR || mode == FG_FP8_BLOCK128;
      const int64_t want = mode == FG_FP8_TENSOR ? 1 : M * (K / (mode == FG_MXFP8 || mode == FG_FP8_BLOCK128 ? 128 : 32));
      const at::ScalarType t = s.scalar_type();
      if (s.device() != device || !s.is_contiguous() || s.numel() != want ||
          !(fp32 ? t == at::kFloat : is_bytes(t) || t == at::kFloat8_e8m0fnu))
        Py_RETURN_NONE;
      scales = s.data_ptr();
    } else if (v[3] != Py_None) {
      Py_RETURN_NONE;
    }
    const long split = PyLong_AsLong(v[4]);
    if (PyErr_Occurred()) return nullptr;
    if (split < 0 || split > 16) Py_RETURN_NONE;
    const Launch launch = launch_of(v[5], device);
    at::Tensor Y, ws;
    {
      Unlocked u;
      Pool pool(launch);
      uint64_t need = 0;
      check(fg_gemm_workspace_size(mode, M, b->N, K, (int)split, &need));
      Y = make({M, b->N}, at::kBFloat16, device);
      if (need) ws = make({static_cast<int64_t>(need)}, at::kByte, device);
      check(fg_gemm(A.data_ptr(), scales, M, b, mode, (int)split, Y.data_ptr(), data(ws), need, 0, launch.stream));
      keep(launch, {&Y}, {&A, &weight, a_scales});
    }
    return wrap(Y);
  });
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef fast(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {fast<quantize>("quantize"),
                         fast<rmsnorm_quantize>("rmsnorm_quantize"),
                         fast<moe_route>("moe_route"),
                         fast<grouped_gemm>("grouped_gemm"),
                         fast<moe_combine>("moe_combine"),
                         fast<gemm>("gemm"),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "fg_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fg_torch() { return PyModule_Create(&module); }
