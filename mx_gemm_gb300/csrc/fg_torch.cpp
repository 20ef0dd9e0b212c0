// Python binding of the operators around the GEMM (mx_gemm_gb300/moe.py, train.py)
// and of the GEMM's ordinary call: the checks of their tensors, their outputs'
// allocation, and the call of the C ABI.  A call of theirs on one token keeps the GPU busy for 2 to 5 us, while
// allocating each output from Python takes 1.5 us and a ctypes call of fifteen
// arguments as much again (routing: 17 us a call that way); from here the same
// steps cost a third of it.
//
// Errors: ValueError for tensors that the library would misread, the package's
// FgError for a status of the C ABI, and torch's own for the allocations.
#define PY_SSIZE_T_CLEAN  // "y#" takes a Py_ssize_t
#include <Python.h>
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <cstdarg>
#include <cstdio>
#include <string>
#include <utility>

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

// Tensors that always go together, in one allocation, which costs the host about as
// much as a launch: values and their scales, a loss and what comes with it.  Each begins
// at a multiple of 128 bytes.
struct Shape {
  at::IntArrayRef sizes;
  at::ScalarType type;
};

template <size_t N>
std::array<at::Tensor, N> make_together(const Shape (&what)[N], const at::Device& device) {
  int64_t at[N], bytes = 0;
  for (size_t i = 0; i < N; ++i) {
    at[i] = bytes = (bytes + 127) / 128 * 128;
    int64_t n = static_cast<int64_t>(c10::elementSize(what[i].type));
    for (const int64_t d : what[i].sizes) n *= d;
    bytes += n;
  }
  const at::Tensor whole = make({bytes}, at::kByte, device);
  std::array<at::Tensor, N> out;
  for (size_t i = 0; i < N; ++i) {
    out[i] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(),
                                                      c10::scalarTypeToTypeMeta(what[i].type));
    c10::TensorImpl* t = out[i].unsafeGetTensorImpl();
    t->set_storage_offset(at[i] / static_cast<int64_t>(c10::elementSize(what[i].type)));
    t->set_sizes_contiguous(what[i].sizes);
  }
  return out;
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

// together: in one allocation (0.4 us of host time less), for what a training step makes
// and drops as one.  quantize() and rmsnorm_quantize() give each its own: theirs are kept,
// and saved to files, one without the other.
Codes make_codes(int mode, int64_t m, int64_t k, const at::Device& device, bool together) {
  const bool half = mode == FG_MXFP4, wide = mode == FG_FP8_BLOCK128;
  const int64_t of_codes[] = {m, half ? k / 2 : k}, of_scales[] = {m, k / (wide || mode == FG_MXFP8 ? 128 : 32)};
  const Shape parts[] = {{of_codes, half ? at::kByte : at::kFloat8_e4m3fn}, {of_scales, wide ? at::kFloat : at::kFloat8_e8m0fnu}};
  if (!together) return {make(parts[0].sizes, parts[0].type, device), make(parts[1].sizes, parts[1].type, device)};
  auto [codes, scales] = make_together(parts, device);
  return {std::move(codes), std::move(scales)};
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
      c = make_codes(mode, r.m, r.k, device, false);
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
      if (!plain) c = make_codes(mode, r.m, r.k, device, false);
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
//  Y or None, workspace or None, flags, stream, weight's scale image or None) -> Y
PyObject* grouped_gemm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 11, "grouped_gemm");
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
    const at::Tensor* sf = v[10] == Py_None ? nullptr : &tensor(v[10], "the scale image");
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
      keep(launch, {&Y}, {&A, &weight, sf, &offsets, scales, rows, &Y, &ws});
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

// ------------------------------------------------- training in 8 bits

// A 1-D or 2-D int32 index tensor of the operands' device.
const at::Tensor* indexes(PyObject* o, const char* name, const at::Device& device) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  on(t, name, device);
  contiguous(t, name);
  typed(t, name, t.scalar_type() == at::kInt, "torch.int32");
  return &t;
}

const at::Tensor* floats(PyObject* o, const char* name, const at::Device& device) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  on(t, name, device);
  contiguous(t, name);
  typed(t, name, t.scalar_type() == at::kFloat, "torch.float32");
  return &t;
}

const int32_t* ints(const at::Tensor* t) { return t ? t->data_ptr<int32_t>() : nullptr; }

// Experts of offsets [E + 1]; 1 without any.
int experts_of(const at::Tensor* offsets) {
  if (!offsets) return 1;
  if (offsets->dim() != 1 || offsets->numel() < 2 || offsets->numel() > INT32_MAX)
    refuse("offsets must hold E + 1 values, got shape %s", shape_of(*offsets).c_str());
  return static_cast<int>(offsets->numel() - 1);
}

// Codes [M][K] of an 8-bit mode and their scales, as quantize() makes them.
void check_codes(int mode, const at::Tensor& codes, const at::Tensor& scales, const char* name, const at::Device& device,
                 int64_t m, int64_t k) {
  on(codes, name, device);
  contiguous(codes, name);
  typed(codes, name, is_bytes(codes.scalar_type()) || codes.scalar_type() == at::kFloat8_e4m3fn, "torch.float8_e4m3fn or bytes");
  if (codes.dim() != 2 || codes.size(0) != m || codes.size(1) != k)
    refuse("%s has shape %s, expected (%lld, %lld)", name, shape_of(codes).c_str(), (long long)m, (long long)k);
  on(scales, "its scales", device);
  contiguous(scales, "its scales");
  const at::ScalarType s = scales.scalar_type();
  if (mode == FG_FP8_BLOCK128) typed(scales, "its scales", s == at::kFloat, "torch.float32");
  else typed(scales, "its scales", is_bytes(s) || s == at::kFloat8_e8m0fnu, "torch.float8_e8m0fnu or bytes");
  const int64_t want = m * (k / (mode == FG_MXFP8 || mode == FG_FP8_BLOCK128 ? 128 : 32));
  if (scales.numel() != want)
    refuse("%s of shape (%lld, %lld) has %lld scales, expected %lld", name, (long long)m, (long long)k, (long long)scales.numel(),
           (long long)want);
}

struct ColumnOperand {
  at::Tensor data, sf;
  fg_bshuf desc;
};

void make_columns(ColumnOperand& c, int64_t columns, int64_t rows, int experts, const at::Device& device) {
  int64_t places = 0;
  uint64_t data_bytes = 0, sf_bytes = 0;
  check(fg_columns_size(columns, rows, experts, &places, &data_bytes, &sf_bytes));
  auto [data, sf] =
      make_together({{{static_cast<int64_t>(data_bytes)}, at::kByte}, {{static_cast<int64_t>(sf_bytes)}, at::kByte}}, device);
  c.data = std::move(data);
  c.sf = std::move(sf);
}

PyObject* wrap(const ColumnOperand& c) {
  return Py_BuildValue("(NNy#)", wrap(c.data), wrap(c.sf), reinterpret_cast<const char*>(&c.desc),
                       static_cast<Py_ssize_t>(sizeof c.desc));
}

// (mode, w, transpose, stream) -> (codes, scales)
PyObject* quantize_weight(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 4, "quantize_weight");
    const int mode = small(a[0], "mode");
    const at::Tensor& w = tensor(a[1], "w");
    const int type = type_of(w, "w");
    if (w.dim() != 2 && w.dim() != 3) refuse("w must be [N][K] or [E][N][K], got shape %s", shape_of(w).c_str());
    const int64_t d = w.dim(), E = d == 3 ? w.size(0) : 1, N = w.size(d - 2), K = w.size(d - 1);
    if (w.stride(d - 1) != 1 && K > 1) refuse("w must have contiguous rows (shape %s)", shape_of(w).c_str());
    if (E < 1 || E > INT32_MAX) refuse("w has no experts (shape %s)", shape_of(w).c_str());
    const int64_t ld = N > 1 ? w.stride(d - 2) : K, stride = d == 3 ? w.stride(0) : 0;
    const bool transpose = truth(a[2], "transpose");
    const at::Device device = w.device();
    const Launch launch = launch_of(a[3], device);
    at::Tensor codes, scales;
    {
      Unlocked u;
      Pool pool(launch);
      const int64_t rows = transpose ? K : N, cols = transpose ? N : K;
      auto both = make_together({{{E * rows, cols}, at::kFloat8_e4m3fn}, {{E * rows / 128, cols / 128}, at::kFloat}}, device);
      codes = std::move(both[0]);
      scales = std::move(both[1]);
      check(fg_quantize_weight(mode, w.data_ptr(), type, (int)E, N, K, ld, stride, transpose, codes.data_ptr(), scales.data_ptr(),
                               launch.stream));
      keep(launch, {&codes, &scales}, {&w});
    }
    return Py_BuildValue("(NN)", wrap(codes), wrap(scales));
  });
}

// (mode, x, stream) -> (codes, scales, saved, saved scales)
PyObject* swiglu_checkpoint(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 3, "swiglu_checkpoint");
    const int mode = small(a[0], "mode");
    if (mode == FG_MXFP4) refuse("mode mxfp4 keeps no 8-bit blocks");  // (its codes would be made half as wide)
    const at::Tensor& x = tensor(a[1], "x");
    const Rows r = rows_of(x, "x");
    const int type = type_of(x, "x");
    if (r.k % 2) refuse("x must have rows (g, u) of two equal halves, got %lld columns", (long long)r.k);
    const at::Device device = x.device();
    const Launch launch = launch_of(a[2], device);
    Codes c, s;
    {
      Unlocked u;
      Pool pool(launch);
      c = make_codes(mode, r.m, r.k / 2, device, true);
      s = make_codes(mode, r.m, r.k, device, true);
      check(fg_swiglu_checkpoint(mode, x.data_ptr(), type, r.m, r.k / 2, r.ld, c.codes.data_ptr(), c.scales.data_ptr(),
                                 s.codes.data_ptr(), s.scales.data_ptr(), launch.stream));
      keep(launch, {&c.codes, &c.scales, &s.codes, &s.scales}, {&x});
    }
    return Py_BuildValue("(NNNN)", wrap(c.codes), wrap(c.scales), wrap(s.codes), wrap(s.scales));
  });
}

// (x, offsets or None, scales or None, rows or None, stream) -> ((data, sf, descriptor), R, E)
PyObject* quantize_columns(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 5, "quantize_columns");
    const at::Tensor& x = tensor(a[0], "x");
    const at::Device device = x.device();
    const Rows r = rows_of(x, "x");
    const at::Tensor* offsets = indexes(a[1], "offsets", device);
    const int E = experts_of(offsets);
    const at::Tensor* scales = nullptr;
    int mode = FG_BF16, type = FG_TYPE_BF16;
    if (a[2] == Py_None) {
      type = type_of(x, "x");
    } else {
      scales = &tensor(a[2], "scales");
      mode = scales->scalar_type() == at::kFloat ? FG_FP8_BLOCK128
             : scales->numel() * 128 == r.m * r.k && r.m * r.k > 0 ? FG_MXFP8 : FG_MXFP8_B32;
      check_codes(mode, x, *scales, "x", device, r.m, r.k);
    }
    const at::Tensor* rows = indexes(a[3], "rows", device);
    const int64_t R = rows ? rows->numel() : r.m;
    const Launch launch = launch_of(a[4], device);
    ColumnOperand c;
    {
      Unlocked u;
      Pool pool(launch);
      make_columns(c, r.k, R, E, device);
      check(fg_quantize_columns(mode, x.data_ptr(), scales ? scales->data_ptr() : nullptr, type, r.m, r.k, scales ? r.k : r.ld,
                                ints(rows), R, ints(offsets), E, c.data.data_ptr(), c.sf.data_ptr(), &c.desc, launch.stream));
      keep(launch, {&c.data, &c.sf}, {&x, offsets, scales, rows});
    }
    return Py_BuildValue("(NLi)", wrap(c), (long long)R, E);
  });
}

// (mode, dy, saved, saved scales, weights, rows, slots, offsets (None: without routing), columns, plain, stream)
//   -> (codes, scales, dx, dweights, dx's columns or None, act's columns or None, R, E)
PyObject* swiglu_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 11, "swiglu_backward");
    const int mode = small(a[0], "mode");
    if (mode != FG_MXFP8 && mode != FG_MXFP8_B32 && mode != FG_MXFP4_FP8A && mode != FG_FP8_BLOCK128)
      refuse("mode %d keeps no 8-bit blocks", mode);
    const at::Tensor& dy = tensor(a[1], "dy");
    const at::Device device = dy.device();
    const Rows r = rows_of(dy, "dy");
    const int type = type_of(dy, "dy");
    const at::Tensor &saved = tensor(a[2], "saved"), &saved_scales = tensor(a[3], "saved_scales");
    check_codes(mode, saved, saved_scales, "saved", device, r.m, 2 * r.k);
    const at::Tensor* weights = floats(a[4], "weights", device);
    const at::Tensor* rows = indexes(a[5], "rows", device);
    const at::Tensor* slots = indexes(a[6], "slots", device);
    const at::Tensor* offsets = indexes(a[7], "offsets", device);
    const int E = experts_of(offsets);
    int64_t T = 0, k = 0;
    if (weights) {
      if (!rows || !slots || !offsets) refuse("weights need rows, slots and offsets");
      if (slots->dim() != 2 || weights->sizes() != slots->sizes())
        refuse("weights and slots must be [T][top_k], got shapes %s and %s", shape_of(*weights).c_str(), shape_of(*slots).c_str());
      T = slots->size(0);
      k = slots->size(1);
      if (rows->numel() != r.m || T * k != r.m)
        refuse("dy has %lld rows, the routing %lld choices and %lld rows", (long long)r.m, (long long)(T * k), (long long)rows->numel());
    }
    const bool columns = truth(a[8], "columns"), plain = truth(a[9], "plain");
    const Launch launch = launch_of(a[10], device);
    Codes c;
    at::Tensor dx, dweights, ws;
    ColumnOperand dxc, actc;
    {
      Unlocked u;
      Pool pool(launch);
      uint64_t need = 0;
      if (r.m > 0 || columns) check(fg_swiglu_backward_workspace_size(r.m, r.k, weights != nullptr, &need));
      if (need) ws = make({static_cast<int64_t>(need)}, at::kByte, device);
      c = make_codes(mode, r.m, 2 * r.k, device, true);
      if (plain) dx = make({r.m, 2 * r.k}, dy.scalar_type(), device);
      if (weights) dweights = make({T, k}, at::kFloat, device);
      if (columns) {
        make_columns(dxc, 2 * r.k, r.m, E, device);
        make_columns(actc, r.k, r.m, E, device);
      }
      check(fg_swiglu_backward(mode, dy.data_ptr(), type, r.m, r.k, r.ld, saved.data_ptr(), saved_scales.data_ptr(),
                               weights ? weights->data_ptr<float>() : nullptr, ints(rows), ints(slots), T,
                               (int)(k < 1024 ? k : 1024), ints(offsets), E, c.codes.data_ptr(), c.scales.data_ptr(), data(dx),
                               dweights.defined() ? dweights.data_ptr<float>() : nullptr, data(dxc.data), data(dxc.sf), &dxc.desc,
                               data(actc.data), data(actc.sf), &actc.desc, data(ws), need, launch.stream));
      keep(launch, {&c.codes, &c.scales, &dx, &dweights, &dxc.data, &dxc.sf, &actc.data, &actc.sf},
           {&dy, &saved, &saved_scales, weights, rows, slots, offsets});
    }
    PyObject* of_dx = columns ? wrap(dxc) : Py_NewRef(Py_None);
    PyObject* of_act = columns ? wrap(actc) : Py_NewRef(Py_None);
    return Py_BuildValue("(NNNNNNLi)", wrap(c.codes), wrap(c.scales), wrap(dx), wrap(dweights), of_dx, of_act, (long long)r.m, E);
  });
}

// (a's data, sf and descriptor's address, b's, offsets, R, E, out or None, accumulate, type, flags, stream) -> out
PyObject* grouped_wgrad(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 14, "grouped_wgrad");
    const at::Tensor* t[4];
    const fg_bshuf* d[2];
    const at::Device device = tensor(v[0], "a").device();
    for (int i = 0; i < 2; ++i) {
      t[2 * i] = &tensor(v[3 * i], i ? "b" : "a");
      t[2 * i + 1] = &tensor(v[3 * i + 1], "the scale image");
      on(*t[2 * i], i ? "b" : "a", device);
      on(*t[2 * i + 1], "the scale image", device);
      d[i] = reinterpret_cast<const fg_bshuf*>(static_cast<intptr_t>(integer(v[3 * i + 2], "the descriptor's address")));
      if (d[i]->data != t[2 * i]->data_ptr() || d[i]->sf != t[2 * i + 1]->data_ptr())
        refuse("the column operand's tensors are not those of its descriptor");
    }
    const at::Tensor* offsets = indexes(v[6], "offsets", device);
    if (!offsets) refuse("offsets must be a torch.Tensor");
    const int64_t R = integer(v[7], "rows");
    const int E = small(v[8], "experts");
    if (experts_of(offsets) != E) refuse("offsets hold %d experts, the operands %d", experts_of(offsets), E);
    const int64_t N = d[0]->N, K = d[1]->N;
    const bool accumulate = truth(v[10], "accumulate");
    const int type = small(v[11], "dtype");
    at::Tensor out;
    if (v[9] != Py_None) {
      out = tensor(v[9], "out");
      on(out, "out", device);
      contiguous(out, "out");
      typed(out, "out", out.scalar_type() == (type == FG_TYPE_F32 ? at::kFloat : at::kBFloat16), "that of dtype");
      if (out.dim() != 3 || out.size(0) != E || out.size(1) != N || out.size(2) != K)
        refuse("out has shape %s, expected (%d, %lld, %lld)", shape_of(out).c_str(), E, (long long)N, (long long)K);
    } else if (accumulate) {
      refuse("accumulate needs out");
    }
    const uint32_t flags = flag_bits(v[12], "flags");
    const Launch launch = launch_of(v[13], device);
    {
      Unlocked u;
      Pool pool(launch);
      if (!out.defined()) out = make({E, N, K}, type == FG_TYPE_F32 ? at::kFloat : at::kBFloat16, device);
      check(fg_grouped_wgrad(d[0], d[1], ints(offsets), R, E, type, accumulate, out.data_ptr(), flags, launch.stream));
      keep(launch, {&out}, {t[0], t[1], t[2], t[3], offsets, &out});
    }
    return wrap(out);
  });
}

// (logits, offsets, coefficient, stream) -> (loss, counts, probs, slopes)
PyObject* moe_balance_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 4, "moe_balance_loss");
    const at::Tensor& x = tensor(a[0], "logits");
    const Rows r = rows_of(x, "logits");
    const int type = type_of(x, "logits");
    const at::Device device = x.device();
    const at::Tensor* offsets = indexes(a[1], "offsets", device);
    if (!offsets || offsets->dim() != 1 || offsets->numel() != r.k + 1)
      refuse("offsets must hold E + 1 = %lld values", (long long)(r.k + 1));
    const double coefficient = PyFloat_AsDouble(a[2]);
    if (coefficient == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      refuse("coefficient must be a number");
    }
    const Launch launch = launch_of(a[3], device);
    at::Tensor loss, counts, probs, slopes, ws;
    {
      Unlocked u;
      Pool pool(launch);
      const int E = (int)(r.k < (1 << 30) ? r.k : 1 << 30);
      uint64_t need = 0;
      check(fg_moe_balance_loss_workspace_size(r.m, E, &need));
      if (need) ws = make({static_cast<int64_t>(need)}, at::kByte, device);
      auto all = make_together({{{}, at::kFloat}, {{r.k}, at::kInt}, {{r.k}, at::kFloat}, {{r.k}, at::kFloat}}, device);
      loss = std::move(all[0]);
      counts = std::move(all[1]);
      probs = std::move(all[2]);
      slopes = std::move(all[3]);
      check(fg_moe_balance_loss(x.data_ptr(), type, r.m, E, r.ld, ints(offsets), (float)coefficient, loss.data_ptr<float>(),
                                counts.data_ptr<int32_t>(), probs.data_ptr<float>(), slopes.data_ptr<float>(), data(ws), need,
                                launch.stream));
      keep(launch, {&loss, &counts, &probs, &slopes}, {&x, offsets});
    }
    return Py_BuildValue("(NNNN)", wrap(loss), wrap(counts), wrap(probs), wrap(slopes));
  });
}

// (logits, experts or None, dweights or None, slopes or None, renormalize, stream) -> gradient of the logits
PyObject* moe_route_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 6, "moe_route_backward");
    const at::Tensor& x = tensor(a[0], "logits");
    const Rows r = rows_of(x, "logits");
    const int type = type_of(x, "logits");
    const at::Device device = x.device();
    const at::Tensor* experts = indexes(a[1], "experts", device);
    const at::Tensor* dweights = floats(a[2], "dweights", device);
    const at::Tensor* slopes = floats(a[3], "slopes", device);
    int64_t k = 0;
    if (dweights) {
      if (!experts || experts->dim() != 2 || experts->size(0) != r.m || dweights->sizes() != experts->sizes())
        refuse("dweights has shape %s, expected that of the routing's experts, [%lld][top_k]", shape_of(*dweights).c_str(),
               (long long)r.m);
      k = experts->size(1);
    }
    if (slopes && (slopes->dim() != 1 || slopes->numel() != r.k))
      refuse("slopes has shape %s, expected (%lld,)", shape_of(*slopes).c_str(), (long long)r.k);
    const bool renormalize = truth(a[4], "renormalize");
    const Launch launch = launch_of(a[5], device);
    at::Tensor out;
    {
      Unlocked u;
      Pool pool(launch);
      out = make({r.m, r.k}, x.scalar_type(), device);
      check(fg_moe_route_backward(x.data_ptr(), type, r.m, (int)(r.k < (1 << 30) ? r.k : 1 << 30), r.ld, ints(experts),
                                  dweights ? dweights->data_ptr<float>() : nullptr, (int)(k < 1024 ? k : 1024),
                                  slopes ? slopes->data_ptr<float>() : nullptr, renormalize ? FG_FLAG_RENORMALIZE : 0,
                                  out.data_ptr(), launch.stream));
      keep(launch, {&out}, {&x, experts, dweights, slopes});
    }
    return wrap(out);
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
                         fast<quantize_weight>("quantize_weight"),
                         fast<swiglu_checkpoint>("swiglu_checkpoint"),
                         fast<quantize_columns>("quantize_columns"),
                         fast<swiglu_backward>("swiglu_backward"),
                         fast<grouped_wgrad>("grouped_wgrad"),
                         fast<moe_balance_loss>("moe_balance_loss"),
                         fast<moe_route_backward>("moe_route_backward"),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "fg_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fg_torch() { return PyModule_Create(&module); }
