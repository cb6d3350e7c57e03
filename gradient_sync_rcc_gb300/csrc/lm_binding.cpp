// lm_binding.cpp -- the language-model operators for torch tensors, as a
// CPython module: argument checks, outputs and workspaces that the caller left
// out, and the call of librcc's C entry point.  On small inputs the time of a
// call is the host's; through ctypes a lookup of 8 tokens took 10 us of it.
//
// librcc is not linked: lm.py hands over the addresses of its entry points,
// so the library that the rest of the binding loaded is the one that runs.
#include <Python.h>

#include <ATen/Context.h>
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <ATen/record_function.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <stdexcept>

#include "rcc.h"

namespace {

// ---- librcc ---------------------------------------------------------------------

struct Entries {
  decltype(&rcc_embedding_forward) embedding_forward;
  decltype(&rcc_embedding_backward) embedding_backward;
  decltype(&rcc_embedding_backward_workspace) embedding_backward_workspace;
  decltype(&rcc_rmsnorm_forward) rmsnorm_forward;
  decltype(&rcc_rmsnorm_backward) rmsnorm_backward;
  decltype(&rcc_rmsnorm_backward_workspace) rmsnorm_backward_workspace;
  decltype(&rcc_linear_ce_forward) linear_ce_forward;
  decltype(&rcc_linear_ce_backward) linear_ce_backward;
  decltype(&rcc_linear_ce_workspace) linear_ce_workspace;
  decltype(&rcc_add_rmsnorm_forward) add_rmsnorm_forward;
  decltype(&rcc_add_rmsnorm_backward) add_rmsnorm_backward;
  decltype(&rcc_rotary_forward) rotary_forward;
  decltype(&rcc_rotary_backward) rotary_backward;
  decltype(&rcc_adamw_step) adamw_step;
} rcc_;
PyObject* on_error = nullptr;  // called with a status that is not RCC_OK; raises

// ---- arguments ------------------------------------------------------------------

// An argument that does not fit: a ValueError
struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
[[noreturn]] void refuse(const char* fmt, ...) {
  char text[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof(text), fmt, ap);
  va_end(ap);
  throw Refused(text);
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse("%s must be a tensor", what);
  return THPVariable_Unpack(o);
}
bool given(PyObject* o) { return o != Py_None; }

bool dtype_of(at::ScalarType t, rcc_dtype* out) {
  if (t == at::kBFloat16) *out = RCC_BF16;
  else if (t == at::kFloat) *out = RCC_F32;
  else return false;
  return true;
}
rcc_dtype dtype_of(const at::Tensor& t, const char* what) {
  rcc_dtype d;
  if (!dtype_of(t.scalar_type(), &d)) refuse("%s must be float32 or bfloat16", what);
  return d;
}
at::ScalarType scalar_of(rcc_dtype d) { return d == RCC_BF16 ? at::kBFloat16 : at::kFloat; }
rcc_dtype dtype_arg(PyObject* o, const char* what) {
  rcc_dtype d;
  if (!THPDtype_Check(o) || !dtype_of(reinterpret_cast<THPDtype*>(o)->scalar_type, &d))
    refuse("%s must be torch.float32 or torch.bfloat16", what);
  return d;
}

// A matrix whose rows are contiguous
struct Matrix {
  int64_t rows, cols, ld;
};
Matrix matrix(const at::Tensor& t, const char* what, at::Device dev) {
  if (t.dim() != 2 || t.device() != dev) refuse("%s must be a matrix on the inputs' device", what);
  const int64_t n = t.size(0), d = t.size(1);
  if (d != 1 && t.stride(1) != 1) refuse("the rows of %s must be contiguous", what);
  if (n < 2) return {n, d, d};
  if (t.stride(0) < d) refuse("the rows of %s overlap", what);
  return {n, d, t.stride(0)};
}
rcc_index index_of(const at::Tensor& t, const char* what, at::Device dev, int64_t n) {
  const auto s = t.scalar_type();
  if ((s != at::kInt && s != at::kLong) || t.dim() != 1 || t.device() != dev || t.numel() != n ||
      !t.is_contiguous())
    refuse("%s must be a contiguous vector of %lld int32 or int64 on the inputs' device", what,
           (long long)n);
  return s == at::kLong ? RCC_I64 : RCC_I32;
}
float* floats(const at::Tensor& t, const char* what, at::Device dev, int64_t n) {
  if (t.scalar_type() != at::kFloat || t.dim() != 1 || t.device() != dev || t.numel() != n ||
      !t.is_contiguous())
    refuse("%s must be a contiguous vector of %lld float32 on the inputs' device", what,
           (long long)n);
  return static_cast<float*>(t.data_ptr());
}

// Whether someone looks at new tensors on their way through the dispatcher: a mode
// (each has a key of its own in the thread's set), a profiler, the filling of new
// memory in deterministic runs
bool watched() {
  const at::Context& c = at::globalContext();
  return !(c10::impl::tls_local_dispatch_key_set().included_ - c10::default_included_set).empty() ||
         at::getStepCallbacksUnlessEmpty(at::RecordScope::FUNCTION).has_value() ||
         (c.deterministicAlgorithms() && c.deterministicFillUninitializedMemory());
}
// at::empty, or where nobody looks what it comes to, without the 0.5 to 1 us of its
// way there (three new tensors, forward with a kept input: 6.0 us of host time a call
// instead of 7.5)
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
  if (watched()) return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
  return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}
// The caller's output, checked, or a new one
at::Tensor output(PyObject* o, const char* what, at::IntArrayRef shape, at::ScalarType type,
                  at::Device dev) {
  if (!given(o)) return fresh(shape, type, dev);
  const at::Tensor& t = tensor(o, what);
  if (t.sizes() != shape || t.scalar_type() != type || t.device() != dev || !t.is_contiguous())
    refuse("%s must be a contiguous tensor of its type and shape on the inputs' device", what);
  return t;
}
struct Workspace {
  at::Tensor t;
  void* p;
  size_t bytes;
};
Workspace workspace(PyObject* o, size_t need, at::Device dev) {
  if (!given(o)) {
    at::Tensor t = fresh({(int64_t)need}, at::kByte, dev);
    void* p = t.data_ptr();
    return {std::move(t), p, need};
  }
  const at::Tensor& t = tensor(o, "workspace");
  if (t.device() != dev || !t.is_contiguous())
    refuse("the workspace must be a contiguous tensor on the inputs' device");
  return {t, t.data_ptr(), (size_t)t.nbytes()};
}

// librcc launches on the current device, whose default stream goes by the same
// handle as any other's
void require_current(int device, int current) {
  if (device != current)
    refuse("current CUDA device %d is not the inputs' device %d", current, device);
}

// The stream of a call: the caller's (an address or an object with
// cuda_stream), or the current one.  The last check of a call: nothing before
// it needs a GPU.  While this lives the stream is the current one, so what a
// call allocates belongs to it: a block comes without work of another stream
// still queued on it, and a released workspace is given out again on this
// stream alone, behind the kernels that still use it.
class Stream {
 public:
  Stream(PyObject* o, at::Device dev) {
    if (!dev.is_cuda()) refuse("the operators take tensors on a CUDA device");
    require_current(dev.index(), c10::cuda::current_device());
    handle_ = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    if (!given(o)) return;
    PyObject* v = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
    if (!v) throw python_error();
    auto asked = static_cast<cudaStream_t>(PyLong_AsVoidPtr(v));
    Py_DECREF(v);
    if (PyErr_Occurred()) throw python_error();
    if (asked == cudaStreamLegacy) asked = nullptr;  // two names of the default stream
    if (asked == handle_) return;
    handle_ = asked;
    current_.reset_stream(c10::cuda::getStreamFromExternal(asked, dev.index()));
  }
  rcc_stream_t handle() const { return reinterpret_cast<rcc_stream_t>(handle_); }

 private:
  cudaStream_t handle_;
  c10::cuda::OptionalCUDAStreamGuard current_;
};

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

void check(rcc_status st) {
  if (st == RCC_OK) return;
  PyObject* r = PyObject_CallFunction(on_error, "i", (int)st);  // raises
  Py_XDECREF(r);
  throw python_error();
}

// One C call, without the interpreter's lock
template <typename F, typename... A>
void call(F f, A... args) {
  rcc_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f(args...);
  Py_END_ALLOW_THREADS
  check(st);
}

// Runs `body` with `n` arguments; C++ exceptions become Python's
template <typename F>
PyObject* entry(const char* name, Py_ssize_t got, Py_ssize_t n, F body) {
  HANDLE_TH_ERRORS
  if (got != n) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, n, got);
    return nullptr;
  }
  try {
    return body();
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }
PyObject* wrap(at::Tensor a, at::Tensor b) {
  PyObject* r = PyTuple_New(2);
  if (!r) throw python_error();
  PyTuple_SET_ITEM(r, 0, a.defined() ? wrap(std::move(a)) : Py_NewRef(Py_None));
  PyTuple_SET_ITEM(r, 1, b.defined() ? wrap(std::move(b)) : Py_NewRef(Py_None));
  return r;
}

// ---- embedding ------------------------------------------------------------------

// table, ids, scale, out, out_dtype, stream
PyObject* embedding_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("embedding_forward", n, 6, [&] {
    const at::Tensor &table = tensor(a[0], "table"), &ids = tensor(a[1], "ids");
    const at::Device dev = table.device();
    const Matrix m = matrix(table, "table", dev);
    const int64_t tokens = ids.numel();
    const rcc_index index = index_of(ids, "ids", dev, tokens);
    const rcc_dtype kind = dtype_of(table, "table");
    rcc_dtype out_kind = kind;
    if (given(a[4])) out_kind = dtype_arg(a[4], "out_dtype");
    else if (given(a[3])) out_kind = dtype_of(tensor(a[3], "out"), "out");
    const float scale = (float)number(a[2]);
    at::Tensor out;
    if (given(a[3])) out = output(a[3], "out", {tokens, m.cols}, scalar_of(out_kind), dev);
    const Stream stream(a[5], dev);
    if (!out.defined()) out = fresh({tokens, m.cols}, scalar_of(out_kind), dev);
    call(rcc_.embedding_forward, table.data_ptr(), kind, (size_t)m.ld, ids.data_ptr(), index,
         (size_t)tokens, (size_t)m.rows, (size_t)m.cols, scale, out.data_ptr(), out_kind,
         stream.handle());
    return wrap(std::move(out));
  });
}

// dout, ids, dtable, scale, accumulate, workspace, stream
PyObject* embedding_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("embedding_backward", n, 7, [&] {
    const at::Tensor &dout = tensor(a[0], "dout"), &ids = tensor(a[1], "ids"),
                     &dtable = tensor(a[2], "dtable");
    const at::Device dev = dout.device();
    const Matrix m = matrix(dout, "dout", dev);
    if (dtable.dim() != 2 || dtable.size(1) != m.cols || dtable.device() != dev ||
        !dtable.is_contiguous())
      refuse("dtable must be a contiguous matrix of dout's %lld columns on the inputs' device",
             (long long)m.cols);
    const size_t vocab = dtable.size(0);
    const rcc_index index = index_of(ids, "ids", dev, m.rows);
    const rcc_dtype kind = dtype_of(dout, "dout"), grad = dtype_of(dtable, "dtable");
    const float scale = (float)number(a[3]);
    const int accumulate = truth(a[4]);
    const Stream stream(a[6], dev);
    const Workspace ws =
        workspace(a[5], rcc_.embedding_backward_workspace(m.rows, vocab, m.cols), dev);
    call(rcc_.embedding_backward, dout.data_ptr(), kind, (size_t)m.ld, ids.data_ptr(), index,
         (size_t)m.rows, vocab, (size_t)m.cols, scale, dtable.data_ptr(), grad, accumulate, ws.p,
         ws.bytes, stream.handle());
    return Py_NewRef(a[2]);
  });
}

// ---- RMS norm -------------------------------------------------------------------

constexpr int64_t kGroup = 128;
int64_t groups_of(int64_t dim) { return (dim + kGroup - 1) / kGroup; }

int64_t kept_bytes(int64_t tokens, int64_t dim) { return tokens * groups_of(dim) * (kGroup + 4); }

// The 8-bit form: values, then scales, in one buffer of bytes
struct Kept {
  int8_t* values;
  float* scales;
};
Kept kept_in(const at::Tensor& data, int64_t tokens, int64_t dim) {
  char* p = static_cast<char*>(data.data_ptr());
  return {reinterpret_cast<int8_t*>(p),
          reinterpret_cast<float*>(p + tokens * groups_of(dim) * kGroup)};
}
const at::Tensor& kept_arg(PyObject* data, PyObject* tokens, PyObject* dim, int64_t rows,
                           int64_t cols, at::Device dev) {
  const at::Tensor& t = tensor(data, "kept");
  const long long n = PyLong_AsLongLong(tokens), d = PyErr_Occurred() ? -1 : PyLong_AsLongLong(dim);
  if (PyErr_Occurred()) throw python_error();
  if (n != rows || d != cols || t.device() != dev)
    refuse("kept must hold %lld x %lld on the inputs' device", (long long)rows, (long long)cols);
  const int64_t need = kept_bytes(rows, cols);
  if (t.scalar_type() != at::kByte || !t.is_contiguous() || t.numel() < need)
    refuse("kept's buffer must be %lld contiguous bytes (uint8)", (long long)need);
  return t;
}

// x, weight, eps, keep (None, True, or a buffer), its tokens, its dim, out, stream
PyObject* rmsnorm_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("rmsnorm_forward", n, 8, [&] {
    const at::Tensor &x = tensor(a[0], "x"), &weight = tensor(a[1], "weight");
    const at::Device dev = x.device();
    const Matrix m = matrix(x, "x", dev);
    const rcc_dtype kind = dtype_of(x, "x");
    const float* w = floats(weight, "weight", dev, m.cols);
    const float eps = (float)number(a[2]);
    at::Tensor data;
    if (given(a[3]) && a[3] != Py_True) data = kept_arg(a[3], a[4], a[5], m.rows, m.cols, dev);
    const Stream stream(a[7], dev);
    at::Tensor y = output(a[6], "out", {m.rows, m.cols}, x.scalar_type(), dev);
    if (a[3] == Py_True)
      data = fresh({kept_bytes(m.rows, m.cols)}, at::kByte, dev);
    const Kept k = data.defined() ? kept_in(data, m.rows, m.cols) : Kept{nullptr, nullptr};
    call(rcc_.rmsnorm_forward, x.data_ptr(), kind, (size_t)m.ld, w, eps, (size_t)m.rows,
         (size_t)m.cols, y.data_ptr(), k.values, k.scales, stream.handle());
    return a[3] == Py_True ? wrap(std::move(y), std::move(data)) : wrap(std::move(y));
  });
}

// dy, kept's buffer, tokens and dim, weight, eps, dx, dweight, accumulate, workspace, stream
PyObject* rmsnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("rmsnorm_backward", n, 11, [&] {
    const at::Tensor &dy = tensor(a[0], "dy"), &weight = tensor(a[4], "weight");
    const at::Device dev = dy.device();
    const Matrix m = matrix(dy, "dy", dev);
    const rcc_dtype kind = dtype_of(dy, "dy");
    const Kept k =
        kept_in(kept_arg(a[1], a[2], a[3], m.rows, m.cols, dev), m.rows, m.cols);
    const float* w = floats(weight, "weight", dev, m.cols);
    const float eps = (float)number(a[5]);
    const int accumulate = truth(a[8]);
    if (accumulate && !given(a[7])) refuse("accumulate needs the dweight to add to");
    const Stream stream(a[10], dev);
    at::Tensor dx = output(a[6], "dx", {m.rows, m.cols}, dy.scalar_type(), dev);
    at::Tensor dweight = output(a[7], "dweight", {m.cols}, at::kFloat, dev);
    const Workspace ws = workspace(a[9], rcc_.rmsnorm_backward_workspace(m.rows, m.cols), dev);
    call(rcc_.rmsnorm_backward, dy.data_ptr(), kind, (size_t)m.ld, k.values, k.scales, w, eps,
         (size_t)m.rows, (size_t)m.cols, dx.data_ptr(), static_cast<float*>(dweight.data_ptr()),
         accumulate, ws.p, ws.bytes, stream.handle());
    return wrap(std::move(dx), std::move(dweight));
  });
}

// ---- RMS norm with the residual's addition, output in 8 bits ---------------------

PyObject* none_or(at::Tensor t) {
  return t.defined() ? wrap(std::move(t)) : Py_NewRef(Py_None);
}

// x, residual, weight, eps, 8-bit output, keep (None, True, or a buffer), its tokens, its dim, h,
// out, out's scales, stream: (out, its scales, h, keep's new buffer)
PyObject* add_rmsnorm_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("add_rmsnorm_forward", n, 12, [&] {
    const at::Tensor &x = tensor(a[0], "x"), &weight = tensor(a[2], "weight");
    const at::Device dev = x.device();
    const Matrix m = matrix(x, "x", dev);
    const rcc_dtype kind = dtype_of(x, "x");
    const bool eight = truth(a[4]);
    Matrix mr = {m.rows, m.cols, m.cols};
    const void* residual = nullptr;
    if (given(a[1])) {
      const at::Tensor& r = tensor(a[1], "residual");
      mr = matrix(r, "residual", dev);
      if (mr.rows != m.rows || mr.cols != m.cols || r.scalar_type() != x.scalar_type())
        refuse("residual must be of x's type and shape");
      residual = r.data_ptr();
    } else {
      if (!eight) refuse("without a residual the output has to be 8-bit");
      if (given(a[8])) refuse("h is the sum with a residual");
    }
    const float* w = floats(weight, "weight", dev, m.cols);
    const float eps = (float)number(a[3]);
    at::Tensor data, h, y, scales;
    if (given(a[5]) && a[5] != Py_True) data = kept_arg(a[5], a[6], a[7], m.rows, m.cols, dev);
    const auto type = eight ? at::kFloat8_e4m3fn : x.scalar_type();
    if (given(a[8])) h = output(a[8], "h", {m.rows, m.cols}, x.scalar_type(), dev);
    if (given(a[9])) y = output(a[9], "out", {m.rows, m.cols}, type, dev);
    if (given(a[10])) {
      if (!eight) refuse("out_scales come with an 8-bit output");
      scales = output(a[10], "out_scales", {m.rows, groups_of(m.cols)}, at::kFloat, dev);
    }
    const Stream stream(a[11], dev);
    if (given(a[1]) && !h.defined()) h = fresh({m.rows, m.cols}, x.scalar_type(), dev);
    if (!y.defined()) y = fresh({m.rows, m.cols}, type, dev);
    if (eight && !scales.defined()) scales = fresh({m.rows, groups_of(m.cols)}, at::kFloat, dev);
    if (a[5] == Py_True) data = fresh({kept_bytes(m.rows, m.cols)}, at::kByte, dev);
    const Kept k = data.defined() ? kept_in(data, m.rows, m.cols) : Kept{nullptr, nullptr};
    call(rcc_.add_rmsnorm_forward, x.data_ptr(), (size_t)m.ld, residual, (size_t)mr.ld, kind, w,
         eps, (size_t)m.rows, (size_t)m.cols, h.defined() ? h.data_ptr() : nullptr, y.data_ptr(),
         eight ? static_cast<float*>(scales.data_ptr()) : nullptr, k.values, k.scales,
         stream.handle());
    PyObject* r = PyTuple_New(4);
    if (!r) throw python_error();
    PyTuple_SET_ITEM(r, 0, wrap(std::move(y)));
    PyTuple_SET_ITEM(r, 1, none_or(std::move(scales)));
    PyTuple_SET_ITEM(r, 2, none_or(std::move(h)));
    PyTuple_SET_ITEM(r, 3, none_or(a[5] == Py_True ? std::move(data) : at::Tensor()));
    return r;
  });
}

// dy, dh, kept's buffer, tokens and dim, weight, eps, dx, dweight, accumulate, workspace, stream
PyObject* add_rmsnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("add_rmsnorm_backward", n, 12, [&] {
    const at::Tensor &dy = tensor(a[0], "dy"), &weight = tensor(a[5], "weight");
    const at::Device dev = dy.device();
    const Matrix m = matrix(dy, "dy", dev);
    const rcc_dtype kind = dtype_of(dy, "dy");
    Matrix mh = {m.rows, m.cols, m.cols};
    const void* dh = nullptr;
    if (given(a[1])) {
      const at::Tensor& t = tensor(a[1], "dh");
      mh = matrix(t, "dh", dev);
      if (mh.rows != m.rows || mh.cols != m.cols || t.scalar_type() != dy.scalar_type())
        refuse("dh must be of dy's type and shape");
      dh = t.data_ptr();
    }
    const Kept k = kept_in(kept_arg(a[2], a[3], a[4], m.rows, m.cols, dev), m.rows, m.cols);
    const float* w = floats(weight, "weight", dev, m.cols);
    const float eps = (float)number(a[6]);
    const int accumulate = truth(a[9]);
    if (accumulate && !given(a[8])) refuse("accumulate needs the dweight to add to");
    at::Tensor dx, dweight;
    if (given(a[7])) dx = output(a[7], "dx", {m.rows, m.cols}, dy.scalar_type(), dev);
    if (given(a[8])) dweight = output(a[8], "dweight", {m.cols}, at::kFloat, dev);
    const Stream stream(a[11], dev);
    if (!dx.defined()) dx = fresh({m.rows, m.cols}, dy.scalar_type(), dev);
    if (!dweight.defined()) dweight = fresh({m.cols}, at::kFloat, dev);
    const Workspace ws = workspace(a[10], rcc_.rmsnorm_backward_workspace(m.rows, m.cols), dev);
    call(rcc_.add_rmsnorm_backward, dy.data_ptr(), (size_t)m.ld, dh, (size_t)mh.ld, kind, k.values,
         k.scales, w, eps, (size_t)m.rows, (size_t)m.cols, dx.data_ptr(),
         static_cast<float*>(dweight.data_ptr()), accumulate, ws.p, ws.bytes, stream.handle());
    return wrap(std::move(dx), std::move(dweight));
  });
}

// ---- rotary positions -----------------------------------------------------------

// [tokens, heads, head_dim] with neighbouring elements of a head
struct Heads {
  int64_t tokens, heads, head_dim;
  size_t token, head;
};
Heads heads_of(const at::Tensor& t, const char* what, at::Device dev) {
  if (t.dim() != 3 || t.device() != dev)
    refuse("%s must be [tokens, heads, head_dim] on the inputs' device", what);
  const Heads h = {t.size(0), t.size(1), t.size(2),
                   (size_t)(t.size(0) < 2 ? t.size(1) * t.size(2) : t.stride(0)),
                   (size_t)(t.size(1) < 2 ? t.size(2) : t.stride(1))};
  if (h.head_dim > 1 && t.stride(2) != 1) refuse("the heads of %s must be contiguous", what);
  return h;
}

// inverse, q, k, turns, positions, offset, layout, scale, q_out, k_out, stream
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("rotary", n, 11, [&] {
    const bool inverse = truth(a[0]);
    const char* names[2] = {"q", "k"};
    const char* out_names[2] = {"q_out", "k_out"};
    const at::Tensor& q = tensor(a[1], "q");
    const at::Device dev = q.device();
    const rcc_dtype kind = dtype_of(q, "q");
    const int count = given(a[2]) ? 2 : 1;
    if (count == 1 && given(a[9])) refuse("k_out without k");
    Heads in[2];
    at::Tensor out[2];
    rcc_rotary_rows rows[2] = {};
    for (int i = 0; i < count; ++i) {
      const at::Tensor& t = tensor(a[1 + i], names[i]);
      in[i] = heads_of(t, names[i], dev);
      if (t.scalar_type() != q.scalar_type() || in[i].tokens != in[0].tokens ||
          in[i].head_dim != in[0].head_dim)
        refuse("q and k must have one type, tokens and head_dim");
      if (given(a[8 + i])) {
        out[i] = tensor(a[8 + i], out_names[i]);
        if (out[i].sizes() != t.sizes() || out[i].scalar_type() != t.scalar_type())
          refuse("%s must be of %s's type and shape", out_names[i], names[i]);
        heads_of(out[i], out_names[i], dev);
      }
      rows[i].in = t.data_ptr();
      rows[i].heads = in[i].heads;
      rows[i].in_token = in[i].token;
      rows[i].in_head = in[i].head;
    }
    const at::Tensor& turns = tensor(a[3], "turns");
    if (turns.scalar_type() != at::kLong || turns.dim() != 1 || turns.device() != dev ||
        !turns.is_contiguous() || 2 * turns.numel() > in[0].head_dim)
      refuse("turns must be a contiguous vector of int64, at most half of head_dim, on the inputs' "
             "device");
    rcc_index index = RCC_I32;
    const void* positions = nullptr;
    if (given(a[4])) {
      const at::Tensor& p = tensor(a[4], "positions");
      index = index_of(p, "positions", dev, in[0].tokens);
      positions = p.data_ptr();
    }
    const long long offset = PyLong_AsLongLong(a[5]);
    const long layout = PyErr_Occurred() ? 0 : PyLong_AsLong(a[6]);
    if (PyErr_Occurred()) throw python_error();
    const float scale = (float)number(a[7]);
    const Stream stream(a[10], dev);
    for (int i = 0; i < count; ++i) {
      if (!out[i].defined())
        out[i] = fresh({in[i].tokens, in[i].heads, in[i].head_dim}, q.scalar_type(), dev);
      const Heads h = heads_of(out[i], out_names[i], dev);
      rows[i].out = out[i].data_ptr();
      rows[i].out_token = h.token;
      rows[i].out_head = h.head;
    }
    call(inverse ? rcc_.rotary_backward : rcc_.rotary_forward,
         static_cast<const rcc_rotary_rows*>(&rows[0]),
         static_cast<const rcc_rotary_rows*>(count == 2 ? &rows[1] : nullptr), kind,
         (size_t)in[0].tokens, (size_t)in[0].head_dim,
         static_cast<const uint64_t*>(turns.data_ptr()), (size_t)turns.numel(),
         (rcc_rotary_layout)layout, positions, index, (int64_t)offset, scale, stream.handle());
    return wrap(std::move(out[0]), std::move(out[1]));
  });
}

// ---- AdamW over many tensors -----------------------------------------------------

// plan, cfg's address, scale, device, stream: the stream's handle
PyObject* adamw_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("adamw_step", n, 5, [&] {
    auto plan = static_cast<rcc_adamw>(PyLong_AsVoidPtr(a[0]));
    if (PyErr_Occurred()) throw python_error();
    auto cfg = static_cast<const rcc_adamw_cfg*>(PyLong_AsVoidPtr(a[1]));
    if (PyErr_Occurred()) throw python_error();
    const double scale = number(a[2]);
    const long device = PyLong_AsLong(a[3]);
    if (PyErr_Occurred()) throw python_error();
    const Stream stream(a[4], at::Device(at::kCUDA, (c10::DeviceIndex)device));
    call(rcc_.adamw_step, plan, cfg, scale, stream.handle());
    return PyLong_FromVoidPtr(stream.handle());
  });
}

// ---- output layer ---------------------------------------------------------------

struct Scores {
  const at::Tensor &x, &w, &labels;
  at::Device dev;
  Matrix mx, mw;
  rcc_index index;
};
Scores scores(PyObject* px, PyObject* pw, PyObject* pl) {
  const at::Tensor &x = tensor(px, "x"), &w = tensor(pw, "w"), &labels = tensor(pl, "labels");
  const at::Device dev = x.device();
  if (x.scalar_type() != at::kBFloat16 || w.scalar_type() != at::kBFloat16)
    refuse("x and w must be bfloat16");
  const Matrix mx = matrix(x, "x", dev), mw = matrix(w, "w", dev);
  if (mx.cols != mw.cols)
    refuse("x has %lld columns, w %lld", (long long)mx.cols, (long long)mw.cols);
  return {x, w, labels, dev, mx, mw, index_of(labels, "labels", dev, mx.rows)};
}

// x, w, labels, loss, lse, workspace, stream
PyObject* linear_ce_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("linear_ce_forward", n, 7, [&] {
    const Scores s = scores(a[0], a[1], a[2]);
    const Stream stream(a[6], s.dev);
    at::Tensor loss = output(a[3], "loss", {s.mx.rows}, at::kFloat, s.dev);
    at::Tensor lse = output(a[4], "lse", {s.mx.rows}, at::kFloat, s.dev);
    const Workspace ws = workspace(
        a[5], rcc_.linear_ce_workspace(s.mx.rows, s.mw.rows, s.mx.cols, 0, RCC_F32), s.dev);
    call(rcc_.linear_ce_forward, s.x.data_ptr(), (size_t)s.mx.ld, s.w.data_ptr(),
         (size_t)s.mw.ld, s.labels.data_ptr(), s.index, (size_t)s.mx.rows, (size_t)s.mw.rows,
         (size_t)s.mx.cols, static_cast<float*>(loss.data_ptr()),
         static_cast<float*>(lse.data_ptr()), ws.p, ws.bytes, stream.handle());
    return wrap(std::move(loss), std::move(lse));
  });
}

// x, w, labels, lse, dloss, grad_dtype, dx, dw, accumulate, workspace, need_dx, need_dw, stream
PyObject* linear_ce_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("linear_ce_backward", n, 13, [&] {
    const Scores s = scores(a[0], a[1], a[2]);
    const float* lse = floats(tensor(a[3], "lse"), "lse", s.dev, s.mx.rows);
    const float* dloss = floats(tensor(a[4], "dloss"), "dloss", s.dev, s.mx.rows);
    const int accumulate = truth(a[8]);
    if (accumulate && !given(a[7])) refuse("accumulate needs the dw to add to");
    rcc_dtype grad = RCC_BF16;
    if (given(a[5])) grad = dtype_arg(a[5], "grad_dtype");
    else if (given(a[6])) grad = dtype_of(tensor(a[6], "dx"), "dx");
    else if (given(a[7])) grad = dtype_of(tensor(a[7], "dw"), "dw");
    const bool need_dx = truth(a[10]), need_dw = truth(a[11]);
    at::Tensor dx, dw;
    // what the caller passed is checked before anything is allocated
    if (need_dx && given(a[6]))
      dx = output(a[6], "dx", {s.mx.rows, s.mx.cols}, scalar_of(grad), s.dev);
    if (need_dw && given(a[7]))
      dw = output(a[7], "dw", {s.mw.rows, s.mx.cols}, scalar_of(grad), s.dev);
    const Stream stream(a[12], s.dev);
    if (need_dx && !dx.defined()) dx = fresh({s.mx.rows, s.mx.cols}, scalar_of(grad), s.dev);
    if (need_dw && !dw.defined()) dw = fresh({s.mw.rows, s.mx.cols}, scalar_of(grad), s.dev);
    const Workspace ws = workspace(
        a[9], rcc_.linear_ce_workspace(s.mx.rows, s.mw.rows, s.mx.cols, 1, grad), s.dev);
    call(rcc_.linear_ce_backward, s.x.data_ptr(), (size_t)s.mx.ld, s.w.data_ptr(),
         (size_t)s.mw.ld, s.labels.data_ptr(), s.index, lse, dloss, (size_t)s.mx.rows,
         (size_t)s.mw.rows, (size_t)s.mx.cols, dx.defined() ? dx.data_ptr() : nullptr,
         dw.defined() ? dw.data_ptr() : nullptr, grad, accumulate, ws.p, ws.bytes, stream.handle());
    return wrap(std::move(dx), std::move(dw));
  });
}

// ---- the module -----------------------------------------------------------------

// on_error, then the addresses of Entries' members in their order
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr Py_ssize_t kEntries = sizeof(Entries) / sizeof(void*);
  if (n != 1 + kEntries) {
    PyErr_Format(PyExc_TypeError, "bind takes %zd arguments", 1 + kEntries);
    return nullptr;
  }
  void* p[kEntries];
  for (Py_ssize_t i = 0; i < kEntries; ++i) {
    p[i] = PyLong_AsVoidPtr(a[1 + i]);
    if (PyErr_Occurred()) return nullptr;
  }
  memcpy(&rcc_, p, sizeof(rcc_));
  Py_XDECREF(on_error);
  on_error = Py_NewRef(a[0]);
  Py_RETURN_NONE;
}

// device, current device: ValueError unless they are the same
PyObject* check_device(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("check_device", n, 2, [&] {
    const long device = PyLong_AsLong(a[0]);
    const long current = PyErr_Occurred() ? -1 : PyLong_AsLong(a[1]);
    if (PyErr_Occurred()) throw python_error();
    require_current((int)device, (int)current);
    return Py_NewRef(Py_None);
  });
}

#define RCC_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {
    {"bind", RCC_FAST(bind), "Takes the error callback and librcc's entry points."},
    {"check_device", RCC_FAST(check_device), nullptr},
    {"embedding_forward", RCC_FAST(embedding_forward), nullptr},
    {"embedding_backward", RCC_FAST(embedding_backward), nullptr},
    {"rmsnorm_forward", RCC_FAST(rmsnorm_forward), nullptr},
    {"rmsnorm_backward", RCC_FAST(rmsnorm_backward), nullptr},
    {"add_rmsnorm_forward", RCC_FAST(add_rmsnorm_forward), nullptr},
    {"add_rmsnorm_backward", RCC_FAST(add_rmsnorm_backward), nullptr},
    {"rotary", RCC_FAST(rotary), nullptr},
    {"adamw_step", RCC_FAST(adamw_step), nullptr},
    {"linear_ce_forward", RCC_FAST(linear_ce_forward), nullptr},
    {"linear_ce_backward", RCC_FAST(linear_ce_backward), nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lm",
                      "librcc's language-model operators for torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lm() { return PyModule_Create(&module); }
