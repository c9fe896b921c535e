// Torch binding of the norm and router calls of the C ABI: what ops.py does in
// Python for the other calls (argument checks, output allocation, marshalling),
// in C++, since these calls take microseconds on the device and their Python
// form took 20 to 27 us a call on the host.  No computation happens here: every
// function ends in one call of include/mpm.h on the current stream.
//
// Errors: TypeError and ValueError for what the library cannot see (element
// types, shapes, dense rows, devices), MpmError for a status of the library.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mpm.h"

namespace {

using at::ScalarType;
using at::Tensor;

// Thrown with a Python error already set.
struct PyError {};

[[noreturn]] void fail(PyObject* type, const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  throw PyError();
}

const char* type_name(ScalarType t) {
  switch (t) {
    case ScalarType::BFloat16: return "bfloat16";
    case ScalarType::Float: return "float32";
    case ScalarType::Int: return "int32";
    case ScalarType::Byte: return "uint8";
    default: return c10::toString(t);
  }
}

// ---------------------------------------------------------------- arguments
// A tensor argument; null for None where it may be missing
const Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s: expected a tensor, got %s", name, Py_TYPE(o)->tp_name);
  return &THPVariable_Unpack(o);
}
long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyError();
  return v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyError();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PyError();
  return v != 0;
}
int small_int(long long v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX) fail(PyExc_ValueError, "%s = %lld does not fit 32 bits", name, v);
  return (int)v;
}

std::string shape_of(const Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

void need_type(const Tensor& t, const char* name, ScalarType want) {
  if (t.scalar_type() != want)
    fail(PyExc_TypeError, "%s: expected %s, got %s", name, type_name(want), type_name(t.scalar_type()));
}
// a dense buffer of one type that holds at least n elements
void need_buffer(const Tensor& t, const char* name, ScalarType want, int64_t n) {
  need_type(t, name, want);
  if (!t.is_contiguous()) fail(PyExc_ValueError, "%s: expected a contiguous tensor", name);
  if (t.numel() < n)
    fail(PyExc_ValueError, "%s: holds %lld elements, the call needs %lld", name, (long long)t.numel(), (long long)n);
}
// Row pitch in elements of a [rows, cols] matrix with dense rows (torch leaves
// the strides of axes of length one open)
int64_t row_pitch(const Tensor& t, const char* name) {
  if (t.dim() != 2) fail(PyExc_ValueError, "%s: expected a 2-d tensor, got shape %s", name, shape_of(t).c_str());
  if (t.stride(1) != 1 && t.size(1) != 1)
    fail(PyExc_ValueError, "%s: rows must be dense (stride(1) == 1)", name);
  const int64_t ld = t.stride(0);
  return t.size(0) > 1 || ld >= t.size(1) ? ld : t.size(1);
}
int64_t matrix(const Tensor& t, const char* name, ScalarType want, int64_t rows, int64_t cols) {
  need_type(t, name, want);
  const int64_t ld = row_pitch(t, name);
  if (t.size(0) != rows || t.size(1) != cols)
    fail(PyExc_ValueError, "%s: expected shape (%lld, %lld), got %s", name, (long long)rows, (long long)cols,
         shape_of(t).c_str());
  return ld;
}
int weight_type(const Tensor& w, int64_t K) {
  if (w.scalar_type() != ScalarType::Float && w.scalar_type() != ScalarType::BFloat16)
    fail(PyExc_TypeError, "weight: expected bf16 or fp32, got %s", type_name(w.scalar_type()));
  if (w.dim() != 1 || w.size(0) != K || !w.is_contiguous())
    fail(PyExc_ValueError, "weight: expected a contiguous [%lld], got shape %s", (long long)K, shape_of(w).c_str());
  return w.scalar_type() == ScalarType::Float ? MPM_DTYPE_F32 : MPM_DTYPE_BF16;
}
// all given tensors on the first one's CUDA device, which is the current one while
// the result lives: the library launches on the current device
[[nodiscard]] c10::cuda::CUDAGuard need_cuda(std::initializer_list<const Tensor*> ts) {
  c10::DeviceIndex dev = -1;
  for (const Tensor* t : ts) {
    if (!t) continue;
    if (!t->is_cuda()) fail(PyExc_ValueError, "libmpm operates on CUDA tensors only");
    if (dev < 0) dev = t->device().index();
    if (t->device().index() != dev) fail(PyExc_ValueError, "the tensors are on different CUDA devices");
  }
  return c10::cuda::CUDAGuard(dev);
}

// A new tensor on the current device, with memory of its own: straight from the
// caching allocator, in 0.5 us where the generic factory takes 0.8 (outputs that
// share one allocation are 0.3 each, but a resize of one reaches the others)
Tensor make(at::IntArrayRef size, ScalarType type) {
  c10::Allocator* memory = c10::cuda::CUDACachingAllocator::get();
  int64_t bytes = (int64_t)c10::elementSize(type);
  for (const int64_t n : size) bytes *= n;
  auto storage = c10::make_intrusive<c10::StorageImpl>(c10::StorageImpl::use_byte_size_t(), (size_t)bytes,
                                                       memory->allocate((size_t)bytes), memory, /*resizable=*/true);
  Tensor t = at::detail::make_tensor<c10::TensorImpl>(std::move(storage), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                      c10::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_sizes_contiguous(size);
  return t;
}

void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
cudaStream_t stream_of(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

void check(mpm_status status, const char* what) {
  if (status == MPM_OK) return;
  PyObject* lib = PyImport_ImportModule("microscaled_precision_moe_gb300._lib");
  PyObject* r = lib ? PyObject_CallMethod(lib, "check", "is", (int)status, what) : nullptr;
  Py_XDECREF(r);
  Py_XDECREF(lib);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, what);
  throw PyError();
}

// ---------------------------------------------------------------- result dicts
struct Ref {
  PyObject* o;
  explicit Ref(PyObject* p = nullptr) : o(p) {}
  ~Ref() { Py_XDECREF(o); }
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
  PyObject* give() { PyObject* p = o; o = nullptr; return p; }
};

// the dict to return: `out`, or a new one
PyObject* result_dict(PyObject* out) {
  if (out == Py_None) {
    PyObject* d = PyDict_New();
    if (!d) throw PyError();
    return d;
  }
  if (!PyDict_Check(out)) fail(PyExc_TypeError, "out: expected a dict, got %s", Py_TYPE(out)->tp_name);
  Py_INCREF(out);
  return out;
}
// a tensor of the dict, or null
const Tensor* item(PyObject* d, PyObject* key, const char* name) {
  PyObject* v = PyDict_GetItemWithError(d, key);
  if (!v && PyErr_Occurred()) throw PyError();
  return v && v != Py_None ? tensor(v, name) : nullptr;
}
void put(PyObject* d, PyObject* key, const Tensor& t) {
  Ref v(THPVariable_Wrap(t));
  if (!v.o || PyDict_SetItem(d, key, v.o) < 0) throw PyError();
}

PyObject *kY, *kH, *kRstd, *kRowQ, *kRowS, *kIds, *kProb, *kCounts, *kLoad, *kTokens, *kLoss, *kLogp, *kLse,
    *kEntropy, *kTopIds, *kTopLogp;

void need_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) fail(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
}

// ---------------------------------------------------------------- calls
// (x, weight, residual, eps, want_y, quantize, out)
PyObject* add_rmsnorm(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 7);
  const Tensor &x = *tensor(a[0], "x"), &w = *tensor(a[1], "weight");
  const Tensor* res = tensor(a[2], "residual", true);
  need_type(x, "x", ScalarType::BFloat16);
  const int64_t ldx = row_pitch(x, "x"), M = x.size(0), K = x.size(1);
  const int wt = weight_type(w, K);
  const double eps = real(a[3]);
  const bool want_y = truth(a[4]), quantize = truth(a[5]);
  const int64_t ldr = res ? matrix(*res, "residual", ScalarType::BFloat16, M, K) : 0;
  if (quantize && K % 32 != 0)
    fail(PyExc_ValueError, "x: K = %lld is not a multiple of the 32-value MXFP8 block", (long long)K);
  Ref d(result_dict(a[6]));
  const Tensor *y = nullptr, *h = nullptr, *q = nullptr, *s = nullptr;
  int64_t ldy = K, ldh = K;
  const int64_t sb = quantize ? (int64_t)mpm_scale_bytes(M, K / 32) : 0;
  const Tensor* rstd = item(d.o, kRstd, "rstd");
  if (rstd) need_buffer(*rstd, "rstd", ScalarType::Float, M);
  if (want_y && (y = item(d.o, kY, "y"))) ldy = matrix(*y, "y", ScalarType::BFloat16, M, K);
  if (res && (h = item(d.o, kH, "h"))) ldh = matrix(*h, "h", ScalarType::BFloat16, M, K);
  if (quantize && (q = item(d.o, kRowQ, "row_q"))) need_buffer(*q, "row_q", ScalarType::Byte, M * K);
  if (quantize && (s = item(d.o, kRowS, "row_s"))) need_buffer(*s, "row_s", ScalarType::Byte, sb);
  const auto device = need_cuda({&x, &w, res, y, h, rstd, q, s});
  Tensor ny, nh, nr, nq, ns;
  if (want_y && !y) { ny = make({M, K}, ScalarType::BFloat16); y = &ny; }
  if (res && !h) { nh = make({M, K}, ScalarType::BFloat16); h = &nh; }
  if (!rstd) { nr = make({M}, ScalarType::Float); rstd = &nr; }
  if (quantize && !q) { nq = make({M, K}, ScalarType::Byte); q = &nq; }
  if (quantize && !s) { ns = make({sb}, ScalarType::Byte); s = &ns; }
  if (y == &ny) put(d.o, kY, ny);
  if (h == &nh) put(d.o, kH, nh);
  if (rstd == &nr) put(d.o, kRstd, nr);
  if (q == &nq) put(d.o, kRowQ, nq);
  if (s == &ns) put(d.o, kRowS, ns);
  check(mpm_add_rmsnorm(x.data_ptr(), M, K, ldx, ptr(res), ldr, w.data_ptr(), wt, (float)eps, ptr(h), ldh, ptr(y),
                        ldy, static_cast<float*>(ptr(rstd)), static_cast<uint8_t*>(ptr(q)),
                        static_cast<uint8_t*>(ptr(s)), stream_of(x)),
        "mpm_add_rmsnorm");
  return d.give();
}

// (dy, h, rstd, weight, dy2, dh, want_dw, out, ws)
PyObject* add_rmsnorm_backward(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 9);
  const Tensor &dy = *tensor(a[0], "dy"), &h = *tensor(a[1], "h"), &rstd = *tensor(a[2], "rstd"),
               &w = *tensor(a[3], "weight");
  const Tensor *dy2 = tensor(a[4], "dy2", true), *dh = tensor(a[5], "dh", true), *ws = tensor(a[8], "ws", true);
  const bool want_dw = truth(a[6]);
  const ScalarType bf = ScalarType::BFloat16;
  need_type(dy, "dy", bf);
  const int64_t lddy = row_pitch(dy, "dy"), M = dy.size(0), K = dy.size(1);
  const int64_t ldh = matrix(h, "h", bf, M, K);
  const int wt = weight_type(w, K);
  need_buffer(rstd, "rstd", ScalarType::Float, M);
  const int64_t lddy2 = dy2 ? matrix(*dy2, "dy2", bf, M, K) : 0, lddh = dh ? matrix(*dh, "dh", bf, M, K) : 0;
  const Tensor *dx = nullptr, *dw = nullptr;
  int64_t lddx = K;
  if (a[7] != Py_None) {
    if (!PyTuple_Check(a[7]) || PyTuple_GET_SIZE(a[7]) != 2) fail(PyExc_TypeError, "out: expected a pair (dx, dw)");
    dx = tensor(PyTuple_GET_ITEM(a[7], 0), "dx");
    lddx = matrix(*dx, "dx", bf, M, K);
    if (want_dw) {
      dw = tensor(PyTuple_GET_ITEM(a[7], 1), "dw");
      need_buffer(*dw, "dw", ScalarType::Float, K);
    }
  }
  const size_t wsb = want_dw ? mpm_add_rmsnorm_backward_workspace_bytes(M, K) : 0;
  if (!want_dw) ws = nullptr;
  if (ws) need_buffer(*ws, "ws", ScalarType::Byte, (int64_t)wsb);
  const auto device = need_cuda({&dy, &h, &rstd, &w, dy2, dh, dx, dw, ws});
  Tensor nx, nw, nws;
  if (!dx) { nx = make({M, K}, bf); dx = &nx; }
  if (want_dw && !dw) { nw = make({K}, ScalarType::Float); dw = &nw; }
  if (want_dw && !ws) { nws = make({(int64_t)wsb}, ScalarType::Byte); ws = &nws; }
  check(mpm_add_rmsnorm_backward(dy.data_ptr(), lddy, ptr(dy2), lddy2, h.data_ptr(), ldh,
                                 static_cast<float*>(rstd.data_ptr()), w.data_ptr(), wt, ptr(dh), lddh, M, K,
                                 dx->data_ptr(), lddx, static_cast<float*>(ptr(dw)), ptr(ws), wsb, stream_of(dy)),
        "mpm_add_rmsnorm_backward");
  Ref r(PyTuple_New(2));
  if (!r.o) throw PyError();
  PyObject* px = a[7] != Py_None ? PyTuple_GET_ITEM(a[7], 0) : nullptr;
  if (px) Py_INCREF(px);
  else px = THPVariable_Wrap(*dx);
  PyTuple_SET_ITEM(r.o, 0, px);
  PyObject* pw = nullptr;
  if (!dw) { pw = Py_None; Py_INCREF(pw); }
  else if (a[7] != Py_None) { pw = PyTuple_GET_ITEM(a[7], 1); Py_INCREF(pw); }
  else pw = THPVariable_Wrap(*dw);
  PyTuple_SET_ITEM(r.o, 1, pw);
  if (!px || !pw) throw PyError();
  return r.give();
}

// what the router's two calls share
struct Router {
  const Tensor *logits, *bias, *mask;
  int64_t T, E, ld;
  int type, score;
  Router(PyObject* l, PyObject* sc, PyObject* b, PyObject* m)
      : logits(tensor(l, "logits")), bias(tensor(b, "bias", true)), mask(tensor(m, "token_mask", true)) {
    const ScalarType t = logits->scalar_type();
    if (t != ScalarType::Float && t != ScalarType::BFloat16)
      fail(PyExc_TypeError, "logits: expected bf16 or fp32, got %s", type_name(t));
    type = t == ScalarType::Float ? MPM_DTYPE_F32 : MPM_DTYPE_BF16;
    ld = row_pitch(*logits, "logits");
    T = logits->size(0);
    E = logits->size(1);
    if (PyUnicode_Check(sc) && PyUnicode_CompareWithASCIIString(sc, "softmax") == 0) score = MPM_SCORE_SOFTMAX;
    else if (PyUnicode_Check(sc) && PyUnicode_CompareWithASCIIString(sc, "sigmoid") == 0) score = MPM_SCORE_SIGMOID;
    else fail(PyExc_ValueError, "score must be 'softmax' or 'sigmoid', got %R", sc);
    if (bias) {
      need_buffer(*bias, "bias", ScalarType::Float, E);
      if (bias->dim() != 1 || bias->size(0) != E)
        fail(PyExc_ValueError, "bias: expected [%lld], got shape %s", (long long)E, shape_of(*bias).c_str());
      if (score != MPM_SCORE_SIGMOID) fail(PyExc_ValueError, "bias: the choice bias belongs to sigmoid scores");
    }
    if (mask) {
      if (mask->scalar_type() != ScalarType::Bool && mask->scalar_type() != ScalarType::Byte)
        fail(PyExc_TypeError, "token_mask: expected bool or uint8, got %s", type_name(mask->scalar_type()));
      if (mask->dim() != 1 || mask->size(0) != T || !mask->is_contiguous())
        fail(PyExc_ValueError, "token_mask: expected a contiguous [%lld], got %s", (long long)T,
             shape_of(*mask).c_str());
    }
  }
};

// (logits, k, score, normalize, scale, bias, token_mask, out, ws)
PyObject* moe_route(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 9);
  const Router r(a[0], a[2], a[5], a[6]);
  const int k = small_int(integer(a[1]), "k");
  const bool normalize = truth(a[3]);
  const double scale = real(a[4]);
  if (k < 1) fail(PyExc_ValueError, "k = %d: at least one expert a token", k);
  struct { PyObject* key; const char* name; ScalarType type; int64_t rows, cols; } o[6] = {
      {kIds, "ids", ScalarType::Int, r.T, k},    {kProb, "prob", ScalarType::Float, r.T, k},
      {kCounts, "counts", ScalarType::Int, r.E, 0}, {kLoad, "load", ScalarType::Float, r.E, 0},
      {kTokens, "n_tokens", ScalarType::Int, 1, 0}, {kLoss, "loss", ScalarType::Float, 1, 0}};
  const bool fresh = a[7] == Py_None;
  Ref d(result_dict(a[7]));
  const Tensor* t[6] = {};
  Tensor made[6];
  for (int i = 0; i < 6 && !fresh; ++i) {
    t[i] = item(d.o, o[i].key, o[i].name);
    if (!t[i]) fail(PyExc_ValueError, "out: %s is missing", o[i].name);
    need_buffer(*t[i], o[i].name, o[i].type, o[i].rows * (o[i].cols ? o[i].cols : 1));
  }
  const Tensor* ws = tensor(a[8], "ws", true);
  const size_t wsb = mpm_moe_route_workspace_bytes(r.T, r.E);
  if (ws) need_buffer(*ws, "ws", ScalarType::Byte, (int64_t)wsb);
  const auto device = need_cuda({r.logits, r.bias, r.mask, ws, t[0], t[1], t[2], t[3], t[4], t[5]});
  for (int i = 0; i < 6 && fresh; ++i) {
    const int64_t size[2] = {o[i].rows, o[i].cols};
    made[i] = make(at::IntArrayRef(size, o[i].cols ? 2 : 1), o[i].type);
    t[i] = &made[i];
    put(d.o, o[i].key, made[i]);
  }
  Tensor nws;
  if (!ws && wsb) { nws = make({(int64_t)wsb}, ScalarType::Byte); ws = &nws; }
  check(mpm_moe_route(r.logits->data_ptr(), r.type, r.T, r.E, r.ld, k, r.score, normalize, (float)scale,
                      static_cast<float*>(ptr(r.bias)), static_cast<uint8_t*>(ptr(r.mask)),
                      static_cast<int32_t*>(ptr(t[0])), static_cast<float*>(ptr(t[1])),
                      static_cast<int32_t*>(ptr(t[2])), static_cast<float*>(ptr(t[3])),
                      static_cast<int32_t*>(ptr(t[4])), static_cast<float*>(ptr(t[5])), ptr(ws), wsb,
                      stream_of(*r.logits)),
        "mpm_moe_route");
  return d.give();
}

// (logits, ids, counts, n_tokens, dprob, dloss, score, normalize, scale, bias, token_mask, out)
PyObject* moe_route_backward(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 12);
  const Router r(a[0], a[6], a[9], a[10]);
  const Tensor &ids = *tensor(a[1], "ids"), &counts = *tensor(a[2], "counts"), &nt = *tensor(a[3], "n_tokens");
  const Tensor *dprob = tensor(a[4], "dprob", true), *dloss = tensor(a[5], "dloss", true);
  const bool normalize = truth(a[7]);
  const double scale = real(a[8]);
  if (ids.dim() != 2 || ids.size(0) != r.T)
    fail(PyExc_ValueError, "ids: expected [%lld, k], got shape %s", (long long)r.T, shape_of(ids).c_str());
  need_buffer(ids, "ids", ScalarType::Int, 0);
  const int k = small_int(ids.size(1), "k");
  need_buffer(counts, "counts", ScalarType::Int, r.E);
  need_buffer(nt, "n_tokens", ScalarType::Int, 1);
  if (dprob) {
    need_buffer(*dprob, "dprob", ScalarType::Float, 0);
    if (dprob->sizes() != ids.sizes())
      fail(PyExc_ValueError, "dprob: expected %s, got shape %s", shape_of(ids).c_str(), shape_of(*dprob).c_str());
  }
  if (dloss) need_buffer(*dloss, "dloss", ScalarType::Float, 1);
  const Tensor* out = tensor(a[11], "out", true);
  int64_t ldd = r.E;
  int out_type = r.type;
  if (out) {
    const ScalarType t = out->scalar_type();
    if (t != ScalarType::Float && t != ScalarType::BFloat16)
      fail(PyExc_TypeError, "out: expected bf16 or fp32, got %s", type_name(t));
    out_type = t == ScalarType::Float ? MPM_DTYPE_F32 : MPM_DTYPE_BF16;
    ldd = matrix(*out, "out", t, r.T, r.E);
  }
  const auto device = need_cuda({r.logits, &ids, &counts, &nt, dprob, dloss, r.bias, r.mask, out});
  Tensor made;
  if (!out) { made = make({r.T, r.E}, r.logits->scalar_type()); out = &made; }
  check(mpm_moe_route_backward(r.logits->data_ptr(), r.type, r.T, r.E, r.ld, k, r.score, normalize,
                               (float)scale, static_cast<float*>(ptr(r.bias)), static_cast<uint8_t*>(ptr(r.mask)),
                               static_cast<int32_t*>(ids.data_ptr()), static_cast<int32_t*>(counts.data_ptr()),
                               static_cast<int32_t*>(nt.data_ptr()), static_cast<float*>(ptr(dprob)),
                               static_cast<float*>(ptr(dloss)), out->data_ptr(), out_type, ldd,
                               stream_of(*r.logits)),
        "mpm_moe_route_backward");
  if (a[11] != Py_None) { Py_INCREF(a[11]); return a[11]; }
  PyObject* p = THPVariable_Wrap(made);
  if (!p) throw PyError();
  return p;
}

// (dout, y_perm, inv_perm, prob, out)
PyObject* moe_combine_dprob(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 5);
  const Tensor &dout = *tensor(a[0], "dout"), &y = *tensor(a[1], "y_perm"), &inv = *tensor(a[2], "inv_perm"),
               &prob = *tensor(a[3], "prob");
  const Tensor* out = tensor(a[4], "out", true);
  need_buffer(dout, "dout", ScalarType::BFloat16, 0);
  need_buffer(y, "y_perm", ScalarType::BFloat16, 0);
  need_buffer(prob, "prob", ScalarType::Float, 0);
  if (dout.dim() != 2 || y.dim() != 2 || prob.dim() != 2 || dout.size(0) != prob.size(0) || y.size(1) != dout.size(1))
    fail(PyExc_ValueError, "dout %s and y_perm %s do not match prob %s", shape_of(dout).c_str(), shape_of(y).c_str(),
         shape_of(prob).c_str());
  const int64_t T = prob.size(0);
  const int k = small_int(prob.size(1), "k");
  need_buffer(inv, "inv_perm", ScalarType::Int, T * k);
  if (out) need_buffer(*out, "out", ScalarType::Float, T * k);
  const auto device = need_cuda({&dout, &y, &inv, &prob, out});
  Tensor made;
  if (!out) { made = make({T, k}, ScalarType::Float); out = &made; }
  check(mpm_moe_combine_dprob(dout.data_ptr(), y.data_ptr(), static_cast<int32_t*>(inv.data_ptr()),
                              static_cast<float*>(prob.data_ptr()), T, k, dout.size(1), y.size(0),
                              static_cast<float*>(out->data_ptr()), stream_of(dout)),
        "mpm_moe_combine_dprob");
  if (a[4] != Py_None) { Py_INCREF(a[4]); return a[4]; }
  PyObject* p = THPVariable_Wrap(made);
  if (!p) throw PyError();
  return p;
}

// (q, s, perm, seg, E, k, cap, out)
PyObject* moe_gather_mxfp8(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 8);
  const ScalarType u8 = ScalarType::Byte;
  const Tensor &q = *tensor(a[0], "q"), &s = *tensor(a[1], "s"), &perm = *tensor(a[2], "perm"),
               &seg = *tensor(a[3], "seg_offsets");
  const int64_t E = integer(a[4]), cap = integer(a[6]);
  const int k = small_int(integer(a[5]), "k");
  if (E < 1 || cap < 1) fail(PyExc_ValueError, "E = %lld and cap = %lld: both at least 1", (long long)E, (long long)cap);
  need_buffer(q, "q", u8, 0);
  if (q.dim() != 2) fail(PyExc_ValueError, "q: expected a 2-d tensor, got shape %s", shape_of(q).c_str());
  const int64_t T = q.size(0), K = q.size(1);
  if (K % 32 != 0)
    fail(PyExc_ValueError, "q: K = %lld is not a multiple of the 32-value MXFP8 block", (long long)K);
  need_buffer(s, "s", u8, (int64_t)mpm_scale_bytes(T, K / 32));
  need_buffer(perm, "perm", ScalarType::Int, cap);
  need_buffer(seg, "seg_offsets", ScalarType::Int, 0);
  if (E >= seg.numel())
    fail(PyExc_ValueError, "seg_offsets: holds %lld elements, E = %lld experts need one more than that",
         (long long)seg.numel(), (long long)E);
  const int64_t sb = (int64_t)mpm_scale_bytes(cap, K / 32);
  const Tensor *dq = nullptr, *ds = nullptr;
  if (a[7] != Py_None) {
    if (!PyTuple_Check(a[7]) || PyTuple_GET_SIZE(a[7]) != 2)
      fail(PyExc_TypeError, "out: expected a pair (codes, scales)");
    dq = tensor(PyTuple_GET_ITEM(a[7], 0), "out codes");
    ds = tensor(PyTuple_GET_ITEM(a[7], 1), "out scales");
    need_buffer(*dq, "out codes", u8, cap * K);
    need_buffer(*ds, "out scales", u8, sb);
  }
  const auto device = need_cuda({&q, &s, &perm, &seg, dq, ds});
  Tensor nq, ns;
  if (!dq) {
    nq = make({cap, K}, u8);
    ns = make({sb}, u8);
    dq = &nq;
    ds = &ns;
  }
  check(mpm_moe_gather_mxfp8(static_cast<uint8_t*>(q.data_ptr()), static_cast<uint8_t*>(s.data_ptr()), T, K, k,
                             static_cast<int32_t*>(perm.data_ptr()), static_cast<int32_t*>(seg.data_ptr()), E, cap,
                             static_cast<uint8_t*>(dq->data_ptr()), static_cast<uint8_t*>(ds->data_ptr()),
                             stream_of(q)),
        "mpm_moe_gather_mxfp8");
  if (a[7] != Py_None) { Py_INCREF(a[7]); return a[7]; }
  PyObject *pq = THPVariable_Wrap(nq), *ps = pq ? THPVariable_Wrap(ns) : nullptr;
  PyObject* r = ps ? PyTuple_Pack(2, pq, ps) : nullptr;
  Py_XDECREF(pq);
  Py_XDECREF(ps);
  if (!r) throw PyError();
  return r;
}

int float_type(const Tensor& t, const char* name) {
  if (t.scalar_type() != ScalarType::Float && t.scalar_type() != ScalarType::BFloat16)
    fail(PyExc_TypeError, "%s: expected bf16 or fp32, got %s", name, type_name(t.scalar_type()));
  return t.scalar_type() == ScalarType::Float ? MPM_DTYPE_F32 : MPM_DTYPE_BF16;
}
// one number a row
void need_rows(const Tensor* t, const char* name, ScalarType type, int64_t rows) {
  if (!t) return;
  need_buffer(*t, name, type, rows);
  if (t->dim() != 1 || t->size(0) != rows)
    fail(PyExc_ValueError, "%s: expected [%lld], got shape %s", name, (long long)rows, shape_of(*t).c_str());
}
int index_type(const Tensor* t, int64_t rows) {
  if (!t) return MPM_INDEX_I32;
  if (t->scalar_type() != ScalarType::Int && t->scalar_type() != ScalarType::Long)
    fail(PyExc_TypeError, "targets: expected int32 or int64, got %s", type_name(t->scalar_type()));
  need_rows(t, "targets", t->scalar_type(), rows);
  return t->scalar_type() == ScalarType::Long ? MPM_INDEX_I64 : MPM_INDEX_I32;
}

// (logits, targets, temperature, entropy, top, out)
PyObject* token_logprob(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 6);
  const Tensor& l = *tensor(a[0], "logits");
  const Tensor* targets = tensor(a[1], "targets", true);
  const int type = float_type(l, "logits");
  const int64_t ld = row_pitch(l, "logits"), T = l.size(0), V = l.size(1);
  const int it = index_type(targets, T);
  const double temperature = real(a[2]);
  const bool entropy = truth(a[3]);
  const int top = small_int(integer(a[4]), "top");
  if (top < 0 || top > 32 || top > V)
    fail(PyExc_ValueError, "top = %d: at most 32 and at most the %lld tokens", top, (long long)V);
  struct { PyObject* key; const char* name; ScalarType type; int64_t cols; bool wanted; } o[5] = {
      {kLogp, "logp", ScalarType::Float, 0, targets != nullptr}, {kLse, "lse", ScalarType::Float, 0, true},
      {kEntropy, "entropy", ScalarType::Float, 0, entropy},      {kTopIds, "top_ids", ScalarType::Int, top, top > 0},
      {kTopLogp, "top_logp", ScalarType::Float, top, top > 0}};
  Ref d(result_dict(a[5]));
  const Tensor* t[5] = {};
  Tensor made[5];
  for (int i = 0; i < 5; ++i) {
    if (!o[i].wanted || !(t[i] = item(d.o, o[i].key, o[i].name))) continue;
    need_buffer(*t[i], o[i].name, o[i].type, T * (o[i].cols ? o[i].cols : 1));
  }
  const auto device = need_cuda({&l, targets, t[0], t[1], t[2], t[3], t[4]});
  for (int i = 0; i < 5; ++i) {
    if (!o[i].wanted || t[i]) continue;
    const int64_t size[2] = {T, o[i].cols};
    made[i] = make(at::IntArrayRef(size, o[i].cols ? 2 : 1), o[i].type);
    t[i] = &made[i];
    put(d.o, o[i].key, made[i]);
  }
  check(mpm_token_logprob(l.data_ptr(), type, T, V, ld, ptr(targets), it, (float)temperature, top,
                          static_cast<float*>(ptr(t[0])), static_cast<float*>(ptr(t[1])),
                          static_cast<float*>(ptr(t[2])), static_cast<int32_t*>(ptr(t[3])),
                          static_cast<float*>(ptr(t[4])), stream_of(l)),
        "mpm_token_logprob");
  return d.give();
}

// (logits, targets, lse, dlogp, entropy, dentropy, temperature, out, logp)
PyObject* token_logprob_backward(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 9);
  const Tensor &l = *tensor(a[0], "logits"), &lse = *tensor(a[2], "lse");
  const Tensor *targets = tensor(a[1], "targets", true), *dlogp = tensor(a[3], "dlogp", true),
               *h = tensor(a[4], "entropy", true), *dh = tensor(a[5], "dentropy", true), *out = tensor(a[7], "out", true),
               *logp = tensor(a[8], "logp", true);
  const int type = float_type(l, "logits");
  const int64_t ld = row_pitch(l, "logits"), T = l.size(0), V = l.size(1);
  const int it = index_type(targets, T);
  const ScalarType f32 = ScalarType::Float;
  need_rows(&lse, "lse", f32, T);
  need_rows(logp, "logp", f32, T);
  need_rows(dlogp, "dlogp", f32, T);
  need_rows(h, "entropy", f32, T);
  need_rows(dh, "dentropy", f32, T);
  if (logp && !targets) fail(PyExc_ValueError, "logp: log probabilities of targets need targets");
  if (dlogp && !targets) fail(PyExc_ValueError, "dlogp: a gradient of logp needs targets");
  if (dh && !h) fail(PyExc_ValueError, "dentropy: a gradient of the entropy needs the forward's entropy");
  const double temperature = real(a[6]);
  int64_t ldd = V;
  int out_type = type;
  if (out) {
    out_type = float_type(*out, "out");
    ldd = matrix(*out, "out", out->scalar_type(), T, V);
  }
  const auto device = need_cuda({&l, targets, logp, &lse, dlogp, h, dh, out});
  Tensor made;
  if (!out) { made = make({T, V}, l.scalar_type()); out = &made; }
  check(mpm_token_logprob_backward_from(l.data_ptr(), type, T, V, ld, ptr(targets), it, static_cast<float*>(ptr(logp)),
                                        static_cast<float*>(lse.data_ptr()), static_cast<float*>(ptr(dlogp)),
                                        static_cast<float*>(ptr(h)), static_cast<float*>(ptr(dh)), (float)temperature,
                                        out->data_ptr(), out_type, ldd, stream_of(l)),
        "mpm_token_logprob_backward");
  if (a[7] != Py_None) { Py_INCREF(a[7]); return a[7]; }
  PyObject* p = THPVariable_Wrap(made);
  if (!p) throw PyError();
  return p;
}

// the tensors of a weight: codes, tiled scales and, for NVFP4, outer scales
struct Weight {
  const Tensor *q, *s, *ts = nullptr;
  Weight(PyObject* o, const char* name, bool nv, int64_t E, int64_t rows, int64_t K) {
    const Py_ssize_t want = nv ? 3 : 2;
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != want)
      fail(PyExc_TypeError, nv ? "%s: expected a tuple (codes, scales, outer scales)" : "%s: expected a tuple (codes, scales)", name);
    q = tensor(PyTuple_GET_ITEM(o, 0), name);
    s = tensor(PyTuple_GET_ITEM(o, 1), name);
    need_buffer(*q, name, ScalarType::Byte, E * rows * (nv ? K / 2 : K));
    if (q->size(-1) != (nv ? K / 2 : K))
      fail(PyExc_ValueError, "%s: expected rows of %lld code bytes, got shape %s", name, (long long)(nv ? K / 2 : K), shape_of(*q).c_str());
    need_buffer(*s, name, ScalarType::Byte, (int64_t)mpm_scale_bytes(E * rows, K / (nv ? 16 : 32)));
    if (nv) {
      ts = tensor(PyTuple_GET_ITEM(o, 2), name);
      need_buffer(*ts, name, ScalarType::Float, E);
    }
  }
};

// (kind, x, topk_ids, topk_prob, w1, w2, E, I, out, ws)
PyObject* moe_few_tokens(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 10);
  mpm_moe_few_tokens_desc d{};
  d.kind = small_int(integer(a[0]), "kind");
  if (d.kind != MPM_KIND_NVFP4 && d.kind != MPM_KIND_MXFP8)
    fail(PyExc_ValueError, "kind = %d: KIND_NVFP4 or KIND_MXFP8", d.kind);
  const bool nv = d.kind == MPM_KIND_NVFP4;
  const Tensor &x = *tensor(a[1], "x"), &ids = *tensor(a[2], "topk_ids"), &prob = *tensor(a[3], "topk_prob");
  need_type(x, "x", ScalarType::BFloat16);
  d.ldx = row_pitch(x, "x");
  d.T = x.size(0);
  d.H = x.size(1);
  d.E = integer(a[6]);
  d.I = integer(a[7]);
  need_buffer(ids, "topk_ids", ScalarType::Int, 0);
  need_buffer(prob, "topk_prob", ScalarType::Float, 0);
  if (ids.dim() != 2 || ids.size(0) != d.T)
    fail(PyExc_ValueError, "topk_ids: expected [%lld, k], got shape %s", (long long)d.T, shape_of(ids).c_str());
  if (prob.sizes() != ids.sizes())
    fail(PyExc_ValueError, "topk_prob: expected %s, got shape %s", shape_of(ids).c_str(), shape_of(prob).c_str());
  d.k = small_int(ids.size(1), "k");
  const size_t wsb = mpm_moe_few_tokens_workspace_bytes(d.kind, d.T, d.k, d.E, d.H, d.I);
  if (!wsb)
    fail(PyExc_ValueError,
         "T = %lld, k = %d, E = %lld, H = %lld, I = %lld: at most 64 tokens, 1024 slots and 1024 experts, H a multiple "
         "of 256 and I of %d, both at most 16384",
         (long long)d.T, d.k, (long long)d.E, (long long)d.H, (long long)d.I, nv ? 256 : 128);
  const Weight w1(a[4], "w1", nv, d.E, 2 * d.I, d.H), w2(a[5], "w2", nv, d.E, d.H, d.I);
  const Tensor *out = tensor(a[8], "out", true), *ws = tensor(a[9], "ws", true);
  d.ldo = out ? matrix(*out, "out", ScalarType::BFloat16, d.T, d.H) : d.H;
  if (ws) need_buffer(*ws, "ws", ScalarType::Byte, (int64_t)wsb);
  const auto device = need_cuda({&x, &ids, &prob, w1.q, w1.s, w1.ts, w2.q, w2.s, w2.ts, out, ws});
  Tensor made, nws;
  if (!out) { made = make({d.T, d.H}, ScalarType::BFloat16); out = &made; }
  if (!ws) { nws = make({(int64_t)wsb}, ScalarType::Byte); ws = &nws; }
  d.x_dev = x.data_ptr();
  d.ids_dev = static_cast<int32_t*>(ids.data_ptr());
  d.prob_dev = static_cast<float*>(prob.data_ptr());
  d.w1_q_dev = static_cast<uint8_t*>(w1.q->data_ptr());
  d.w1_s_dev = static_cast<uint8_t*>(w1.s->data_ptr());
  d.w1_ts_dev = static_cast<float*>(ptr(w1.ts));
  d.w2_q_dev = static_cast<uint8_t*>(w2.q->data_ptr());
  d.w2_s_dev = static_cast<uint8_t*>(w2.s->data_ptr());
  d.w2_ts_dev = static_cast<float*>(ptr(w2.ts));
  d.out_dev = out->data_ptr();
  d.ws_dev = ws->data_ptr();
  d.ws_bytes = wsb;
  check(mpm_moe_few_tokens(&d, stream_of(x)), "mpm_moe_few_tokens");
  if (a[8] != Py_None) { Py_INCREF(a[8]); return a[8]; }
  PyObject* p = THPVariable_Wrap(made);
  if (!p) throw PyError();
  return p;
}

// no C++ exception leaves a call: errors of torch (an allocation that fails)
// become Python's, an error already set passes on
template <PyObject* (*f)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return f(args, n);
  } catch (const PyError&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*f)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&guarded<f>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<add_rmsnorm>("add_rmsnorm"),
                         method<add_rmsnorm_backward>("add_rmsnorm_backward"),
                         method<moe_route>("moe_route"),
                         method<moe_route_backward>("moe_route_backward"),
                         method<moe_combine_dprob>("moe_combine_dprob"),
                         method<moe_gather_mxfp8>("moe_gather_mxfp8"),
                         method<moe_few_tokens>("moe_few_tokens"),
                         method<token_logprob>("token_logprob"),
                         method<token_logprob_backward>("token_logprob_backward"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  struct { PyObject** key; const char* name; } keys[] = {
      {&kY, "y"},     {&kH, "h"},         {&kRstd, "rstd"}, {&kRowQ, "row_q"},     {&kRowS, "row_s"}, {&kIds, "ids"},
      {&kProb, "prob"}, {&kCounts, "counts"}, {&kLoad, "load"}, {&kTokens, "n_tokens"}, {&kLoss, "loss"},
      {&kLogp, "logp"}, {&kLse, "lse"}, {&kEntropy, "entropy"}, {&kTopIds, "top_ids"}, {&kTopLogp, "top_logp"}};
  for (auto& k : keys)
    if (!(*k.key = PyUnicode_InternFromString(k.name))) return nullptr;
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", MPM_BINDING_FOR) < 0) Py_CLEAR(m);
  return m;
}
