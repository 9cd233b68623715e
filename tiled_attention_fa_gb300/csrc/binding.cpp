// Python binding of the calls that run once per token and layer, or several
// times per training step: argument checks, output allocation and the call of
// the C ABI in one C++ function each.  The same through ctypes costs about
// 25 us of host time per call (three allocations and a dozen checks as separate
// Python calls), more than the kernels of a short context take.
//
// Every function takes its arguments by position and returns the outputs, or
// the fa_status as an int when that is not FA_OK; Python raises from it.
#include <Python.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <cstdarg>
#include <string>

#include "../../include/fa.h"

namespace {

using at::Tensor;

constexpr auto kF32 = at::kFloat;
constexpr auto kI32 = at::kInt;

// Raise a Python error of the type.
[[noreturn]] void fail(PyObject* type, const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  throw python_error();
}

std::string text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda())
    fail(PyExc_TypeError, "%s must be a CUDA tensor", name);
  return THPVariable_Unpack(o);
}

void want(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType dt, int dev) {
  if (t.scalar_type() != dt)
    fail(PyExc_TypeError, "%s has dtype %s, expected %s", name, c10::toString(t.scalar_type()),
         c10::toString(dt));
  if (t.sizes() != shape)
    fail(PyExc_ValueError, "%s has shape %s, expected %s", name, text(t.sizes()).c_str(),
         text(shape).c_str());
  if (!t.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", name);
  if (t.get_device() != dev)
    fail(PyExc_ValueError, "%s lies on cuda:%d, the current device is cuda:%d", name,
         static_cast<int>(t.get_device()), dev);
}

const Tensor& wanted(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType dt, int dev) {
  const Tensor& t = tensor(o, name);
  want(t, name, shape, dt, dev);
  return t;
}

// The tensor given, checked, or a new one.
Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType dt, int dev,
              const Tensor& like) {
  if (o == Py_None) return at::empty(shape, like.options().dtype(dt));
  return wanted(o, name, shape, dt, dev);
}

// A workspace given, or a new one of n bytes.
Tensor workspace(PyObject* o, size_t n, int dev, const Tensor& like) {
  if (o == Py_None)
    return at::empty({static_cast<int64_t>(n < 16 ? 16 : n)}, like.options().dtype(at::kByte));
  const Tensor& t = tensor(o, "workspace");
  want(t, "workspace", t.sizes(), t.scalar_type(), dev);
  return t;
}

int number(PyObject* o, const char* name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  if (v < INT_MIN || v > INT_MAX) fail(PyExc_ValueError, "%s = %ld is out of range", name, v);
  return static_cast<int>(v);
}

// The stream of a call: a stream object, a raw handle, or None for the current
// stream.  While it lives, what the call allocates belongs to that stream, so
// that its memory is not given to another's work before the kernels are done.
class Stream {
 public:
  Stream(PyObject* o, int dev) {
    const auto d = static_cast<c10::DeviceIndex>(dev);
    if (o == Py_None) {
      handle_ = c10::cuda::getCurrentCUDAStream(d).stream();
      return;
    }
    PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
    if (h == nullptr) {
      PyErr_Clear();
      Py_INCREF(o);
      h = o;
    }
    handle_ = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (handle_ == nullptr && PyErr_Occurred()) throw python_error();
    guard_.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle_), d));
  }
  operator void*() const { return handle_; }

 private:
  void* handle_ = nullptr;
  c10::cuda::OptionalCUDAStreamGuard guard_;
};

bool truth(PyObject* o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw python_error();
  return r == 1;
}

int dtype_code(const Tensor& t) {
  if (t.scalar_type() == at::kHalf) return FA_F16;
  if (t.scalar_type() == at::kBFloat16) return FA_BF16;
  fail(PyExc_TypeError, "dtype %s unsupported: use float16 or bfloat16", c10::toString(t.scalar_type()));
}

// Sizes of a 4-D tensor.
struct Four {
  int64_t a, b, c, d;
};
Four four(const Tensor& t, const char* name) {
  if (t.dim() != 4) fail(PyExc_ValueError, "%s must have four dimensions", name);
  return {t.size(0), t.size(1), t.size(2), t.size(3)};
}

int small(int64_t v) {
  if (v > INT_MAX) fail(PyExc_ValueError, "a size of %lld is out of range", static_cast<long long>(v));
  return static_cast<int>(v);
}

// Two pools [pages, page, Hkv, D] alike, whose pages may lie apart but are
// contiguous in themselves.
struct Pools {
  const Tensor &k, &v;
  int64_t pages, page, hkv, d;
  long long kst, vst;  // elements between two pages
};
Pools pools(PyObject* ko, PyObject* vo, at::ScalarType dt, int dev) {
  const Tensor &k = tensor(ko, "k_cache"), &v = tensor(vo, "v_cache");
  const Four s = four(k, "k_cache");
  Pools p{k, v, s.a, s.b, s.c, s.d, 0, 0};
  for (const Tensor* t : {&k, &v}) {
    const char* name = t == &k ? "k_cache" : "v_cache";
    if (t->scalar_type() != dt)
      fail(PyExc_TypeError, "%s has dtype %s, expected %s", name, c10::toString(t->scalar_type()),
                             c10::toString(dt));
    if (t->sizes() != k.sizes())
      fail(PyExc_ValueError, "%s must be [pages, page, Hkv, D], both pools alike", name);
    if (t->stride(3) != 1 || t->stride(2) != s.d || t->stride(1) != s.c * s.d)
      fail(PyExc_ValueError, "the pages of %s must be contiguous", name);
    if (t->get_device() != dev)
      fail(PyExc_ValueError, "%s lies on cuda:%d, the current device is cuda:%d", name,
           static_cast<int>(t->get_device()), dev);
    (t == &k ? p.kst : p.vst) = s.a > 1 ? t->stride(0) : s.b * s.c * s.d;
  }
  return p;
}

// Key weights [B, Hkv, >= cap] fp32; the elements between their rows in `stride`.
float* weights_of(PyObject* o, int64_t B, int64_t hkv, int64_t cap, int dev, long long& stride) {
  const Tensor& t = tensor(o, "weights");
  if (t.dim() != 3 || t.size(0) != B || t.size(1) != hkv || t.size(2) < cap)
    fail(PyExc_ValueError, "weights has shape %s, expected (%lld, %lld, >= %lld)",
                            text(t.sizes()).c_str(), static_cast<long long>(B),
                            static_cast<long long>(hkv), static_cast<long long>(cap));
  want(t, "weights", t.sizes(), kF32, dev);
  stride = t.size(2);
  return t.data_ptr<float>();
}

int64_t columns(const Tensor& t, const char* name) {
  if (t.dim() != 2) fail(PyExc_ValueError, "%s must have two dimensions", name);
  return t.size(1);
}

const int* ints(const Tensor& t) { return t.data_ptr<int>(); }

PyObject* status(fa_status st) { return PyLong_FromLong(st); }

PyObject* tuple_of(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (r == nullptr) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
  return r;
}

void arguments(Py_ssize_t n, Py_ssize_t expected) {
  if (n != expected)
    fail(PyExc_TypeError, "%lld arguments, expected %lld", static_cast<long long>(n),
                           static_cast<long long>(expected));
}

// (q, k, v, window, sinks, out, lse, stream)
PyObject* window_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 8);
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
  const int dev = c10::cuda::current_device();
  const Four s = four(q, "q"), c = four(k, "k");
  const auto dt = q.scalar_type();
  const int code = dtype_code(q);
  const int64_t kv[4] = {s.a, c.b, c.c, s.d}, ls[3] = {s.a, s.c, s.b};
  want(q, "q", q.sizes(), dt, dev);
  want(k, "k", kv, dt, dev);
  const Tensor& v = wanted(a[2], "v", kv, dt, dev);
  const int window = number(a[3], "window"), sinks = number(a[4], "sinks");
  const Stream stream(a[7], dev);
  const Tensor out = output(a[5], "out", q.sizes(), dt, dev, q);
  const Tensor lse = output(a[6], "lse", ls, kF32, dev, q);
  const fa_status st =
      fa_window_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr<float>(),
                    small(s.a), small(s.b), small(c.b), small(s.c), small(c.c), small(s.d), window,
                    sinks, code, stream);
  return st == FA_OK ? tuple_of({out, lse}) : status(st);
  END_HANDLE_TH_ERRORS
}

// (q, k, v, o or None, lse, do, delta or None, window, sinks, dq, dk, dv,
//  workspace, zeroed, stream): with o, Delta is computed (and the workspace's
// accumulator zeroed) first.  Returns dq, dk, dv, delta.
PyObject* window_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 15);
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
  const int dev = c10::cuda::current_device();
  const Four s = four(q, "q"), c = four(k, "k");
  const auto dt = q.scalar_type();
  const int code = dtype_code(q);
  const int64_t kv[4] = {s.a, c.b, c.c, s.d}, ls[3] = {s.a, s.c, s.b};
  want(q, "q", q.sizes(), dt, dev);
  want(k, "k", kv, dt, dev);
  const Tensor& v = wanted(a[2], "v", kv, dt, dev);
  const Tensor& lse = wanted(a[4], "lse", ls, kF32, dev);
  const Tensor& grad = wanted(a[5], "do", q.sizes(), dt, dev);
  const int window = number(a[7], "window"), sinks = number(a[8], "sinks");
  const int B = small(s.a), L = small(s.b), Lk = small(c.b), H = small(s.c), Hkv = small(c.c),
            D = small(s.d);
  const bool prep = a[3] != Py_None, zeroed = a[12] != Py_None && truth(a[13]);
  const Stream stream(a[14], dev);
  if (prep) wanted(a[3], "o", q.sizes(), dt, dev);
  const Tensor delta = output(a[6], "delta", ls, kF32, dev, q);
  if (!prep && a[6] == Py_None) fail(PyExc_TypeError, "delta must be a CUDA tensor");
  const Tensor dq = output(a[9], "dq", q.sizes(), dt, dev, q);
  const Tensor dk = output(a[10], "dk", kv, dt, dev, q);
  const Tensor dv = output(a[11], "dv", kv, dt, dev, q);
  const size_t need = fa_window_bwd_workspace_size(B, L, Lk, H, Hkv, D, window, sinks);  // 0: refused below
  const Tensor ws = workspace(a[12], need, dev, q);
  const size_t bytes = ws.numel() * ws.element_size();
  if (bytes < need) return status(FA_ERR_SCRATCH_TOO_SMALL);
  fa_status st = FA_OK;
  if (prep && need != 0) {
    st = fa_bwd_preprocess(THPVariable_Unpack(a[3]).data_ptr(), grad.data_ptr(),
                           delta.data_ptr<float>(), static_cast<float*>(ws.data_ptr()), B, L, H, D,
                           code, stream);
    if (st != FA_OK) return status(st);
  }
  st = fa_window_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), grad.data_ptr(), lse.data_ptr<float>(),
                     delta.data_ptr<float>(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                     static_cast<float*>(ws.data_ptr()), bytes, prep || zeroed ? 0 : 1, B, L, Lk, H,
                     Hkv, D, window, sinks, code, stream);
  return st == FA_OK ? tuple_of({dq, dk, dv, delta}) : status(st);
  END_HANDLE_TH_ERRORS
}

// (k, v, k_cache, v_cache, block_table, start, counts, weights, new_weights, stream)
PyObject* paged_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 10);
  const Tensor& k = tensor(a[0], "k");
  const int dev = c10::cuda::current_device();
  const Four s = four(k, "k");
  const auto dt = k.scalar_type();
  const int code = dtype_code(k);
  const Pools p = pools(a[2], a[3], dt, dev);
  const int64_t shape[4] = {s.a, s.b, p.hkv, p.d};
  want(k, "k", shape, dt, dev);
  const Tensor& v = wanted(a[1], "v", shape, dt, dev);
  const Tensor& table = tensor(a[4], "block_table");
  const int64_t P = columns(table, "block_table"), ts[2] = {s.a, P}, bs[1] = {s.a};
  want(table, "block_table", ts, kI32, dev);
  const Tensor& start = wanted(a[5], "start", bs, kI32, dev);
  const int* counts = a[6] == Py_None ? nullptr : ints(wanted(a[6], "counts", bs, kI32, dev));
  long long wst = 0;
  float* w = a[7] == Py_None ? nullptr : weights_of(a[7], s.a, p.hkv, P * p.page, dev, wst);
  const int64_t ns[3] = {s.a, p.hkv, s.b};
  const float* nw =
      a[8] == Py_None ? nullptr : wanted(a[8], "new_weights", ns, kF32, dev).data_ptr<float>();
  return status(fa_paged_write(k.data_ptr(), v.data_ptr(), p.k.data_ptr(), p.v.data_ptr(), p.kst,
                               p.vst, ints(table), ints(start), counts, w, wst, nw, small(s.a),
                               small(s.b), small(p.hkv), small(p.d), small(p.page), small(P),
                               small(p.pages), code, Stream(a[9], dev)));
  END_HANDLE_TH_ERRORS
}

// (q, k_cache, v_cache, block_table, lens, window, sinks, weights, out, lse, workspace, stream)
PyObject* paged_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 12);
  const Tensor& q = tensor(a[0], "q");
  const int dev = c10::cuda::current_device();
  const Four s = four(q, "q");
  const auto dt = q.scalar_type();
  const int code = dtype_code(q);
  const Pools p = pools(a[1], a[2], dt, dev);
  const int64_t qs[4] = {s.a, s.b, s.c, p.d}, ls[3] = {s.a, s.c, s.b}, bs[1] = {s.a};
  want(q, "q", qs, dt, dev);
  const Tensor& table = tensor(a[3], "block_table");
  const int64_t P = columns(table, "block_table"), ts[2] = {s.a, P};
  want(table, "block_table", ts, kI32, dev);
  const Tensor& lens = wanted(a[4], "lens", bs, kI32, dev);
  const int window = number(a[5], "window"), sinks = number(a[6], "sinks");
  long long wst = 0;
  float* w = a[7] == Py_None ? nullptr : weights_of(a[7], s.a, p.hkv, P * p.page, dev, wst);
  const int B = small(s.a), Lq = small(s.b), H = small(s.c), Hkv = small(p.hkv), D = small(p.d),
            page = small(p.page);
  const Stream stream(a[11], dev);
  const Tensor out = output(a[8], "out", qs, dt, dev, q);
  const Tensor lse = output(a[9], "lse", ls, kF32, dev, q);
  const Tensor ws = workspace(
      a[10], fa_paged_decode_workspace_size(B, Lq, H, Hkv, D, page, small(P), w != nullptr), dev, q);
  const fa_status st = fa_paged_decode(
      q.data_ptr(), p.k.data_ptr(), p.v.data_ptr(), p.kst, p.vst, ints(table), ints(lens),
      out.data_ptr(), lse.data_ptr<float>(), w, wst, ws.data_ptr(), ws.numel() * ws.element_size(), B,
      Lq, H, Hkv, D, page, small(P), small(p.pages), window, sinks, code, stream);
  return st == FA_OK ? tuple_of({out, lse}) : status(st);
  END_HANDLE_TH_ERRORS
}

// (k_cache, v_cache, block_table, lens, weights, dst_table, keep, sinks, recent, kept,
//  new_lens, new_weights, stream)
PyObject* paged_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 13);
  const Tensor& k = tensor(a[0], "k_cache");
  const int dev = c10::cuda::current_device();
  const int code = dtype_code(k);
  const Pools p = pools(a[0], a[1], k.scalar_type(), dev);
  const Tensor &table = tensor(a[2], "block_table"), &dst = tensor(a[5], "dst_table");
  const int64_t P = columns(table, "block_table"), P2 = columns(dst, "dst_table"), B = table.size(0);
  const int64_t ts[2] = {B, P}, ds[2] = {B, P2}, bs[1] = {B};
  want(table, "block_table", ts, kI32, dev);
  want(dst, "dst_table", ds, kI32, dev);
  const Tensor& lens = wanted(a[3], "lens", bs, kI32, dev);
  long long wst = 0;
  const float* w = weights_of(a[4], B, p.hkv, P * p.page, dev, wst);
  const int keep = number(a[6], "keep"), sinks = number(a[7], "sinks"), recent = number(a[8], "recent");
  if (keep < 1) fail(PyExc_ValueError, "keep must be at least 1");
  const int64_t ks[3] = {B, p.hkv, keep}, ns[3] = {B, p.hkv, P2 * p.page};
  const Stream stream(a[12], dev);
  const Tensor kept = output(a[9], "kept", ks, kI32, dev, k);
  const Tensor new_lens = output(a[10], "new_lens", bs, kI32, dev, k);
  const Tensor new_w = output(a[11], "new_weights", ns, kF32, dev, k);
  const fa_status st = fa_paged_evict(
      p.k.data_ptr(), p.v.data_ptr(), p.kst, p.vst, ints(table), ints(lens), w, wst, ints(dst), keep,
      sinks, recent, kept.data_ptr<int>(), new_lens.data_ptr<int>(), new_w.data_ptr<float>(), small(B),
      small(p.hkv), small(p.d), small(p.page), small(P), small(P2), small(p.pages), code,
      stream);
  return st == FA_OK ? tuple_of({kept, new_lens, new_w}) : status(st);
  END_HANDLE_TH_ERRORS
}

// (q, k, lse, causal, window, sinks, out, workspace, stream)
PyObject* key_weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 9);
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
  const int dev = c10::cuda::current_device();
  const Four s = four(q, "q"), c = four(k, "k");
  const auto dt = q.scalar_type();
  const int code = dtype_code(q);
  const int64_t kv[4] = {s.a, c.b, c.c, s.d}, ls[3] = {s.a, s.c, s.b}, os[3] = {s.a, c.c, c.b};
  want(q, "q", q.sizes(), dt, dev);
  want(k, "k", kv, dt, dev);
  const Tensor& lse = wanted(a[2], "lse", ls, kF32, dev);
  const int causal = truth(a[3]) ? 1 : 0;
  const int window = number(a[4], "window"), sinks = number(a[5], "sinks");
  const Stream stream(a[8], dev);
  const Tensor out = output(a[6], "out", os, kF32, dev, q);
  const Tensor ws = workspace(a[7], fa_key_weights_workspace_size(), dev, q);
  const fa_status st = fa_key_weights(
      q.data_ptr(), k.data_ptr(), lse.data_ptr<float>(), out.data_ptr<float>(), ws.data_ptr(),
      ws.numel() * ws.element_size(), small(s.a), small(s.b), small(c.b), small(s.c), small(c.c),
      small(s.d), causal, window, sinks, code, stream);
  return st == FA_OK ? THPVariable_Wrap(out) : status(st);
  END_HANDLE_TH_ERRORS
}

#define FA_METHOD(f) \
  { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {FA_METHOD(window_fwd),   FA_METHOD(window_bwd),  FA_METHOD(paged_write),
                         FA_METHOD(paged_decode), FA_METHOD(paged_evict), FA_METHOD(key_weights),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
