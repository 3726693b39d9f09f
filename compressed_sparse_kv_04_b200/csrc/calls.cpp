// Python calls of the 4-bit cache, its attention and the 4-bit projection:
// argument checks on torch tensors and the C entry point (include/csa.h) in one
// step.
//
// These calls are short on the device (a few microseconds), so a program that
// makes them one by one waits for the host.  Of that a cache write takes 3.2 us
// here, an attention call 6, the projection 8.5; through Python checks and ctypes
// they took 7.4, 13 and 16.  (One launch alone, from C: 2.9.)
//
// The module holds no copy of the library: bind() gets the entry points'
// addresses from the one that the binding has loaded.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>
#include <exception>
#include <initializer_list>
#include <sstream>
#include <string>

#include "../../include/csa.h"

namespace {

decltype(&::mxfp4_row_bytes) row_bytes = nullptr;
decltype(&::mxfp4_cache_write) cache_write = nullptr;
decltype(&::mxfp4_cache_read) cache_read = nullptr;
decltype(&::sparse_mqa_decode_mxfp4) sparse_decode = nullptr;
decltype(&::dense_mqa_decode_mxfp4) dense_decode = nullptr;
decltype(&::grouped_out_proj_mxfp4) out_proj = nullptr;

// A Python exception is set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& msg) {
  PyErr_SetString(type, msg.c_str());
  throw Raised();
}

constexpr auto kU8 = at::kByte;
constexpr auto kBf16 = at::kBFloat16;
constexpr auto kF32 = at::kFloat;
constexpr auto kI32 = at::kInt;
constexpr auto kI64 = at::kLong;

const char* type_name(at::ScalarType t) {
  switch (t) {
    case kU8: return "torch.uint8";
    case kBf16: return "torch.bfloat16";
    case kF32: return "torch.float32";
    case kI32: return "torch.int32";
    case kI64: return "torch.int64";
    default: return c10::toString(t);
  }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o))
    raise(PyExc_TypeError,
          std::string(name) + ": expected a torch.Tensor, got " + Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

// The current CUDA device, which every tensor of a call has to be on; -2 (no
// tensor's device) where there is none.
int current_device() {
  try {
    return c10::cuda::current_device();
  } catch (const std::exception&) {
    return -2;
  }
}

void on_device(const at::Tensor& t, const char* name, int dev) {
  if (!t.is_cuda() || t.get_device() != dev) {
    std::ostringstream s;
    s << name << " is on " << t.device() << ", not on the current CUDA device";
    raise(PyExc_ValueError, s.str());
  }
}

// Address of a tensor that must have this type and shape, be contiguous and sit
// on the device; None passes as null.
void* need(PyObject* o, const char* name, int dev, at::ScalarType type,
           std::initializer_list<int64_t> shape) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  const at::IntArrayRef want(shape);
  if (t.scalar_type() != type || t.sizes() != want) {
    std::ostringstream s;
    s << name << " must be " << type_name(type) << ' ' << want << ", not "
      << type_name(t.scalar_type()) << ' ' << t.sizes();
    raise(PyExc_ValueError, s.str());
  }
  on_device(t, name, dev);
  if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
  return t.data_ptr();
}

template <typename T>
T* need_as(PyObject* o, const char* name, int dev, at::ScalarType type,
           std::initializer_list<int64_t> shape) {
  return static_cast<T*>(need(o, name, dev, type, shape));
}

// Length of a dimension that the call itself reads.
int64_t length(PyObject* o, const char* name, int64_t dim) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() <= dim)
    raise(PyExc_ValueError,
          std::string(name) + " has " + std::to_string(t.dim()) + " dimensions");
  return t.size(dim);
}

// A workspace: any type and shape.
std::pair<void*, size_t> workspace(PyObject* o, int dev) {
  if (o == Py_None) return {nullptr, 0};
  const at::Tensor& t = tensor(o, "ws");
  on_device(t, "ws", dev);
  if (!t.is_contiguous()) raise(PyExc_ValueError, "ws must be contiguous");
  return {t.data_ptr(), t.nbytes()};
}

// The csa_params behind its ctypes structure.
class Params {
 public:
  explicit Params(PyObject* o) {
    if (PyObject_GetBuffer(o, &view_, PyBUF_SIMPLE) != 0) throw Raised();
    if (view_.len != (Py_ssize_t)sizeof(csa_params)) {
      PyBuffer_Release(&view_);
      raise(PyExc_TypeError, "p: expected csa_params");
    }
  }
  ~Params() { PyBuffer_Release(&view_); }
  Params(const Params&) = delete;
  Params& operator=(const Params&) = delete;
  const csa_params* get() const { return static_cast<const csa_params*>(view_.buf); }
  const csa_params* operator->() const { return get(); }

 private:
  Py_buffer view_;
};

void* raw_stream(PyObject* o, int dev) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
  PyObject* v = PyObject_GetAttrString(o, "cuda_stream");
  if (!v) throw Raised();
  void* s = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  if (!s && PyErr_Occurred()) throw Raised();
  return s;
}

int64_t* opt_i64(PyObject* o, const char* name, int dev, int64_t B) {
  return need_as<int64_t>(o, name, dev, kI64, {B});
}
int32_t* status_word(PyObject* o, int dev) {
  return need_as<int32_t>(o, "dev_status", dev, kI32, {1});
}

// mxfp4_row_bytes(d), or -1 where the library refuses d.
int64_t row_of(int d) {
  const size_t n = row_bytes(d);
  return n ? (int64_t)n : -1;
}

template <typename F>
long without_gil(F&& f) {
  long st;
  Py_BEGIN_ALLOW_THREADS;
  st = (long)f();
  Py_END_ALLOW_THREADS;
  return st;
}

// (p, rows, kv4, first_entry, count, dev_status, stream)
long do_write(PyObject* const* a) {
  const int dev = current_device();
  const Params p(a[0]);
  const int64_t B = p->B, d = p->d, n = length(a[1], "rows", 1), N = length(a[2], "kv4", 1);
  const int64_t row = row_of(p->d);
  if (row < 0) return CSA_ERR_UNSUPPORTED_SHAPE;
  const at::Tensor& rows = tensor(a[1], "rows");
  if (rows.scalar_type() != kBf16 || rows.sizes() != at::IntArrayRef({B, n, d})) {
    std::ostringstream s;
    s << "rows must be torch.bfloat16 " << at::IntArrayRef({B, n, d}) << ", not "
      << type_name(rows.scalar_type()) << ' ' << rows.sizes();
    raise(PyExc_ValueError, s.str());
  }
  // Sequences may lie apart, a sequence's rows not.
  if (n > 0 && (rows.stride(2) != 1 || (n > 1 && rows.stride(1) != d)))
    raise(PyExc_ValueError, "each sequence's rows must be contiguous");
  on_device(rows, "rows", dev);
  const void* src = rows.data_ptr();
  const int64_t stride = B > 1 ? rows.stride(0) : n * d;
  const int64_t* first = opt_i64(a[3], "first_entry", dev, B);
  const int64_t* count = opt_i64(a[4], "count", dev, B);
  void* kv4 = need(a[2], "kv4", dev, kU8, {B, N, row});
  int32_t* status = status_word(a[5], dev);
  void* stream = raw_stream(a[6], dev);
  return without_gil([&] {
    return cache_write(p.get(), src, stride, n, first, count, kv4, N, status, stream);
  });
}

// (p, kv4, rows, idx, first_entry, count, dev_status, stream)
long do_read(PyObject* const* a) {
  const int dev = current_device();
  const Params p(a[0]);
  const int64_t B = p->B, d = p->d, n = length(a[2], "rows", 1), N = length(a[1], "kv4", 1);
  const int64_t row = row_of(p->d);
  if (row < 0) return CSA_ERR_UNSUPPORTED_SHAPE;
  void* rows = need(a[2], "rows", dev, kBf16, {B, n, d});
  const void* kv4 = need(a[1], "kv4", dev, kU8, {B, N, row});
  const int32_t* idx = need_as<int32_t>(a[3], "idx", dev, kI32, {B, n});
  const int64_t* first = opt_i64(a[4], "first_entry", dev, B);
  const int64_t* count = opt_i64(a[5], "count", dev, B);
  int32_t* status = status_word(a[6], dev);
  void* stream = raw_stream(a[7], dev);
  return without_gil([&] {
    return cache_read(p.get(), kv4, N, idx, first, count, n, rows, status, stream);
  });
}

// (p, q, pos_q, kv4, [topk_idx, topk_cnt,] kv_tok, sink, out, gamma_q, gamma_kv,
// lse, ws, dev_status, stream)
template <bool kSparse>
long do_decode(PyObject* const* a) {
  constexpr int k = kSparse ? 2 : 0;
  const int dev = current_device();
  const Params p(a[0]);
  const int64_t B = p->B, H = p->H, d = p->d;
  const int64_t N = length(a[3], "kv4", 1), L = length(a[4 + k], "kv_tok", 1);
  const int64_t row = row_of(p->d);
  if (row < 0) return CSA_ERR_UNSUPPORTED_SHAPE;
  const void* q = need(a[1], "q", dev, kBf16, {B, H, d});
  const int64_t* pos = opt_i64(a[2], "pos_q", dev, B);
  const void* kv4 = need(a[3], "kv4", dev, kU8, {B, N, row});
  const int32_t *idx = nullptr, *cnt = nullptr;
  if (kSparse) {
    idx = need_as<int32_t>(a[4], "topk_idx", dev, kI32, {B, p->k});
    cnt = need_as<int32_t>(a[5], "topk_cnt", dev, kI32, {B});
  }
  const void* tok = need(a[4 + k], "kv_tok", dev, kBf16, {B, L, d});
  const float* sink = need_as<float>(a[5 + k], "sink", dev, kF32, {H});
  void* out = need(a[6 + k], "out", dev, kBf16, {B, H, d});
  const float* gq = need_as<float>(a[7 + k], "gamma_q", dev, kF32, {d});
  const float* gkv = need_as<float>(a[8 + k], "gamma_kv", dev, kF32, {d});
  float* lse = need_as<float>(a[9 + k], "lse", dev, kF32, {B, H});
  const auto ws = workspace(a[10 + k], dev);
  int32_t* status = status_word(a[11 + k], dev);
  void* stream = raw_stream(a[12 + k], dev);
  return without_gil([&] {
    if (kSparse)
      return sparse_decode(p.get(), q, pos, kv4, N, idx, cnt, tok, L, sink, gq, gkv, out, lse,
                           ws.first, ws.second, status, stream);
    return dense_decode(p.get(), q, pos, kv4, N, tok, L, sink, gq, gkv, out, lse, ws.first,
                        ws.second, status, stream);
  });
}

// Scale tiles: `bytes` bytes in any shape.
const void* need_scales(PyObject* o, const char* name, int dev, int64_t bytes) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != kU8 || t.numel() != bytes) {
    std::ostringstream s;
    s << name << " must hold " << bytes << " bytes, not " << t.numel() << " of "
      << type_name(t.scalar_type());
    raise(PyExc_ValueError, s.str());
  }
  on_device(t, name, dev);
  if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
  return t.data_ptr();
}

int checked_int(int64_t v, const char* what) {
  if (v > INT32_MAX) raise(PyExc_ValueError, std::string(what) + " is too long");
  return (int)v;
}

// (o, w_g, w_g_scale, w_o, w_o_scale, z, y, ws, dev_status, stream)
long do_project(PyObject* const* a) {
  const int dev = current_device();
  const at::Tensor& o = tensor(a[0], "o");
  if (o.dim() != 3) raise(PyExc_ValueError, "o must be [T, H, D]");
  const int T = checked_int(o.size(0), "o"), H = checked_int(o.size(1), "o"),
            D = checked_int(o.size(2), "o");
  const int g = checked_int(length(a[1], "w_g", 0), "w_g"),
            d_g = checked_int(length(a[1], "w_g", 1), "w_g"),
            d_model = checked_int(length(a[3], "w_o", 0), "w_o");
  // (Products of two such sizes fit 64 bits; the library refuses large ones.)
  const int64_t k1 = (int64_t)(H / std::max(g, 1)) * D, k2 = (int64_t)g * d_g;
  const void* op = need(a[0], "o", dev, kBf16, {T, H, D});
  const void* wg = need(a[1], "w_g", dev, kU8, {g, d_g, k1 / 2});
  const void* wgs = need_scales(a[2], "w_g_scale", dev, (k2 + 127) / 128 * (k1 / 128) * 512);
  const void* wo = need(a[3], "w_o", dev, kU8, {d_model, k2 / 2});
  const void* wos =
      need_scales(a[4], "w_o_scale", dev, ((int64_t)d_model + 127) / 128 * (k2 / 128) * 512);
  void* z = need(a[5], "z", dev, kBf16, {T, d_model});
  void* y = need(a[6], "y", dev, kBf16, {T, k2});
  const auto ws = workspace(a[7], dev);
  int32_t* status = status_word(a[8], dev);
  void* stream = raw_stream(a[9], dev);
  return without_gil([&] {
    return out_proj(T, H, D, g, d_g, d_model, op, wg, wgs, wo, wos, y, z, ws.first, ws.second,
                    status, stream);
  });
}

// A call of kArgs positional arguments; its csa_status as an int.
template <long (*kCall)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs || !cache_write) {
    PyErr_SetString(PyExc_TypeError, n != kArgs ? "wrong number of arguments" : "not bound");
    return nullptr;
  }
  try {
    return PyLong_FromLong(kCall(args));
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// bind(row_bytes, cache_write, cache_read, sparse_decode, dense_decode, out_proj):
// the addresses of the entry points.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  constexpr int kN = 6;
  void* f[kN];
  if (n != kN) {
    PyErr_SetString(PyExc_TypeError, "bind takes six addresses");
    return nullptr;
  }
  for (int i = 0; i < kN; ++i) {
    f[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
    if (!f[i]) {
      PyErr_SetString(PyExc_ValueError, "a null address");
      return nullptr;
    }
  }
  row_bytes = reinterpret_cast<decltype(row_bytes)>(f[0]);
  cache_write = reinterpret_cast<decltype(cache_write)>(f[1]);
  cache_read = reinterpret_cast<decltype(cache_read)>(f[2]);
  sparse_decode = reinterpret_cast<decltype(sparse_decode)>(f[3]);
  dense_decode = reinterpret_cast<decltype(dense_decode)>(f[4]);
  out_proj = reinterpret_cast<decltype(out_proj)>(f[5]);
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {
    {"bind", FAST(bind), "Addresses of the library's entry points."},
    {"cache_write", FAST((entry<do_write, 7>)), "mxfp4_cache_write"},
    {"cache_read", FAST((entry<do_read, 8>)), "mxfp4_cache_read"},
    {"sparse_decode", FAST((entry<do_decode<true>, 15>)), "sparse_mqa_decode_mxfp4"},
    {"dense_decode", FAST((entry<do_decode<false>, 13>)), "dense_mqa_decode_mxfp4"},
    {"out_proj", FAST((entry<do_project, 10>)), "grouped_out_proj_mxfp4"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls",
                      "Checked calls of the 4-bit cache, its attention and projection.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the torch and Python whose headers this module was compiled against
// (the build passes it); the binding refuses it under others.
PyMODINIT_FUNC PyInit__calls() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", CSA_CALLS_TAG) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
