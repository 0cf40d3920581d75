// block_calls.cpp -- the marshalling of the calls that a decode step makes between its
// products (norm, rotary positions, the 4-bit cache), for binding.py.
//
// Such a call's kernels take 2 to 10 us; checking a dozen tensors, allocating the
// outputs and converting twenty ctypes arguments in Python takes 10 to 20.  The
// same checks, with the same exceptions, and the allocations are made here, and
// the C calls of include/qk.h with the raw pointers: 3 to 7 us with the launches (2.4 us each).
// Nothing is computed here.  The C calls and the allocations run without the interpreter's lock, as
// through ctypes: a launch waits where the queue is full.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "qk.h"

namespace {

using at::ScalarType;
using at::Tensor;
using std::string;

[[noreturn]] void value_error(const string& s) {
  PyErr_SetString(PyExc_ValueError, s.c_str());
  throw python_error();
}
[[noreturn]] void type_error(const string& s) {
  PyErr_SetString(PyExc_TypeError, s.c_str());
  throw python_error();
}

// What f does, without the interpreter's lock (taken again when it throws, too).
template <typename F>
auto unlocked(F f) {
  struct Lock {
    PyThreadState* state = PyEval_SaveThread();
    ~Lock() { PyEval_RestoreThread(state); }
  } lock;
  return f();
}

string text(at::IntArrayRef v) {
  string s = "(";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + (v.size() == 1 ? ",)" : ")");
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

void need_type(const Tensor& t, ScalarType dtype, const char* name) {
  if (t.scalar_type() != dtype)
    type_error(string(name) + " must be " + c10::toString(dtype) + ", got " + c10::toString(t.scalar_type()));
}

// A contiguous CUDA tensor of a type and number of dims.
const Tensor& need(PyObject* o, ScalarType dtype, int64_t dims, const char* name) {
  const Tensor& t = tensor(o, name);
  need_type(t, dtype, name);
  if (t.dim() != dims)
    value_error(string(name) + " must have " + std::to_string(dims) + " dims, got " + text(t.sizes()));
  if (!t.is_cuda()) value_error(string(name) + " must be a CUDA tensor");
  if (!t.is_contiguous()) value_error(string(name) + " must be contiguous");
  return t;
}

void need_shape(const Tensor& t, at::IntArrayRef shape, const char* name) {
  if (t.sizes() != shape)
    value_error(string(name) + " must have shape " + text(shape) + ", got " + text(t.sizes()));
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

qk_stream_t current_stream() { return c10::cuda::getCurrentCUDAStream().stream(); }
qk_stream_t stream_of(PyObject* o) {
  return o == Py_None ? current_stream() : reinterpret_cast<qk_stream_t>((uintptr_t)integer(o));
}

// New memory for an output, of the pool of the stream that writes it: the current stream's may
// still be read by what that stream has queued.
at::TensorBase memory(at::IntArrayRef shape, at::IntArrayRef stride, ScalarType dtype, at::Device device,
                      qk_stream_t stream) {
  return unlocked([&] {
    if (stream == current_stream()) return at::detail::empty_strided_cuda(shape, stride, dtype, device);
    const c10::cuda::CUDAStreamGuard guard(c10::cuda::getStreamFromExternal(stream, device.index()));
    return at::detail::empty_strided_cuda(shape, stride, dtype, device);
  });
}

// The tensor given for an output, or a new contiguous one.
Tensor output(PyObject* o, at::IntArrayRef shape, ScalarType dtype, const Tensor& beside, const char* name,
              qk_stream_t stream) {
  if (o == Py_None) {
    int64_t stride[4], step = 1;
    for (size_t i = shape.size(); i-- > 0;) {
      stride[i] = step;
      step *= shape[i] > 1 ? shape[i] : 1;
    }
    return Tensor(memory(shape, at::IntArrayRef(stride, shape.size()), dtype, beside.device(), stream));
  }
  const Tensor& t = need(o, dtype, (int64_t)shape.size(), name);
  need_shape(t, shape, name);
  return t;
}

// The row stride of a bf16 [T, heads, D] view whose heads lie next to each other (rows
// of a larger projection may lie further apart).
int64_t rows(const Tensor& t, int64_t heads, int64_t D, const char* name) {
  need_type(t, ScalarType::BFloat16, name);
  if (t.dim() != 3 || t.size(1) != heads || t.size(2) != D)
    value_error(string(name) + " must have shape [T, " + std::to_string(heads) + ", " + std::to_string(D) +
                "], got " + text(t.sizes()));
  if (!t.is_cuda()) value_error(string(name) + " must be a CUDA tensor");
  if (t.size(0) == 0) return heads * D;
  if ((D > 1 && t.stride(2) != 1) || (heads > 1 && t.stride(1) != D))
    value_error(string(name) + ": a row's heads must be contiguous");
  return t.size(0) > 1 ? t.stride(0) : heads * D;  // (of a single row any stride)
}

// New contiguous tensors in one allocation, 256 bytes apart: an allocation and its
// release take 0.8 us, a tensor beside another one 0.15.
class Together {
 public:
  Together(const Tensor& beside, qk_stream_t stream) : device_(beside.device()), stream_(stream) {}
  void add(Tensor* out, std::initializer_list<int64_t> shape, ScalarType dtype) {
    Part& p = parts_[n_++];
    p = {out, {}, (int)shape.size(), dtype, bytes_};
    int64_t count = 1;
    std::copy(shape.begin(), shape.end(), p.shape);
    for (int64_t x : shape) count *= x;
    bytes_ += (count * (int64_t)c10::elementSize(dtype) + 255) / 256 * 256;
  }
  void make() {
    if (n_ == 0) return;
    const int64_t one = 1;
    const at::TensorBase all = memory(bytes_, one, ScalarType::Byte, device_, stream_);
    for (int i = 0; i < n_; ++i) {
      const Part& p = parts_[i];
      auto impl = c10::make_intrusive<at::TensorImpl>(c10::Storage(all.storage()), all.key_set(),
                                                      c10::scalarTypeToTypeMeta(p.dtype));
      impl->set_sizes_contiguous(at::IntArrayRef(p.shape, p.dims));
      impl->set_storage_offset(p.at / (int64_t)c10::elementSize(p.dtype));
      *p.out = Tensor(std::move(impl));
    }
  }

 private:
  struct Part {
    Tensor* out;
    int64_t shape[3];
    int dims;
    ScalarType dtype;
    int64_t at;
  };
  Part parts_[3];
  int n_ = 0;
  int64_t bytes_ = 0;
  at::Device device_;
  qk_stream_t stream_;
};

const Tensor& rows_of_three(PyObject* o, const char* name, const char* shape) {
  if (!THPVariable_Check(o) || THPVariable_Unpack(o).dim() != 3)
    value_error(string(name) + " must be a " + shape + " tensor");
  return THPVariable_Unpack(o);
}

// Every tensor on the current device, where the kernels launch.
template <typename... T>
void same_device(const T&... t) {
  const auto here = c10::cuda::current_device();
  auto check = [&](const Tensor& x) {
    if (x.defined() && (!x.is_cuda() || x.get_device() != here))
      value_error("a tensor of shape " + text(x.sizes()) + " is on " + x.device().str() +
                  ", and the current device is cuda:" + std::to_string((int)here));
  };
  (check(t), ...);
}

template <typename P>
P* ptr(const Tensor& t) {
  return t.defined() ? static_cast<P*>(t.data_ptr()) : nullptr;
}

void check(qk_status st, const char* where) {
  if (st == QK_OK) return;
  PyObject* binding = PyImport_ImportModule("w4a8_quantized_gemm_token_b200.binding");
  PyObject* type = binding ? PyObject_GetAttrString(binding, "QKError") : nullptr;
  PyObject* e = type ? PyObject_CallFunction(type, "is", (int)st, where) : nullptr;
  if (e) PyErr_SetObject(type, e);
  Py_XDECREF(e);
  Py_XDECREF(type);
  Py_XDECREF(binding);
  throw python_error();
}

// The object given, or the tensor that was made in its place.
PyObject* hand_back(PyObject* given, const Tensor& t) {
  if (given != Py_None || !t.defined()) {
    Py_INCREF(given);
    return given;
  }
  return THPVariable_Wrap(t);
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) type_error("wrong number of arguments");
}

PyObject* tuple_of(std::initializer_list<PyObject*> items) {
  PyObject* r = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  for (PyObject* o : items) PyTuple_SET_ITEM(r, i++, o);
  return r;
}

// x, weight, residual, eps, h, xq, sx, xsum, with_xsum, stream
PyObject* rmsnorm_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 10);
  const Tensor& x = need(a[0], ScalarType::BFloat16, 2, "x");
  const int64_t M = x.size(0), K = x.size(1);
  const qk_stream_t stream = stream_of(a[9]);
  Tensor weight, residual, h, xsum;
  if (a[1] != Py_None) {
    weight = need(a[1], ScalarType::Float, 1, "weight");
    if (weight.size(0) != K) value_error("weight must have shape [" + std::to_string(K) + "]");
  }
  if (a[2] != Py_None) {
    residual = need(a[2], ScalarType::BFloat16, 2, "residual");
    if (residual.sizes() != x.sizes()) value_error("residual must have x's shape");
    h = output(a[4], {M, K}, ScalarType::BFloat16, x, "h", stream);
  } else if (a[4] != Py_None) {
    value_error("h is written with a residual only");
  }
  const int sums = PyObject_IsTrue(a[8]);
  if (sums < 0) throw python_error();
  Tensor xq, sx;  // (used and released together, and with the sums)
  Together fresh(x, stream);
  auto take = [&](PyObject* o, Tensor* t, std::initializer_list<int64_t> shape, ScalarType dtype, const char* name) {
    if (o == Py_None)
      fresh.add(t, shape, dtype);
    else
      *t = output(o, shape, dtype, x, name, stream);
  };
  take(a[5], &xq, {M, K}, ScalarType::Char, "xq");
  take(a[6], &sx, {M}, ScalarType::Float, "sx");
  if (sums || a[7] != Py_None) take(a[7], &xsum, {M, K / 64}, ScalarType::Int, "xsum");
  fresh.make();
  same_device(x, weight, residual, h, xq, sx, xsum);
  const float eps = (float)number(a[3]);
  check(unlocked([&] {
          return qk_rmsnorm_quantize(ptr<uint16_t>(x), ptr<uint16_t>(residual), M, K, ptr<float>(weight), eps,
                                     ptr<uint16_t>(h), ptr<int8_t>(xq), ptr<float>(sx), ptr<int32_t>(xsum), stream);
        }),
        "qk_rmsnorm_quantize");
  return tuple_of({hand_back(a[4], h), hand_back(a[5], xq), hand_back(a[6], sx), hand_back(a[7], xsum)});
  END_HANDLE_TH_ERRORS
}

// q, k, positions, freq, layout, amplitude, q_out, k_out, stream
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 9);
  const Tensor& q = rows_of_three(a[0], "q", "[T, H, D]");
  const int64_t T = q.size(0), H = q.size(1), D = q.size(2);
  const int64_t qs = rows(q, H, D, "q");
  const Tensor& positions = need(a[2], ScalarType::Int, 1, "positions");
  const Tensor& freq = need(a[3], ScalarType::Double, 1, "freq");
  if (positions.size(0) != T) value_error("positions must have shape [" + std::to_string(T) + "]");
  const qk_stream_t stream = stream_of(a[8]);
  Tensor k, q_out, k_out;
  Together fresh(q, stream);
  auto out = [&](PyObject* o, Tensor* t, const Tensor& like, const char* name, int64_t* stride) {
    const int64_t heads = like.size(1);
    *stride = heads * D;
    if (o == Py_None) {
      fresh.add(t, {like.size(0), heads, D}, ScalarType::BFloat16);
    } else {
      *t = tensor(o, name);
      *stride = rows(*t, heads, D, name);
    }
  };
  int64_t qos, Hkv = 0, ks = 0, kos = 0;
  out(a[6], &q_out, q, "q_out", &qos);
  if (a[1] != Py_None) {
    k = rows_of_three(a[1], "k", "[T, Hkv, D]");
    Hkv = k.size(1);
    ks = rows(k, Hkv, D, "k");
    out(a[7], &k_out, k, "k_out", &kos);
  } else if (a[7] != Py_None) {
    value_error("k_out without k");
  }
  fresh.make();
  if (q_out.size(0) != T || (k.defined() && (k.size(0) != T || k_out.size(0) != T)))
    value_error("q, k and the outputs must have the same number of rows");
  same_device(q, k, positions, freq, q_out, k_out);
  const int layout = (int)integer(a[4]);
  const float amplitude = (float)number(a[5]);
  check(unlocked([&] {
          return qk_rope(ptr<uint16_t>(q), qs, ptr<uint16_t>(q_out), qos, H, ptr<uint16_t>(k), ks,
                         ptr<uint16_t>(k_out), kos, Hkv, T, D, 2 * freq.size(0), layout, ptr<int32_t>(positions),
                         ptr<double>(freq), amplitude, stream);
        }),
        "qk_rope");
  return tuple_of({hand_back(a[6], q_out), hand_back(a[7], k_out)});
  END_HANDLE_TH_ERRORS
}

// A cache uint8 [num_pages, Hkv, page, D + D/8] and its requests.
struct Cache {
  const Tensor &cache, &table, &lens;
  Tensor cu;
  int64_t num_pages, Hkv, page, D, B, max_pages;

  Cache(PyObject* c, PyObject* t, PyObject* l, PyObject* rows, int64_t T)
      : cache(need(c, ScalarType::Byte, 4, "cache")),
        table(need(t, ScalarType::Int, 2, "page_table")),
        lens(need(l, ScalarType::Int, 1, "kv_lens")) {
    num_pages = cache.size(0);
    Hkv = cache.size(1);
    page = cache.size(2);
    if (cache.size(3) % 9 != 0) value_error("cache must have shape [num_pages, Hkv, page, D + D / 8]");
    D = cache.size(3) / 9 * 8;
    B = table.size(0);
    max_pages = table.size(1);
    if (lens.size(0) != B) value_error("kv_lens must have shape [" + std::to_string(B) + "]");
    if (rows != Py_None) {
      cu = need(rows, ScalarType::Int, 1, "cu_rows");
      if (cu.size(0) != B + 1) value_error("cu_rows must have shape [" + std::to_string(B + 1) + "]");
    } else if (B == 0 ? T != 0 : T % B != 0) {
      value_error("without cu_rows every request has the same number of rows");
    }
  }
};

// k, v, cache, page_table, kv_lens, cu_rows, stream
PyObject* kv4_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 7);
  const int64_t T =
      THPVariable_Check(a[0]) && THPVariable_Unpack(a[0]).dim() == 3 ? THPVariable_Unpack(a[0]).size(0) : 0;
  const Cache c(a[2], a[3], a[4], a[5], T);
  const Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
  const int64_t ks = rows(k, c.Hkv, c.D, "k"), vs = rows(v, c.Hkv, c.D, "v");
  if (v.size(0) != T) value_error("k and v must have the same number of rows");
  same_device(k, v, c.cache, c.table, c.lens, c.cu);
  const qk_stream_t stream = stream_of(a[6]);
  check(unlocked([&] {
          return qk_kv4_append(ptr<uint16_t>(k), ks, ptr<uint16_t>(v), vs, T, c.Hkv, c.D, ptr<int32_t>(c.table), c.B,
                               c.max_pages, ptr<int32_t>(c.lens), ptr<int32_t>(c.cu), ptr<void>(c.cache), c.num_pages,
                               c.page, stream);
        }),
        "qk_kv4_append");
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// cache, page_table, kv_lens, cu_rows, T, k, v, stream
PyObject* kv4_gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 8);
  const int64_t T = integer(a[4]);
  if (T < 0) value_error("T must not be negative");
  const Cache c(a[0], a[1], a[2], a[3], T);
  const qk_stream_t stream = stream_of(a[7]);
  Together fresh(c.cache, stream);
  auto out = [&](PyObject* o, Tensor* t, const char* name, int64_t* stride) {
    *stride = c.Hkv * c.D;
    if (o == Py_None) {
      fresh.add(t, {T, c.Hkv, c.D}, ScalarType::BFloat16);
    } else {
      *t = tensor(o, name);
      *stride = rows(*t, c.Hkv, c.D, name);
    }
  };
  int64_t ks, vs;
  Tensor k, v;
  out(a[5], &k, "k", &ks);
  out(a[6], &v, "v", &vs);
  fresh.make();
  if (k.size(0) != T || v.size(0) != T) value_error("k and v must have " + std::to_string(T) + " rows");
  same_device(k, v, c.cache, c.table, c.lens, c.cu);
  check(unlocked([&] {
          return qk_kv4_gather(ptr<void>(c.cache), c.num_pages, c.page, c.Hkv, c.D, ptr<int32_t>(c.table), c.B,
                               c.max_pages, ptr<int32_t>(c.lens), ptr<int32_t>(c.cu), T, ptr<uint16_t>(k), ks,
                               ptr<uint16_t>(v), vs, stream);
        }),
        "qk_kv4_gather");
  return tuple_of({hand_back(a[5], k), hand_back(a[6], v)});
  END_HANDLE_TH_ERRORS
}

// q, cache, page_table, kv_lens, cu_rows, scale, window, sinks, out, workspace, stream
PyObject* kv4_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 11);
  const Tensor& q = rows_of_three(a[0], "q", "[T, H, D]");
  const int64_t T = q.size(0), H = q.size(1);
  const Cache c(a[1], a[2], a[3], a[4], T);
  const int64_t qs = rows(q, H, c.D, "q");
  const qk_stream_t stream = stream_of(a[10]);
  const Tensor out = output(a[8], {T, H, c.D}, ScalarType::BFloat16, q, "out", stream);
  // without a workspace: torch's allocator on the current stream; on another one the
  // library allocates in that stream's order
  Tensor ws;
  size_t ws_bytes = 0;
  if (a[9] != Py_None) {
    ws = tensor(a[9], "workspace");
    if (!ws.is_contiguous()) value_error("workspace must be contiguous");
    ws_bytes = ws.nbytes();
  } else if (a[10] == Py_None || stream == current_stream()) {
    ws_bytes = qk_kv4_attention_workspace_size(c.D);
    ws = output(Py_None, {(int64_t)ws_bytes}, ScalarType::Byte, q, "workspace", stream);
  }
  const double scale = a[5] == Py_None ? 1.0 / std::sqrt((double)c.D) : number(a[5]);
  same_device(q, out, ws, c.cache, c.table, c.lens, c.cu);
  const int64_t window = integer(a[6]), sinks = integer(a[7]);
  check(unlocked([&] {
          return qk_kv4_attention(ptr<uint16_t>(q), qs, T, H, c.Hkv, c.D, ptr<void>(c.cache), c.num_pages, c.page,
                                  ptr<int32_t>(c.table), c.B, c.max_pages, ptr<int32_t>(c.lens), ptr<int32_t>(c.cu),
                                  (float)scale, window, sinks, ptr<uint16_t>(out), ptr<void>(ws), ws_bytes, stream);
        }),
        "qk_kv4_attention");
  return hand_back(a[8], out);
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef methods[] = {
    {"rmsnorm_quantize", fast<rmsnorm_quantize>(), METH_FASTCALL, nullptr},
    {"rope", fast<rope>(), METH_FASTCALL, nullptr},
    {"kv4_append", fast<kv4_append>(), METH_FASTCALL, nullptr},
    {"kv4_gather", fast<kv4_gather>(), METH_FASTCALL, nullptr},
    {"kv4_attention", fast<kv4_attention>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block_calls() { return PyModule_Create(&module); }
