// The paged operators' Python calls (module _fast): the tensors' checks and the
// call of the C entry point in one step of native code.  A decode step's plan and
// store are shorter on the GPU (paged.cu) than the same checks in Python and a
// call through ctypes, which took 12 and 9 us.  Every function returns the entry point's
// status, or raises ValueError for a tensor of the wrong type, shape, layout or
// device.  Tensors must lie on the current device.
#include <Python.h>
#include <cuda_runtime_api.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "zaya.h"

namespace {

struct Args {
  PyObject* const* v;
  Py_ssize_t n;
  c10::DeviceIndex dev = -1;

  const at::Tensor& tensor(int i, const char* name) const {
    if (!THPVariable_Check(v[i])) throw std::invalid_argument(std::string(name) + ": a tensor is wanted");
    return THPVariable_Unpack(v[i]);
  }
  // The device of the call: the current one, which the first tensor has to be on.
  void here(int i, const char* name) {
    const at::Tensor& t = tensor(i, name);
    if (!t.is_cuda()) throw std::invalid_argument(std::string(name) + ": device tensors are wanted");
    dev = c10::cuda::current_device();
  }
  void check(bool ok, const char* name, const std::string& what) const {
    if (!ok) throw std::invalid_argument(std::string(name) + ": " + what + " on the current device is wanted");
  }
  bool local(const at::Tensor& t) const { return t.is_cuda() && t.get_device() == dev; }
  const at::Tensor& words(int i, const char* name, int64_t numel) const {
    const at::Tensor& t = tensor(i, name);
    check(t.scalar_type() == at::kInt && local(t) && t.is_contiguous() && (numel < 0 || t.numel() == numel), name,
          numel < 0 ? "a contiguous int32 tensor" : "a contiguous int32 tensor of " + std::to_string(numel));
    return t;
  }
  // What a call writes it takes through the mutable pointer, which gives a tensor that shares its
  // storage until it is written (a lazy clone) a storage of its own.
  const int32_t* ints(int i, const char* name, int64_t numel = -1) const {
    return static_cast<const int32_t*>(words(i, name, numel).const_data_ptr());
  }
  int32_t* ints_out(int i, const char* name, int64_t numel = -1) const {
    return static_cast<int32_t*>(words(i, name, numel).mutable_data_ptr());
  }
  // [B, max_pages]
  const at::Tensor& table(int i, int64_t B, int32_t* width) const {
    const at::Tensor& t = words(i, "block_table", -1);
    check(t.dim() == 2 && t.size(0) == B, "block_table", "int32 [" + std::to_string(B) + ", max_pages]");
    *width = count(t.size(1));
    return t;
  }
  // bf16 [T, heads, d] with contiguous heads, tokens any stride apart
  const at::Tensor& rows_of(int i, const char* name, int64_t T, int64_t heads, int64_t d, int32_t* stride) const {
    const at::Tensor& t = tensor(i, name);
    check(t.scalar_type() == at::kBFloat16 && local(t) && t.dim() == 3 && t.size(0) == T && t.size(1) == heads &&
              t.size(2) == d && t.stride(2) == 1 && (heads == 1 || t.stride(1) == d),
          name, "bf16 [" + std::to_string(T) + ", " + std::to_string(heads) + ", " + std::to_string(d) + "] with contiguous heads");
    *stride = count(T > 1 ? t.stride(0) : heads * d);
    return t;
  }
  const void* rows(int i, const char* name, int64_t T, int64_t heads, int64_t d, int32_t* stride) const {
    return rows_of(i, name, T, heads, d, stride).const_data_ptr();
  }
  void* rows_out(int i, const char* name, int64_t T, int64_t heads, int64_t d, int32_t* stride) const {
    return rows_of(i, name, T, heads, d, stride).mutable_data_ptr();
  }
  const at::Tensor& plain(int i, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) const {
    const at::Tensor& t = tensor(i, name);
    std::string want;
    for (int64_t s : shape) want += (want.empty() ? "" : ", ") + std::to_string(s);
    check(t.scalar_type() == type && local(t) && t.is_contiguous() && t.sizes() == c10::IntArrayRef(shape), name,
          "a contiguous " + std::string(c10::toString(type)) + " [" + want + "]");
    return t;
  }
  void* workspace(int i, size_t* bytes) const {
    const at::Tensor& t = tensor(i, "workspace");
    check(local(t) && t.is_contiguous(), "workspace", "a contiguous tensor");
    *bytes = t.nbytes();
    return t.mutable_data_ptr();
  }
  static int32_t count(int64_t x) {
    if (x > INT32_MAX || x < INT32_MIN) throw std::invalid_argument("a size or stride is beyond 32 bits");
    return static_cast<int32_t>(x);
  }
  int32_t integer(int i) const {
    const long x = PyLong_AsLong(v[i]);
    if (x == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      throw std::invalid_argument("an integer is wanted");
    }
    return count(x);
  }
  // a ctypes structure's address
  template <class T>
  const T* at_address(int i) const {
    const T* p = static_cast<const T*>(PyLong_AsVoidPtr(v[i]));
    if (!p && PyErr_Occurred()) PyErr_Clear();
    return p;
  }
  bool none(int i) const { return v[i] == Py_None; }
  // the stream given as an address, or the device's current one
  void* stream(int i) const {
    return none(i) ? static_cast<void*>(c10::cuda::getCurrentCUDAStream(dev).stream()) : PyLong_AsVoidPtr(v[i]);
  }
};

// The C entry points run without the interpreter's lock, as through ctypes: a launch waits where
// the device's queue is full.  What touches Python objects is done before.
template <class F>
int unlocked(F&& f) {
  PyThreadState* st = PyEval_SaveThread();
  const int rc = f();   // C: raises nothing
  PyEval_RestoreThread(st);
  return rc;
}

template <class F>
PyObject* call(PyObject* const* v, Py_ssize_t n, Py_ssize_t want, F&& f) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    Args a{v, n};
    return PyLong_FromLong(f(a));
  } catch (const std::exception& e) {   // nothing may cross into C
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
}

PyObject* paged_plan(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return call(v, n, 15, [](Args& a) {
    a.here(0, "ctx_len");
    const int64_t B = a.tensor(0, "ctx_len").numel(), T = a.tensor(10, "slot_map").numel();
    int32_t width;
    size_t bytes;
    int32_t* table = static_cast<int32_t*>(a.table(3, B, &width).mutable_data_ptr());
    void* ws = a.workspace(13, &bytes);
    const int32_t rows = Args::count(B), tokens = Args::count(T), n_pages = Args::count(a.tensor(4, "free_list").numel());
    const int32_t *ctx = a.ints(0, "ctx_len"), *fresh = a.ints(1, "new_len", B);
    const int32_t* drop = a.none(2) ? nullptr : a.ints(2, "drop_len", B);
    int32_t* free_list = a.ints_out(4, "free_list");
    const int32_t* n_in = a.ints(5, "n_free_in", 1);
    int32_t* n_out = a.ints_out(6, "n_free_out", 1);
    const int32_t page = a.integer(7);
    int32_t *cu = a.ints_out(8, "cu_new", B + 1), *seq = a.ints_out(9, "seq_len", B), *slots = a.ints_out(10, "slot_map");
    int32_t *pos = a.ints_out(11, "positions", T), *row = a.ints_out(12, "token_row", T);
    void* stream = a.stream(14);
    return unlocked([&] {
      return zaya_paged_plan(rows, tokens, ctx, fresh, drop, table, width, free_list, n_pages, n_in, n_out, page, cu, seq, slots, pos,
                             row, ws, bytes, stream);
    });
  });
}

PyObject* paged_store(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return call(v, n, 7, [](Args& a) {
    a.here(3, "slot_map");
    const auto* c = a.at_address<zaya_config>(0);
    const int64_t T = a.tensor(3, "slot_map").numel();
    int32_t ks, vs;
    size_t bytes;
    const void* k = a.rows(1, "k", T, c->n_kv, c->head_dim, &ks);
    const void* val = a.rows(2, "v", T, c->n_kv, c->head_dim, &vs);
    void* ws = a.workspace(5, &bytes);
    const int32_t tokens = Args::count(T), *slots = a.ints(3, "slot_map");
    const auto* kv = a.at_address<zaya_paged_kv>(4);
    void* stream = a.stream(6);
    return unlocked([&] { return zaya_paged_store(c, tokens, k, ks, val, vs, slots, kv, ws, bytes, stream); });
  });
}

PyObject* paged_attention(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return call(v, n, 10, [](Args& a) {
    a.here(2, "q");
    const auto* c = a.at_address<zaya_config>(0);
    const int64_t B = a.tensor(4, "seq_len").numel(), T = a.tensor(2, "q").dim() ? a.tensor(2, "q").size(0) : 0;
    int32_t qs, os, width;
    size_t bytes;
    const void* q = a.rows(2, "q", T, c->n_q, c->head_dim, &qs);
    void* out = a.rows_out(7, "out", T, c->n_q, c->head_dim, &os);
    const auto* table = static_cast<const int32_t*>(a.table(5, B, &width).const_data_ptr());
    void* ws = a.workspace(8, &bytes);
    const int32_t window = a.integer(1), rows = Args::count(B), tokens = Args::count(T);
    const int32_t *cu = a.ints(3, "cu_new", B + 1), *seq = a.ints(4, "seq_len");
    const auto* kv = a.at_address<zaya_paged_kv>(6);
    void* stream = a.stream(9);
    return unlocked([&] {
      return zaya_paged_attention(c, window, rows, tokens, q, qs, cu, seq, table, width, kv, out, os, ws, bytes, stream);
    });
  });
}

PyObject* packed_attention(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return call(v, n, 9, [](Args& a) {
    a.here(2, "q");
    const auto* c = a.at_address<zaya_config>(0);
    const int64_t B = a.tensor(5, "cu_new").numel() - 1, T = a.tensor(2, "q").dim() ? a.tensor(2, "q").size(0) : 0;
    int32_t qs, ks, vs, os;
    size_t bytes;
    const void* q = a.rows(2, "q", T, c->n_q, c->head_dim, &qs);
    const void* k = a.rows(3, "k", T, c->n_kv, c->head_dim, &ks);
    const void* val = a.rows(4, "v", T, c->n_kv, c->head_dim, &vs);
    void* out = a.rows_out(6, "out", T, c->n_q, c->head_dim, &os);
    void* ws = a.workspace(7, &bytes);
    const int32_t window = a.integer(1), rows = Args::count(B), tokens = Args::count(T), *cu = a.ints(5, "cu_new");
    void* stream = a.stream(8);
    return unlocked([&] {
      return zaya_packed_attention(c, window, rows, tokens, q, qs, k, ks, val, vs, cu, out, os, ws, bytes, stream);
    });
  });
}

PyObject* block_paged(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return call(v, n, 18, [](Args& a) {
    a.here(3, "hidden");
    const auto* c = a.at_address<zaya_config>(0);
    const int64_t B = a.tensor(5, "seq_len").numel(), T = a.tensor(6, "slot_map").numel();
    const auto* state = a.at_address<zaya_paged_state>(12);
    int32_t width;
    size_t bytes;
    a.plain(13, "conv_state", at::kBFloat16, {B, int64_t(c->n_q + c->n_kv) * c->head_dim, 2});
    a.plain(14, "prev_hs", at::kBFloat16, {B, c->hidden});
    const auto* table = static_cast<const int32_t*>(a.table(8, B, &width).const_data_ptr());
    void* ws = a.workspace(16, &bytes);
    float* hidden = static_cast<float*>(a.plain(3, "hidden", at::kFloat, {T, c->hidden}).mutable_data_ptr());
    const float* rin = nullptr;
    if (!a.none(10))
      rin = static_cast<const float*>(a.plain(10, "router_state_in", at::kFloat, {T, c->router_hidden}).const_data_ptr());
    float* rout = static_cast<float*>(a.plain(11, "router_state_out", at::kFloat, {T, c->router_hidden}).mutable_data_ptr());
    const auto* weights = a.at_address<zaya_block_weights>(1);
    const int32_t block = a.integer(2), rows = Args::count(B), tokens = Args::count(T), fresh = a.integer(9);
    const int32_t *cu = a.ints(4, "cu_new", B + 1), *seq = a.ints(5, "seq_len"), *slots = a.ints(6, "slot_map");
    const int32_t* row = a.ints(7, "token_row", T);
    const auto* taps = a.none(15) ? nullptr : a.at_address<zaya_taps>(15);
    void* stream = a.stream(17);
    return unlocked([&] {
      return zaya_block_paged(c, weights, block, rows, tokens, hidden, cu, seq, slots, row, table, width, fresh, rin, rout, state, taps,
                              ws, bytes, stream);
    });
  });
}

PyMethodDef kMethods[] = {
    {"paged_plan", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_plan)), METH_FASTCALL, nullptr},
    {"paged_store", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_store)), METH_FASTCALL, nullptr},
    {"paged_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_attention)), METH_FASTCALL, nullptr},
    {"packed_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(packed_attention)), METH_FASTCALL, nullptr},
    {"block_paged", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(block_paged)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast() { return PyModule_Create(&kModule); }
